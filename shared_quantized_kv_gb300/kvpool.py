"""ctypes binding of ``libkvpool.so`` (argument marshalling only).

Every step of the path runs in the library's CUDA kernels; this module only
turns torch tensors into device pointers and the current torch stream into a
``cudaStream_t``. There is no fallback: if the library is missing or the
device is not an sm_103 GPU the calls raise.
"""

from __future__ import annotations

import contextlib
import ctypes
import operator
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libkvpool.so")

OK = 0
ERRORS = {
    -1: "INVALID_ARG", -2: "STATE", -3: "CUDA", -4: "OOM", -5: "NONFINITE", -6: "TIMEOUT",
    -7: "UNSUPPORTED",
}


class KVPoolError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: {ERRORS.get(code, code)} ({_lib().kvpool_strerror(code).decode()})")


class Tail(ctypes.Structure):
    _fields_ = [("K", ctypes.c_void_p), ("V", ctypes.c_void_p), ("len", ctypes.c_void_p),
                ("T_max", ctypes.c_int)]


class Pages(ctypes.Structure):
    _fields_ = [("K", ctypes.c_void_p), ("V", ctypes.c_void_p), ("layers", ctypes.c_int), ("pages", ctypes.c_int),
                ("kv_heads", ctypes.c_int), ("page_tokens", ctypes.c_int), ("head_dim", ctypes.c_int),
                ("status", ctypes.c_void_p)]


class Seqs(ctypes.Structure):
    _fields_ = [("seqs", ctypes.c_int), ("table_stride", ctypes.c_int), ("page_table", ctypes.c_void_p),
                ("kv_len", ctypes.c_void_p), ("q_start", ctypes.c_void_p), ("tokens", ctypes.c_int),
                ("max_q", ctypes.c_int), ("max_kv", ctypes.c_int)]


class Score(ctypes.Structure):
    _fields_ = [("cap", ctypes.c_float), ("window", ctypes.c_int), ("slopes", ctypes.c_void_p),
                ("first", ctypes.c_void_p), ("prefix", ctypes.c_void_p)]


class LayerView(ctypes.Structure):
    _fields_ = [("kq", ctypes.c_void_p), ("vcodes", ctypes.c_void_p), ("vnorm", ctypes.c_void_p),
                ("kscale", ctypes.c_void_p), ("ctx", ctypes.c_int), ("ctx_padded", ctypes.c_int),
                ("bits", ctypes.c_int), ("compressed", ctypes.c_int),
                ("kscales", ctypes.c_void_p), ("k_block", ctypes.c_int), ("len", ctypes.c_int),
                ("group_bits", ctypes.c_void_p), ("group_off", ctypes.c_void_p), ("mixed", ctypes.c_int)]


_LIB = None

# name -> (restype, argtypes); the C declarations are in include/kvpool.h
_SIGS = {
    "kvpool_create": (ctypes.c_int, [ctypes.POINTER(ctypes.c_void_p), ctypes.c_int, ctypes.c_int,
                                     ctypes.c_int, ctypes.c_int, ctypes.c_void_p, ctypes.c_int]),
    "kvpool_create_ex": (ctypes.c_int, [ctypes.POINTER(ctypes.c_void_p), ctypes.c_int, ctypes.c_int,
                                        ctypes.c_int, ctypes.c_int, ctypes.c_void_p, ctypes.c_int,
                                        ctypes.c_int]),
    "kvpool_export_kscales": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p]),
    "kvpool_append": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p,
                                     ctypes.c_int, ctypes.c_void_p]),
    "kvpool_append_bits": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p,
                                          ctypes.c_int, ctypes.c_int, ctypes.c_void_p]),
    "kvpool_layer_widths": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p, ctypes.c_int]),
    "kvpool_layer_len": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int]),
    "kvpool_sensitivity": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_int, ctypes.c_void_p,
                                          ctypes.c_int, ctypes.c_int, ctypes.c_float, ctypes.c_void_p,
                                          ctypes.c_void_p, ctypes.c_void_p]),
    "kvpool_allocate_bits": (ctypes.c_int, [ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64,
                                            ctypes.c_void_p]),
    "kvpool_destroy": (None, [ctypes.c_void_p]),
    "kvpool_compress": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p,
                                       ctypes.c_void_p, ctypes.c_void_p]),
    "kvpool_attend": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p, ctypes.c_int,
                                     ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p,
                                     ctypes.c_float, ctypes.c_void_p]),
    "kvpool_decompress": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p,
                                         ctypes.c_void_p, ctypes.c_void_p]),
    "kvpool_compress_layers": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p,
                                              ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "kvpool_decompress_layers": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p,
                                                ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "kvpool_pool_bytes": (ctypes.c_size_t, [ctypes.c_void_p]),
    "kvpool_device_bytes": (ctypes.c_size_t, [ctypes.c_void_p]),
    "kvpool_status": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p]),
    "kvpool_reset_layer": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int]),
    "kvpool_layer_view": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.POINTER(LayerView)]),
    "kvpool_codebook": (ctypes.c_int, [ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p]),
    "kvpool_export_layer": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int] + [ctypes.c_void_p] * 5),
    "kvpool_import_layer": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int] + [ctypes.c_void_p] * 5),
    "kvpool_import_layer_blocks": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int] + [ctypes.c_void_p] * 5 +
                                   [ctypes.c_int, ctypes.c_void_p]),
    "kvpool_attend_noalloc": (ctypes.c_int, [ctypes.c_void_p] * 5 + [ctypes.c_int] * 4 +
                              [ctypes.c_void_p, ctypes.c_int, ctypes.c_int, ctypes.c_void_p,
                               ctypes.c_void_p, ctypes.c_float, ctypes.c_void_p]),
    "kvpool_attend_ws": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p, ctypes.c_int,
                                        ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_float,
                                        ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "kvpool_attend_ws_bytes": (ctypes.c_size_t, [ctypes.c_void_p, ctypes.c_int, ctypes.c_int]),
    "kvpool_attend_partial": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p, ctypes.c_int,
                                             ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_void_p,
                                             ctypes.c_void_p, ctypes.c_float, ctypes.c_void_p]),
    "kvpool_merge_partials": (ctypes.c_int, [ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int,
                                             ctypes.c_int, ctypes.c_void_p, ctypes.c_int, ctypes.c_int,
                                             ctypes.c_void_p, ctypes.c_void_p, ctypes.c_float,
                                             ctypes.c_void_p]),
    "kvpool_pages_append": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p,
                                           ctypes.c_longlong, ctypes.c_void_p, ctypes.c_longlong,
                                           ctypes.c_void_p]),
    "kvpool_pages_copy": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int,
                                         ctypes.c_void_p]),
    "kvpool_pages_attend": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p,
                                           ctypes.c_longlong, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p,
                                           ctypes.c_void_p, ctypes.c_float, ctypes.c_void_p]),
    "kvpool_attend_pages": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p, ctypes.c_int,
                                           ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p,
                                           ctypes.c_float, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "kvpool_attend_pages_ws_bytes": (ctypes.c_size_t, [ctypes.c_void_p, ctypes.c_int, ctypes.c_int]),
    "kvpool_pages_status": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p]),
    "kvpool_pager_create": (ctypes.c_int, [ctypes.POINTER(ctypes.c_void_p), ctypes.c_int, ctypes.c_int]),
    "kvpool_pager_destroy": (None, [ctypes.c_void_p]),
    "kvpool_pager_new": (ctypes.c_int, [ctypes.c_void_p]),
    "kvpool_pager_extend": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_int, ctypes.c_void_p]),
    "kvpool_pager_truncate": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_int]),
    "kvpool_pager_fork": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int]),
    "kvpool_pager_free": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int]),
    "kvpool_pager_compact": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int]),
    "kvpool_pager_len": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int]),
    "kvpool_pager_table": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p, ctypes.c_int]),
    "kvpool_pager_free_pages": (ctypes.c_int, [ctypes.c_void_p]),
    "kvpool_pager_owners": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int]),
    "kvpool_strerror": (ctypes.c_char_p, [ctypes.c_int]),
}


def _lib():
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m shared_quantized_kv_gb300.build`")
        lib = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _LIB = lib
    return _LIB


def lib():
    """The loaded library (ctypes.CDLL)."""
    return _lib()


def _check(rc: int, what: str):
    if rc != OK:
        raise KVPoolError(rc, what)


def _stream_ptr(stream):
    import torch

    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _dev_ptr(t, dtype, name):
    import torch

    if t is None:
        return None
    if not t.is_cuda or t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor of {dtype}")
    return ctypes.c_void_p(t.data_ptr())


def codebook(bits: int):
    """The library's float32 (centroids, midpoints) for ``bits`` (host)."""
    import numpy as np

    c = np.zeros(1 << bits, np.float32)
    m = np.zeros((1 << bits) - 1, np.float32)
    _check(_lib().kvpool_codebook(bits, c.ctypes.data, m.ctypes.data), "kvpool_codebook")
    return c, m


def sensitivity(Q, recent, kv_heads, softmax_scale=0.0, stream=None):
    """A layer's local attention-error estimate s (float) and the per-row
    values r (float32 [agents * q_heads], device) from recent tokens: Q bf16
    [agents, q_heads, d]; recent = (K, V, lens) with K, V bf16 [agents,
    kv_heads, T_max, d] and lens int32 [agents] (device)."""
    import torch

    A, Hq, d = Q.shape
    K, V, lens = recent
    t = Tail(_dev_ptr(K, torch.bfloat16, "recent K").value, _dev_ptr(V, torch.bfloat16, "recent V").value,
             _dev_ptr(lens, torch.int32, "recent len").value, K.shape[2])
    rows = torch.empty(A * Hq, dtype=torch.float32, device=Q.device)
    score = torch.empty(1, dtype=torch.float32, device=Q.device)
    _check(_lib().kvpool_sensitivity(_dev_ptr(Q, torch.bfloat16, "Q"), A, Hq, ctypes.byref(t), kv_heads, d,
                                     softmax_scale, rows.data_ptr(), score.data_ptr(), _stream_ptr(stream)),
           "kvpool_sensitivity")
    return float(score.cpu()[0]), rows


def merge_partials(ml, acc, Q, kv_heads, tail=None, out=None, softmax_scale=0.0, stream=None):
    """kvpool_merge_partials: ml float32 [parts, kv_heads, rows, 2] and acc
    float32 [parts, kv_heads, rows, d] from attend_partial (device); Q bf16
    [agents, q_heads, d]; tail None or (K, V, lens) as for attend. Returns out
    float32 [agents, q_heads, d]."""
    import torch

    A, Hq, d = Q.shape
    parts = ml.shape[0]
    if out is None:
        out = torch.empty((A, Hq, d), dtype=torch.float32, device=Q.device)
    tp = None
    if tail is not None:
        Kt, Vt, lens = tail
        t = Tail(_dev_ptr(Kt, torch.bfloat16, "tail K").value, _dev_ptr(Vt, torch.bfloat16, "tail V").value,
                 _dev_ptr(lens, torch.int32, "tail len").value, Kt.shape[2])
        tp = ctypes.byref(t)
    _check(_lib().kvpool_merge_partials(parts, _dev_ptr(ml, torch.float32, "ml"), _dev_ptr(acc, torch.float32, "acc"),
                                        kv_heads, d, _dev_ptr(Q, torch.bfloat16, "Q"), A, Hq, tp,
                                        _dev_ptr(out, torch.float32, "out"), softmax_scale, _stream_ptr(stream)),
           "kvpool_merge_partials")
    return out


def allocate_bits(sens, cost, budget):
    """Per-layer V widths (list of 2, 3, 4) minimising sum D_b s^2 within
    sum cost * bits <= budget (host only)."""
    import numpy as np

    L = len(sens)
    s = np.ascontiguousarray(sens, dtype=np.float64)
    c = np.ascontiguousarray(cost, dtype=np.int64)
    out = np.zeros(L, dtype=np.uint8)
    _check(_lib().kvpool_allocate_bits(L, s.ctypes.data, c.ctypes.data, int(budget), out.ctypes.data),
           "kvpool_allocate_bits")
    return [int(b) for b in out]


# ------------------------------------------------------- paged private caches

class Pager:
    """Which pages each sequence owns (a ``kvpool_pager_t``; host only)."""

    def __init__(self, pages, page_tokens):
        h = ctypes.c_void_p()
        _check(_lib().kvpool_pager_create(ctypes.byref(h), _i32(pages, "pages"), _i32(page_tokens, "page_tokens")),
               "kvpool_pager_create")
        self._h, self.pages, self.page_tokens = h, pages, page_tokens

    @property
    def handle(self):
        return self._h

    def close(self):
        if getattr(self, "_h", None):
            _lib().kvpool_pager_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    @staticmethod
    def _count(n, what):
        """n of a call that returns a count or a negative error code."""
        _check(min(0, n), what)
        return n

    def new(self) -> int:
        """A new empty sequence's number."""
        return self._count(_lib().kvpool_pager_new(self._h), "kvpool_pager_new")

    def extend(self, seq, n):
        """Room for n more tokens: None, or the (shared page, own page) pair
        that has to be copied before they are written."""
        pair = (ctypes.c_int32 * 2)()
        due = self._count(_lib().kvpool_pager_extend(self._h, _i32(seq, "seq"), _i32(n, "n"), pair),
                          "kvpool_pager_extend")
        return (pair[0], pair[1]) if due else None

    def truncate(self, seq, length):
        """Cut a sequence to its first `length` tokens."""
        _check(_lib().kvpool_pager_truncate(self._h, _i32(seq, "seq"), _i32(length, "length")), "kvpool_pager_truncate")

    def fork(self, seq) -> int:
        """A new sequence that shares all pages of seq."""
        return self._count(_lib().kvpool_pager_fork(self._h, _i32(seq, "seq")), "kvpool_pager_fork")

    def free(self, seq):
        """End a sequence."""
        _check(_lib().kvpool_pager_free(self._h, _i32(seq, "seq")), "kvpool_pager_free")

    def compact(self):
        """Owned pages become the lowest numbers: lists (src, dst) of the page copies due."""
        src, dst = (ctypes.c_int32 * self.pages)(), (ctypes.c_int32 * self.pages)()
        n = self._count(_lib().kvpool_pager_compact(self._h, src, dst, self.pages), "kvpool_pager_compact")
        return list(src[:n]), list(dst[:n])

    def length(self, seq) -> int:
        return self._count(_lib().kvpool_pager_len(self._h, _i32(seq, "seq")), "kvpool_pager_len")

    def table(self, seq):
        """The sequence's pages in order (list of int)."""
        seq = _i32(seq, "seq")
        n = self._count(_lib().kvpool_pager_table(self._h, seq, None, 0), "kvpool_pager_table")
        buf = (ctypes.c_int32 * max(n, 1))()
        self._count(_lib().kvpool_pager_table(self._h, seq, buf, n), "kvpool_pager_table")
        return list(buf[:n])

    def free_pages(self) -> int:
        return self._count(_lib().kvpool_pager_free_pages(self._h), "kvpool_pager_free_pages")

    def owners(self, page) -> int:
        """Sequences that own the page (0: free)."""
        return self._count(_lib().kvpool_pager_owners(self._h, _i32(page, "page")), "kvpool_pager_owners")


def _i32(x, name):
    """The whole number x, which ctypes would cut to 32 bits without a word."""
    x = operator.index(x)
    if not -(1 << 31) <= x < 1 << 31:
        raise ValueError(f"{name} must fit 32 bits, not {x}")
    return x


def _here():
    """The current CUDA device's number."""
    import torch

    return torch.cuda.current_device()


def _need(t, dtype, name, dev):
    """Address of a contiguous tensor of dtype on device dev (these calls are
    short: a step makes one per layer)."""
    if t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor of {dtype} on the current CUDA device ({dev}), "
                         f"not {t.dtype} on {t.device}")
    return t.data_ptr()


def _raw_stream(stream, dev):
    """cudaStream_t of `stream`, or of the current stream."""
    import torch

    if stream is None:
        return torch.cuda.current_stream(dev).cuda_stream
    if stream.device.index != dev:
        raise ValueError(f"stream must be one of the current CUDA device ({dev})")
    return stream.cuda_stream


def _pages(K_pages, V_pages, status=None, dev=None):
    import torch

    dev = _here() if dev is None else dev
    shape = K_pages.shape
    if len(shape) != 5 or V_pages.shape != shape:
        raise ValueError("K_pages and V_pages must be [layers, pages, kv_heads, page_tokens, head_dim]")
    return Pages(_need(K_pages, torch.bfloat16, "K_pages", dev), _need(V_pages, torch.bfloat16, "V_pages", dev), *shape,
                 None if status is None else _need(status, torch.int32, "status", dev))


def _seqs(table, kv_len, q_start, tokens, max_q, max_kv, dev=None):
    import torch

    dev = _here() if dev is None else dev
    shape = table.shape
    if len(shape) != 2 or kv_len.shape != shape[:1] or q_start.dim() != 1 or q_start.shape[0] != shape[0] + 1:
        raise ValueError("table [seqs, pages], kv_len [seqs] and q_start [seqs + 1] do not fit together")
    i32 = torch.int32
    return Seqs(shape[0], shape[1], _need(table, i32, "table", dev), _need(kv_len, i32, "kv_len", dev),
                _need(q_start, i32, "q_start", dev), tokens, _i32(max_q or 0, "max_q"), _i32(max_kv or 0, "max_kv"))


def _token_rows(t, name, heads, d, dev):
    """Address and token stride of a bf16 [tokens, heads, d] tensor whose heads lie together."""
    import torch

    shape, stride = t.shape, t.stride()
    if len(shape) != 3 or shape[1] != heads or shape[2] != d or t.dtype is not torch.bfloat16 or \
            t.get_device() != dev or stride[2] != 1 or (heads > 1 and stride[1] != d):
        raise ValueError(f"{name} must be a bf16 tensor [tokens, {heads}, {d}] on the current CUDA device ({dev}) whose "
                         "heads lie together")
    return t.data_ptr(), stride[0] if shape[0] > 1 else heads * d


def _check_rows(rows, batch):
    """Fewer rows than the batch has would be taken for the last tokens of their sequence."""
    if rows.shape[0] < batch.tokens:
        raise ValueError(f"a batch of {batch.tokens} tokens takes as many rows at least, not {rows.shape[0]}")


def pages_append(K_pages, V_pages, layer, K, V, table, kv_len, q_start, status=None, stream=None):
    """Write new tokens into their pages (kvpool_pages_append). K_pages,
    V_pages: bf16 [layers, pages, kv_heads, page_tokens, d]; K, V: bf16
    [tokens, kv_heads, d], rows of a fused projection as they are; table int32
    [seqs, pages of a sequence], kv_len int32 [seqs] (the new tokens included),
    q_start int32 [seqs + 1]: sequence s's new tokens are rows q_start[s] ...
    q_start[s + 1] - 1. status: None or an int32 [1] word that records page
    numbers out of range and sequences longer than their table has room for,
    whose tokens are dropped. All on the current device."""
    layer = _i32(layer, "layer")
    dev = _here()
    pg = _pages(K_pages, V_pages, status, dev)
    n = K.shape[0]
    if V.shape[0] != n:
        raise ValueError("K and V must have the same shape")
    kp, ks = _token_rows(K, "K", pg.kv_heads, pg.head_dim, dev)
    vp, vs = _token_rows(V, "V", pg.kv_heads, pg.head_dim, dev)
    sq = _seqs(table, kv_len, q_start, n, 0, 0, dev)
    _check(_lib().kvpool_pages_append(ctypes.byref(pg), layer, ctypes.byref(sq), kp, ks, vp, vs,
                                      _raw_stream(stream, dev)), "kvpool_pages_append")


def pages_copy(K_pages, V_pages, src, dst, stream=None):
    """Page dst[i] of every layer becomes page src[i] (kvpool_pages_copy);
    src, dst: lists of int. No page twice a destination, or both."""
    n = len(src)
    if len(dst) != n:
        raise ValueError("src and dst must have the same length")
    for x in (src, dst) if n else ():
        _i32(min(x), "page"), _i32(max(x), "page")
    dev = _here()
    arr = ctypes.c_int32 * max(n, 1)
    pg = _pages(K_pages, V_pages, None, dev)
    _check(_lib().kvpool_pages_copy(ctypes.byref(pg), arr(*src), arr(*dst), n, _raw_stream(stream, dev)),
           "kvpool_pages_copy")


def pages_attend(K_pages, V_pages, layer, Q, table, kv_len, q_start, max_q=None, max_kv=None, cap=0.0, slopes=None,
                 window=0, first=None, prefix=None, out=None, lse=None, return_lse=False, softmax_scale=0.0, status=None,
                 stream=None):
    """Attention of the new tokens over their sequences' pages
    (kvpool_pages_attend): Q bf16 [tokens, q_heads, d]; pages, table, kv_len,
    q_start as for pages_append. max_q, max_kv: the most new and held tokens of
    a sequence where the caller knows them (they choose kernels, not results).
    Scores: cap (x = cap tanh(x / cap)), slopes float32 [q_heads] (minus slope
    times distance), window (the last keys up to the row's own), first int32
    [tokens] (document mask: no key before it is seen, of a prefix neither),
    prefix int32 [seqs] (keys that every row sees from first on).
    Returns out bf16 [tokens, q_heads, d], or (out, lse float32 [tokens,
    q_heads]) with return_lse or an lse to write to. A row that sees no key
    gets 0 and -inf; rows behind the last sequence are left as they are."""
    import torch

    layer = _i32(layer, "layer")
    dev = _here()
    pg = _pages(K_pages, V_pages, status, dev)
    if Q.dim() != 3:
        raise ValueError("Q must be [tokens, q_heads, head_dim]")
    n, hq, d = Q.shape
    qp, qs = _token_rows(Q, "Q", hq, pg.head_dim, dev)
    sq = _seqs(table, kv_len, q_start, n, max_q, max_kv, dev)

    def given(t, dtype, name, *shape):
        if t is None:
            return None
        if tuple(t.shape) != shape:
            raise ValueError(f"{name} must have shape {shape}")
        return _need(t, dtype, name, dev)

    sc = None
    if cap or window or slopes is not None or first is not None or prefix is not None:
        sc = ctypes.byref(Score(cap, _i32(window, "window"), given(slopes, torch.float32, "slopes", hq),
                                given(first, torch.int32, "first", n), given(prefix, torch.int32, "prefix", sq.seqs)))
    raw = _raw_stream(stream, dev)
    op, lp = given(out, torch.bfloat16, "out", n, hq, d), given(lse, torch.float32, "lse", n, hq)
    if op is None or (return_lse and lp is None):
        # on the stream that writes them, so that the allocator knows it
        with contextlib.nullcontext() if stream is None else torch.cuda.stream(stream):
            if op is None:
                out = torch.empty((n, hq, d), dtype=torch.bfloat16, device=Q.device)
                op = out.data_ptr()
            if return_lse and lp is None:
                lse = torch.empty((n, hq), dtype=torch.float32, device=Q.device)
                lp = lse.data_ptr()
    _check(_lib().kvpool_pages_attend(ctypes.byref(pg), layer, ctypes.byref(sq), qp, qs, hq, sc, op, lp, softmax_scale,
                                      raw), "kvpool_pages_attend")
    return out if lse is None else (out, lse)


class PagedCache:
    """The agents' private caches: bf16 pages of every layer (K, V tensors
    [layers, pages, kv_heads, page_tokens, head_dim]) on the current CUDA
    device, and the pager that says whose they are. Page copies that a fork or
    a compaction makes due are enqueued before the call returns."""

    def __init__(self, layers, kv_heads, head_dim, pages, page_tokens=64):
        import torch

        self.pager = Pager(pages, page_tokens)
        shape = (layers, pages, kv_heads, page_tokens, head_dim)
        self.K = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
        self.V = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
        self.status_word = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.page_tokens = page_tokens

    def close(self):
        self.pager.close()

    def new(self) -> int:
        """A new empty sequence's number."""
        return self.pager.new()

    def fork(self, seq) -> int:
        """A new sequence with seq's tokens, which stay shared until one of the two writes."""
        return self.pager.fork(seq)

    def free(self, seq):
        """End a sequence; pages that no other owns are free."""
        self.pager.free(seq)

    def truncate(self, seq, length):
        """Cut a sequence to its first `length` tokens."""
        self.pager.truncate(seq, length)

    def _usable(self, stream):
        """Another device's cache or stream is refused, before the pager has changed anything."""
        dev = _here()
        _pages(self.K, self.V, self.status_word, dev)
        _raw_stream(stream, dev)

    def compact(self, stream=None):
        """Move owned pages into the lowest numbers; how many moved. Batches
        made before are void."""
        self._usable(stream)
        src, dst = self.pager.compact()
        pages_copy(self.K, self.V, src, dst, stream)
        return len(src)

    def grow(self, seqs, counts, stream=None):
        """Room for counts[i] new tokens at the end of seqs[i]: the batch that
        append and attend take, rows in this order. Fewer free pages than it
        takes: KVPoolError (OOM). Whatever it raises, no sequence has grown."""
        if len(seqs) != len(counts) or not len(seqs) or len(set(seqs)) != len(seqs):
            raise ValueError("one count per sequence, each sequence once")
        counts = [_i32(n, "counts") for n in counts]
        self._usable(stream)
        before = [self.pager.length(s) for s in seqs]
        src, dst = [], []
        try:
            for s, n in zip(seqs, counts):
                pair = self.pager.extend(s, n)
                if pair:
                    src.append(pair[0])
                    dst.append(pair[1])
            pages_copy(self.K, self.V, src, dst, stream)
            return PagedBatch(self, seqs, counts, stream)
        except BaseException:
            # (a page of its own that a sequence got already is copied and kept)
            for s, n in zip(seqs, before):
                self.pager.truncate(s, n)
            live = [(a, b) for a, b in zip(src, dst) if self.pager.owners(b)]
            pages_copy(self.K, self.V, [a for a, _ in live], [b for _, b in live], stream)
            raise

    def append(self, layer, K, V, batch, stream=None):
        """Write the batch's new tokens: K, V bf16 [tokens, kv_heads, d] (rows behind the batch's are padding)."""
        _check_rows(K, batch)
        pages_append(self.K, self.V, layer, K, V, batch.table, batch.kv_len, batch.q_start, self.status_word, stream)

    def attend(self, layer, Q, batch, **options):
        """pages_attend of the batch's new tokens over their sequences (rows behind the batch's are padding)."""
        _check_rows(Q, batch)
        return pages_attend(self.K, self.V, layer, Q, batch.table, batch.kv_len, batch.q_start, batch.max_q,
                            batch.max_kv, status=self.status_word, **options)

    def status(self, stream=None) -> int:
        """Synchronise and return (and clear) the device status code of the pages' calls."""
        pg = _pages(self.K, self.V, self.status_word)
        return int(_lib().kvpool_pages_status(ctypes.byref(pg), _stream_ptr(stream)))


class PagedBatch:
    """The sequences of one step, as the calls take them: table, kv_len and
    q_start (device), max_q and max_kv (host)."""

    def __init__(self, cache, seqs, counts, stream=None):
        import torch

        tables = [cache.pager.table(s) for s in seqs]
        lens = [cache.pager.length(s) for s in seqs]
        width = max(1, max(len(t) for t in tables))
        start = [0]
        for n in counts:
            start.append(start[-1] + n)
        host = torch.tensor([x for t in tables for x in t + [-1] * (width - len(t))] + lens + start, dtype=torch.int32)
        with torch.cuda.stream(stream):
            dev = host.to(cache.K.device)  # one copy
        n = len(seqs)
        self.table = dev[: n * width].view(n, width)
        self.kv_len = dev[n * width: n * width + n]
        self.q_start = dev[n * width + n:]
        self.tokens, self.max_q, self.max_kv = start[-1], max(counts), max(lens)


class KVPool:
    """One shared pool (a ``kvpool_t``) on the current CUDA device."""

    def __init__(self, layers, kv_heads, head_dim, ctx, bits=None, max_rows=0, k_block=0):
        """k_block: 0 (one K scale per layer) or 32 (one per 32 elements)."""
        self.layers, self.kv_heads, self.head_dim, self.ctx = layers, kv_heads, head_dim, ctx
        self.bits = list(bits) if bits is not None else [3] * layers
        self.k_block = k_block
        arr = (ctypes.c_uint8 * layers)(*self.bits)
        h = ctypes.c_void_p()
        _check(_lib().kvpool_create_ex(ctypes.byref(h), layers, kv_heads, head_dim, ctx,
                                       ctypes.cast(arr, ctypes.c_void_p), max_rows, k_block),
               "kvpool_create_ex")
        self._h = h

    @property
    def handle(self):
        return self._h

    def close(self):
        if getattr(self, "_h", None):
            _lib().kvpool_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def compress(self, layer, K, V, stream=None):
        import torch

        _check(_lib().kvpool_compress(self._h, layer, _dev_ptr(K, torch.bfloat16, "K"),
                                      _dev_ptr(V, torch.bfloat16, "V"), _stream_ptr(stream)),
               "kvpool_compress")

    def compress_layers(self, layers, Ks, Vs, stream=None):
        """compress() of every layer in ``layers`` (K = Ks[i], V = Vs[i]) in
        one call: one max|K| kernel for all of them, one encode kernel per V
        width among them."""
        import torch

        n = len(layers)
        if len(Ks) != n or len(Vs) != n:
            raise ValueError("layers, Ks and Vs must have the same length")
        lay = (ctypes.c_int * max(n, 1))(*[int(l) for l in layers])
        kp = (ctypes.c_void_p * max(n, 1))(*[_dev_ptr(K, torch.bfloat16, "K").value for K in Ks])
        vp = (ctypes.c_void_p * max(n, 1))(*[_dev_ptr(V, torch.bfloat16, "V").value for V in Vs])
        _check(_lib().kvpool_compress_layers(self._h, n, lay, kp, vp, _stream_ptr(stream)),
               "kvpool_compress_layers")

    def append(self, layer, K, V, bits=None, stream=None):
        """Append tokens to a block-scaled layer: K, V bf16 [kv_heads, n, d]
        (device) become tokens [len, len + n) of the layer, their V codes at
        `bits` (None: the layer's width; else 2..that width)."""
        import torch

        kp, vp = _dev_ptr(K, torch.bfloat16, "K"), _dev_ptr(V, torch.bfloat16, "V")
        if bits is None:
            _check(_lib().kvpool_append(self._h, layer, kp, vp, int(K.shape[1]), _stream_ptr(stream)),
                   "kvpool_append")
        else:
            _check(_lib().kvpool_append_bits(self._h, layer, kp, vp, int(K.shape[1]), int(bits),
                                             _stream_ptr(stream)), "kvpool_append_bits")

    def layer_widths(self, layer):
        """V width of every 32-token group the layer holds (list of int)."""
        n = int(_lib().kvpool_layer_widths(self._h, layer, None, 0))
        if n < 0:
            raise KVPoolError(n, "kvpool_layer_widths")
        buf = (ctypes.c_uint8 * max(n, 1))()
        _check(min(0, _lib().kvpool_layer_widths(self._h, layer, buf, n)), "kvpool_layer_widths")
        return [int(b) for b in buf[:n]]

    def layer_len(self, layer) -> int:
        """Tokens the layer holds (ctx once compressed)."""
        n = int(_lib().kvpool_layer_len(self._h, layer))
        if n < 0:
            raise KVPoolError(n, "kvpool_layer_len")
        return n

    def attend(self, layer, Q, out=None, tail=None, softmax_scale=0.0, stream=None):
        """Q: bf16 [agents, q_heads, d]; tail: None or (K, V, lens) with K, V
        bf16 [agents, kv_heads, T_max, d] and lens int32 [agents] (device).
        Returns out: float32 [agents, q_heads, d]."""
        import torch

        A, Hq, d = Q.shape
        if out is None:
            out = torch.empty((A, Hq, d), dtype=torch.float32, device=Q.device)
        tp = None
        if tail is not None:
            Kt, Vt, lens = tail
            self._tail = Tail(_dev_ptr(Kt, torch.bfloat16, "tail K").value,
                              _dev_ptr(Vt, torch.bfloat16, "tail V").value,
                              _dev_ptr(lens, torch.int32, "tail len").value, Kt.shape[2])
            tp = ctypes.byref(self._tail)
        _check(_lib().kvpool_attend(self._h, layer, _dev_ptr(Q, torch.bfloat16, "Q"), A, Hq, tp,
                                    _dev_ptr(out, torch.float32, "out"), softmax_scale,
                                    _stream_ptr(stream)), "kvpool_attend")
        return out

    def attend_ws_bytes(self, agents, q_heads) -> int:
        """Workspace bytes kvpool_attend_ws needs for this many agents."""
        return int(_lib().kvpool_attend_ws_bytes(self._h, int(agents), int(q_heads)))

    def attend_ws(self, layer, Q, workspace=None, out=None, tail=None, softmax_scale=0.0, stream=None):
        """kvpool_attend_ws: as attend, through a device workspace (uint8
        tensor of at least attend_ws_bytes bytes; allocated here if None)."""
        import torch

        A, Hq, d = Q.shape
        if out is None:
            out = torch.empty((A, Hq, d), dtype=torch.float32, device=Q.device)
        if workspace is None:
            workspace = torch.empty(max(self.attend_ws_bytes(A, Hq), 16), dtype=torch.uint8, device=Q.device)
        tp = None
        if tail is not None:
            Kt, Vt, lens = tail
            self._tail = Tail(_dev_ptr(Kt, torch.bfloat16, "tail K").value,
                              _dev_ptr(Vt, torch.bfloat16, "tail V").value,
                              _dev_ptr(lens, torch.int32, "tail len").value, Kt.shape[2])
            tp = ctypes.byref(self._tail)
        _check(_lib().kvpool_attend_ws(self._h, layer, _dev_ptr(Q, torch.bfloat16, "Q"), A, Hq, tp,
                                       _dev_ptr(out, torch.float32, "out"), softmax_scale,
                                       workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                       _stream_ptr(stream)), "kvpool_attend_ws")
        return out

    def attend_pages_ws_bytes(self, tokens, q_heads) -> int:
        """Workspace bytes kvpool_attend_pages needs for this many tokens."""
        return int(_lib().kvpool_attend_pages_ws_bytes(self._h, _i32(int(tokens), "tokens"),
                                                       _i32(int(q_heads), "q_heads")))

    def attend_pages(self, layer, Q, cache, batch, page_layer=None, workspace=None, out=None, softmax_scale=0.0,
                     stream=None):
        """kvpool_attend_pages: the new tokens of a PagedCache's batch over this
        pool's layer and their own pages (page_layer, by default the same
        number). Q: bf16 [tokens, q_heads, d]. Returns out: float32, like Q."""
        import torch

        layer = _i32(layer, "layer")
        page_layer = layer if page_layer is None else _i32(page_layer, "page_layer")
        _check_rows(Q, batch)
        n, hq, d = Q.shape
        dev = _here()
        pg = _pages(cache.K, cache.V, cache.status_word, dev)
        if d != pg.head_dim:
            raise ValueError("Q must be [tokens, q_heads, head_dim]")
        sq = _seqs(batch.table, batch.kv_len, batch.q_start, n, batch.max_q, batch.max_kv, dev)
        qp = _need(Q, torch.bfloat16, "Q", dev)
        if out is not None and tuple(out.shape) != (n, hq, d):
            raise ValueError(f"out must have shape {(n, hq, d)}")
        # on the stream that uses them, so that the allocator knows it
        with contextlib.nullcontext() if stream is None else torch.cuda.stream(stream):
            if out is None:
                out = torch.empty((n, hq, d), dtype=torch.float32, device=Q.device)
            if workspace is None:
                workspace = torch.empty(max(self.attend_pages_ws_bytes(n, hq), 16), dtype=torch.uint8, device=Q.device)
        _check(_lib().kvpool_attend_pages(self._h, layer, ctypes.byref(pg), page_layer,
                                          ctypes.byref(sq), qp, hq, _need(out, torch.float32, "out", dev),
                                          softmax_scale, _need(workspace, workspace.dtype, "workspace", dev),
                                          workspace.numel() * workspace.element_size(), _raw_stream(stream, dev)),
               "kvpool_attend_pages")
        return out

    def attend_partial(self, layer, Q, t_begin, t_end, ml=None, acc=None, softmax_scale=0.0, stream=None):
        """kvpool_attend_partial over pool tokens [t_begin, t_end): returns
        (ml float32 [kv_heads, rows, 2], acc float32 [kv_heads, rows, d]),
        rows = agents * (q_heads / kv_heads)."""
        import torch

        A, Hq, d = Q.shape
        R = A * (Hq // self.kv_heads)
        if ml is None:
            ml = torch.empty((self.kv_heads, R, 2), dtype=torch.float32, device=Q.device)
        if acc is None:
            acc = torch.empty((self.kv_heads, R, d), dtype=torch.float32, device=Q.device)
        _check(_lib().kvpool_attend_partial(self._h, layer, _dev_ptr(Q, torch.bfloat16, "Q"), A, Hq, t_begin, t_end,
                                            _dev_ptr(ml, torch.float32, "ml"), _dev_ptr(acc, torch.float32, "acc"),
                                            softmax_scale, _stream_ptr(stream)), "kvpool_attend_partial")
        return ml, acc

    def decompress(self, layer, K_out=None, V_out=None, stream=None):
        import torch

        shape = (self.kv_heads, self.layer_len(layer), self.head_dim)
        dev = torch.device("cuda", torch.cuda.current_device())
        if K_out is None:
            K_out = torch.empty(shape, dtype=torch.bfloat16, device=dev)
        if V_out is None:
            V_out = torch.empty(shape, dtype=torch.bfloat16, device=dev)
        _check(_lib().kvpool_decompress(self._h, layer, _dev_ptr(K_out, torch.bfloat16, "K_out"),
                                        _dev_ptr(V_out, torch.bfloat16, "V_out"),
                                        _stream_ptr(stream)), "kvpool_decompress")
        return K_out, V_out

    def decompress_layers(self, layers, K_outs=None, V_outs=None, stream=None):
        """decompress() of every layer in ``layers`` in one launch per V
        width. K_outs / V_outs: lists of bf16 [kv_heads, len, d] tensors
        (allocated when None). Returns (K_outs, V_outs)."""
        import torch

        n = len(layers)
        dev = torch.device("cuda", torch.cuda.current_device())

        def outs(given):
            if given is not None:
                if len(given) != n:
                    raise ValueError("one output per layer")
                return list(given)
            return [torch.empty((self.kv_heads, self.layer_len(l), self.head_dim), dtype=torch.bfloat16,
                                device=dev) for l in layers]

        K_outs, V_outs = outs(K_outs), outs(V_outs)
        lay = (ctypes.c_int * max(n, 1))(*[int(l) for l in layers])
        kp = (ctypes.c_void_p * max(n, 1))(*[_dev_ptr(K, torch.bfloat16, "K_out").value for K in K_outs])
        vp = (ctypes.c_void_p * max(n, 1))(*[_dev_ptr(V, torch.bfloat16, "V_out").value for V in V_outs])
        _check(_lib().kvpool_decompress_layers(self._h, n, lay, kp, vp, _stream_ptr(stream)),
               "kvpool_decompress_layers")
        return K_outs, V_outs

    def pool_bytes(self) -> int:
        return int(_lib().kvpool_pool_bytes(self._h))

    def device_bytes(self) -> int:
        return int(_lib().kvpool_device_bytes(self._h))

    def status(self, stream=None) -> int:
        """Synchronise and return (and clear) the device status code."""
        return int(_lib().kvpool_status(self._h, _stream_ptr(stream)))

    def reset_layer(self, layer):
        _check(_lib().kvpool_reset_layer(self._h, layer), "kvpool_reset_layer")

    def layer_view(self, layer) -> LayerView:
        v = LayerView()
        _check(_lib().kvpool_layer_view(self._h, layer, ctypes.byref(v)), "kvpool_layer_view")
        return v

    def export_layer(self, layer, stream=None):
        """The layer's stored bytes as device tensors (token padding removed):
        kq int8 [Hk, ctx, d], vcodes uint8 [Hk, ceil(ctx/32), d, 4*bits] (per
        32-token group, one packed code sequence per coordinate; a layer of
        per-group widths: [Hk, sum_g d*4*b_g], its groups back to back),
        vnorm float32 [Hk, ctx], kscale float32 [1]."""
        import torch

        bits = self.bits[layer]
        dev = torch.device("cuda", torch.cuda.current_device())
        Hk, T, d = self.kv_heads, self.layer_len(layer), self.head_dim
        kq = torch.empty((Hk, T, d), dtype=torch.int8, device=dev)
        if self.layer_view(layer).mixed:
            vc = torch.empty((Hk, d * 4 * sum(self.layer_widths(layer))), dtype=torch.uint8, device=dev)
        else:
            vc = torch.empty((Hk, (T + 31) // 32, d, 4 * bits), dtype=torch.uint8, device=dev)
        vn = torch.empty((Hk, T), dtype=torch.float32, device=dev)
        ks = torch.empty(1, dtype=torch.float32, device=dev)
        _check(_lib().kvpool_export_layer(self._h, layer, kq.data_ptr(), vc.data_ptr(),
                                          vn.data_ptr(), ks.data_ptr(), _stream_ptr(stream)),
               "kvpool_export_layer")
        return kq, vc, vn, ks

    def import_layer(self, layer, kq, vcodes, vnorm, kscale, stream=None):
        _check(_lib().kvpool_import_layer(self._h, layer, kq.data_ptr(), vcodes.data_ptr(),
                                          vnorm.data_ptr(), kscale.data_ptr(),
                                          _stream_ptr(stream)), "kvpool_import_layer")

    def import_layer_blocks(self, layer, kq, vcodes, vnorm, kscales, widths=None, stream=None):
        """Load a block-scaled layer: kq int8 [Hk, len, d], vcodes uint8 (the
        layer's groups per head back to back), vnorm float32 [Hk, len],
        kscales float32 [Hk, len, d/32] (device tensors); widths: list of the
        groups' V widths (None: the layer's width)."""
        buf = None
        if widths is not None:
            buf = (ctypes.c_uint8 * max(len(widths), 1))(*widths)
        _check(_lib().kvpool_import_layer_blocks(self._h, layer, kq.data_ptr(), vcodes.data_ptr(), vnorm.data_ptr(),
                                                 kscales.data_ptr(), buf, int(kq.shape[1]), _stream_ptr(stream)),
               "kvpool_import_layer_blocks")

    def export_kscales(self, layer, stream=None):
        """Block scales of a block-scaled pool's layer: float32 [Hk, ctx, d/32]."""
        import torch

        out = torch.empty((self.kv_heads, self.layer_len(layer), self.head_dim // 32), dtype=torch.float32,
                          device="cuda")
        _check(_lib().kvpool_export_kscales(self._h, layer, out.data_ptr(), _stream_ptr(stream)),
               "kvpool_export_kscales")
        return out

    def read_layer(self, layer):
        """Host numpy copies of one layer's stored bytes (see export_layer)."""
        kq, vc, vn, ks = self.export_layer(layer)
        d = dict(kq=kq.cpu().numpy(), vcodes=vc.cpu().numpy(), vnorm=vn.cpu().numpy(),
                 kscale=ks.cpu().numpy()[0])
        if self.k_block:
            d["kscales"] = self.export_kscales(layer).cpu().numpy()
        return d
