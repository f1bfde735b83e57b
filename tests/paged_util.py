"""Helpers of the paged-cache tests: caches whose pages lie scattered and whose
unused slots hold NaN, and the error bounds of the attention kernels."""

import numpy as np

from oracle import paged


def bf16(x):
    """Round to bf16 values (float32 array), nearest even."""
    b = np.ascontiguousarray(x, np.float32).view(np.uint32)
    return (((b + 0x7FFF + ((b >> 16) & 1)) >> 16) << 16).astype(np.uint32).view(np.float32)


class Batch:
    """Sequences with q[i] new and kv[i] held tokens, layer `layer` of `layers`,
    in scattered pages; slots behind a sequence's end are NaN, unused table
    entries garbage."""

    def __init__(self, hk, hq, d, P, q, kv, seed=0, layers=1, layer=0, extra_rows=0, garbage=-7):
        r = np.random.default_rng(seed)
        self.hk, self.hq, self.d, self.P, self.layer = hk, hq, d, P, layer
        self.q, self.kv = list(q), list(kv)
        need = [-(-t // P) for t in kv]
        pages = sum(need) + 2
        order = r.permutation(pages)
        self.table = np.full((len(q), max(1, max(need)) + 1), garbage, np.int32)
        self.K = np.full((layers, pages, hk, P, d), np.nan, np.float32)
        self.V = self.K.copy()
        self.std = np.exp(0.5 * r.standard_normal((2, hk, d))).astype(np.float32)
        at = 0
        for s, n in enumerate(need):
            self.table[s, :n] = order[at: at + n]
            at += n
            page, slot = paged.token_slots(self.table[s], 0, kv[s], P)
            for X, sd in ((self.K, self.std[0]), (self.V, self.std[1])):
                X[layer, page, :, slot] = bf16(r.standard_normal((kv[s], hk, d), dtype=np.float32) * sd)
        self.q_start = np.concatenate([[0], np.cumsum(q)]).astype(np.int32)
        self.kv_len = np.array(kv, np.int32)
        self.tokens = int(sum(q)) + extra_rows
        self.Q = bf16(r.standard_normal((max(self.tokens, 1), hq, d), dtype=np.float32))

    def many(self, room=1 << 16):
        """Room for `room` tokens in every row of the table: with a max_kv of that,
        the attention kernel for many rows takes the call, its keys split over
        clusters where there are many of them."""
        self.table = np.pad(self.table, ((0, 0), (0, max(0, room // self.P - self.table.shape[1]))), constant_values=-9)
        assert reads(self, self.tokens, room) >= 1 << 27
        return self

    def dev(self):
        """(K, V, layer, Q, table, kv_len, q_start) on the GPU."""
        import torch

        f = lambda x: torch.from_numpy(x).cuda().to(torch.bfloat16)
        i = lambda x: torch.from_numpy(x).cuda()
        return f(self.K), f(self.V), self.layer, f(self.Q), i(self.table), i(self.kv_len), i(self.q_start)

    def ref(self, **score):
        with np.errstate(invalid="ignore"):
            return paged.attend(self.K, self.V, self.layer, self.Q, self.table, self.kv_len, self.q_start, **score)


def reads(b, max_q, max_kv):
    """Bytes by which the library chooses between its two attention kernels:
    blocks of 16 rows, each through all keys; 2^27 and more go to the kernel for
    many rows."""
    return len(b.q) * -(-max_q * (b.hq // b.hk) // 16) * b.hk * max_kv * b.d * 4


def check_attend(out, lse, ref, T):
    """out (bf16 values) and lse within the bounds that bf16 weights, a bf16
    output and float32 sums leave: half a step of bf16 (2^-8 relative) for the
    output, half a step for each weight (2^-8 of the weighted mean of |v|),
    and what an error e of the scores (and ex2's, 2^-22) does to weights: a
    factor within e^(+-2e). Sums of T float32 terms: T 2^-24 relative."""
    o, z, mag, err = ref
    mine = ~np.isnan(z)  # rows that belong to a sequence
    o, z, mag, err = o[mine], z[mine], mag[mine], err[mine]
    out, lse = out[mine].astype(np.float64), lse[mine].astype(np.float64)
    rel = np.expm1(2 * err + 2.0 ** -21 + T * 2.0 ** -23)[:, None]
    tol = 2.0 ** -8 * np.abs(o) + (2.0 ** -8 * (1 + 2.0 ** -7) + rel) * mag + 1e-30
    assert np.isfinite(out).all()
    worst = np.max(np.abs(out - o) / tol) if o.size else 0.0
    assert worst <= 1.0, f"output {worst:.3g} times its bound"
    empty = np.isneginf(z)
    assert (np.isneginf(lse) == empty).all() and (out[empty] == 0).all()
    d = np.abs(lse[~empty] - z[~empty])
    tolz = err[~empty] + T * 2.0 ** -23 + 2.0 ** -20 + 2.0 ** -22 * np.abs(z[~empty])
    assert (d <= tolz).all(), f"lse {np.max(d / tolz):.3g} times its bound"
