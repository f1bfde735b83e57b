"""Paged private caches on a machine without a GPU: the pager against the plain
restatement, and what the calls refuse before they touch a device (every call
here is refused: the addresses are never used)."""

import ctypes
import random

import numpy as np
import pytest

from oracle import paged

INVALID, OOM = -1, -4


@pytest.fixture(scope="module")
def kp():
    from shared_quantized_kv_gb300 import build, kvpool

    build.build()
    kvpool.lib()
    return kvpool


def same(p, o):
    """Library pager p (kvpool.Pager) and oracle pager o agree."""
    assert p.free_pages() == len(o.free())
    for s in o.len:
        assert p.length(s) == o.len[s] and p.table(s) == o.table[s], s
    for page in range(o.pages):
        assert p.owners(page) == o.owners(page), page


@pytest.mark.parametrize("P,pages,seed", [(16, 12, 0), (64, 40, 1), (128, 7, 2), (32, 200, 3)])
def test_pager_follows_the_plain_rules(kp, P, pages, seed):
    r = random.Random(seed)
    p, o = kp.Pager(pages, P), paged.Pager(pages, P)
    for _ in range(400):
        live = sorted(o.len)
        what = r.choice(["new", "extend", "extend", "extend", "fork", "truncate", "free", "compact"])
        if what == "new" or not live:
            if len(live) < 9:
                assert p.new() == o.new()
            continue
        s = r.choice(live)
        if what == "extend":
            n = r.choice([0, 1, 1, r.randrange(1, 3 * P), pages * P])
            want = o.extend(s, n)
            if want == "oom":
                with pytest.raises(kp.KVPoolError) as e:
                    p.extend(s, n)
                assert e.value.code == OOM
            else:
                assert p.extend(s, n) == want
        elif what == "fork" and len(live) < 9:
            assert p.fork(s) == o.fork(s)
        elif what == "truncate":
            n = r.randrange(o.len[s] + 1)
            p.truncate(s, n), o.truncate(s, n)
        elif what == "free":
            p.free(s), o.end(s)
        elif what == "compact":
            src, dst = p.compact()
            assert list(zip(src, dst)) == o.compact()
            assert not set(src) & set(dst)
        same(p, o)
    p.close()


def test_pager_compacts_in_parts(kp):
    p = kp.Pager(10, 16)
    a, b = p.new(), p.new()
    p.extend(a, 5 * 16), p.extend(b, 4 * 16)
    p.free(a)
    lib = kp.lib()
    src, dst = (ctypes.c_int32 * 1)(), (ctypes.c_int32 * 1)()
    moves = []
    while lib.kvpool_pager_compact(p.handle, src, dst, 1) == 1:
        moves.append((src[0], dst[0]))
    assert moves == [(8, 0), (7, 1), (6, 2), (5, 3)] and p.table(b) == [3, 2, 1, 0]
    assert p.compact() == ([], [])
    p.close()


def test_numbers_past_32_bits(kp):
    """They are refused, not cut to their low bits."""
    p = kp.Pager(4, 16)
    s = p.new()
    for f in (lambda n: p.extend(s, n), lambda n: p.truncate(s, n)):
        for n in (1 << 31, 1 << 32, -(1 << 31) - 1):
            with pytest.raises(ValueError):
                f(n)
    assert p.length(s) == 0
    p.close()


def test_pager_refusals(kp):
    lib = kp.lib()
    h = ctypes.c_void_p()
    for pages, P in ((0, 16), (-1, 16), (4, 0), (4, 8), (4, 48), (4, 256)):
        assert lib.kvpool_pager_create(ctypes.byref(h), pages, P) == INVALID and not h.value
    assert lib.kvpool_pager_create(None, 4, 16) == INVALID
    p = kp.Pager(4, 16)
    s = p.new()
    pair = (ctypes.c_int32 * 2)()
    for bad in (-1, s + 1, 1 << 30):
        assert lib.kvpool_pager_extend(p.handle, bad, 1, pair) == INVALID
        assert lib.kvpool_pager_truncate(p.handle, bad, 0) == INVALID
        assert lib.kvpool_pager_fork(p.handle, bad) == INVALID
        assert lib.kvpool_pager_free(p.handle, bad) == INVALID
        assert lib.kvpool_pager_len(p.handle, bad) == INVALID
        assert lib.kvpool_pager_table(p.handle, bad, None, 0) == INVALID
    assert lib.kvpool_pager_extend(p.handle, s, -1, pair) == INVALID
    assert lib.kvpool_pager_extend(p.handle, s, 1, None) == INVALID
    assert lib.kvpool_pager_extend(p.handle, s, 4 * 16 + 1, pair) == OOM
    assert p.length(s) == 0 and p.free_pages() == 4
    p.extend(s, 20)
    assert lib.kvpool_pager_truncate(p.handle, s, 21) == INVALID
    assert lib.kvpool_pager_truncate(p.handle, s, -1) == INVALID
    assert lib.kvpool_pager_extend(p.handle, s, (1 << 31) - 1, pair) == INVALID
    assert lib.kvpool_pager_table(p.handle, s, None, 2) == INVALID
    assert lib.kvpool_pager_compact(p.handle, None, None, 1) == INVALID
    assert lib.kvpool_pager_owners(p.handle, 4) == INVALID and lib.kvpool_pager_owners(p.handle, -1) == INVALID
    p.free(s)
    assert lib.kvpool_pager_free(p.handle, s) == INVALID
    for f in (lib.kvpool_pager_new, lib.kvpool_pager_free_pages):
        assert f(None) == INVALID
    lib.kvpool_pager_destroy(None)
    p.close()


A = 1 << 20  # an address that is never used


def pages(kp, **change):
    f = dict(K=A, V=A, layers=2, pages=8, kv_heads=2, page_tokens=16, head_dim=64, status=None)
    f.update(change)
    return kp.Pages(**f)


def seqs(kp, **change):
    f = dict(seqs=2, table_stride=4, page_table=A, kv_len=A, q_start=A, tokens=3, max_q=0, max_kv=0)
    f.update(change)
    return kp.Seqs(**f)


BAD_PAGES = [dict(K=None), dict(V=None), dict(K=A + 8), dict(V=A + 2), dict(layers=0), dict(layers=1 << 16), dict(pages=0),
             dict(kv_heads=0), dict(kv_heads=1 << 17), dict(page_tokens=8), dict(page_tokens=48), dict(page_tokens=256),
             dict(head_dim=96), dict(head_dim=256), dict(pages=1 << 30, kv_heads=4), dict(status=A + 2)]
BAD_SEQS = [dict(seqs=0), dict(table_stride=0), dict(tokens=0), dict(max_q=-1), dict(max_kv=-1), dict(page_table=None),
            dict(kv_len=None), dict(q_start=None), dict(page_table=A + 2), dict(kv_len=A + 1), dict(q_start=A + 3)]


def test_append_refusals(kp):
    f = kp.lib().kvpool_pages_append
    by = ctypes.byref

    def call(pg=None, sq=None, layer=0, K=A, ks=128, V=A, vs=128):
        return f(by(pg or pages(kp)), layer, by(sq or seqs(kp)), K, ks, V, vs, None)

    for c in BAD_PAGES:
        assert call(pg=pages(kp, **c)) == INVALID, c
    for c in BAD_SEQS:
        assert call(sq=seqs(kp, **c)) == INVALID, c
    for c in (dict(layer=-1), dict(layer=2), dict(K=None), dict(V=None), dict(K=A + 8), dict(V=A + 4), dict(ks=120),
              dict(vs=64), dict(ks=132), dict(vs=-128)):
        assert call(**c) == INVALID, c
    assert f(None, 0, by(seqs(kp)), A, 128, A, 128, None) == INVALID
    assert f(by(pages(kp)), 0, None, A, 128, A, 128, None) == INVALID


def test_copy_refusals(kp):
    f = kp.lib().kvpool_pages_copy
    by = ctypes.byref

    def call(src, dst, n=None, pg=None):
        arr = lambda x: None if x is None else (ctypes.c_int32 * max(len(x), 1))(*x)
        return f(by(pg or pages(kp)), arr(src), arr(dst), len(src) if n is None else n, None)

    for c in BAD_PAGES:
        assert call([0], [1], pg=pages(kp, **c)) == INVALID, c
    for src, dst in (([0], [0]), ([0, 1], [2, 2]), ([0, 2], [2, 3]), ([0, 1], [1, 2]), ([8], [0]), ([0], [8]),
                     ([-1], [0]), ([0], [-1]), ([0, 1], [1, 0])):
        assert call(src, dst) == INVALID, (src, dst)
    assert call([0], [1], n=-1) == INVALID
    assert call([0], [1], n=9) == INVALID
    assert call(None, [1], n=1) == INVALID and call([1], None, n=1) == INVALID
    big = pages(kp, pages=1000)
    src, dst = list(range(100)), list(range(100, 200))
    for i, page in ((99, 100), (99, 5), (0, 150)):  # a destination twice, or a source too
        assert call(src, dst[:i] + [page] + dst[i + 1:], pg=big) == INVALID, (i, page)
    assert call([], []) == 0  # nothing to do, no device asked


def test_attend_refusals(kp):
    f = kp.lib().kvpool_pages_attend
    by = ctypes.byref

    def call(pg=None, sq=None, layer=0, Q=A, qs=256, hq=4, score=None, out=A, lse=None, scale=0.0):
        return f(by(pg or pages(kp)), layer, by(sq or seqs(kp)), Q, qs, hq, None if score is None else by(score), out,
                 lse, scale, None)

    for c in BAD_PAGES:
        assert call(pg=pages(kp, **c)) == INVALID, c
    for c in BAD_SEQS:
        assert call(sq=seqs(kp, **c)) == INVALID, c
    nan, inf = float("nan"), float("inf")
    for c in (dict(layer=-1), dict(layer=2), dict(Q=None), dict(Q=A + 8), dict(out=None), dict(out=A + 2), dict(lse=A + 2),
              dict(hq=1), dict(hq=3), dict(hq=0), dict(hq=-2), dict(qs=255), dict(qs=248), dict(qs=260), dict(scale=-1.0),
              dict(scale=nan), dict(scale=inf), dict(sq=seqs(kp, tokens=(1 << 31) - 1))):
        assert call(**c) == INVALID, c
    for c in (dict(cap=-1.0), dict(cap=nan), dict(cap=inf), dict(window=-1), dict(slopes=A + 2), dict(first=A + 1),
              dict(prefix=A + 2)):
        assert call(score=kp.Score(**c)) == INVALID, c
    assert f(None, 0, by(seqs(kp)), A, 256, 4, None, A, None, 0.0, None) == INVALID
    assert f(by(pages(kp)), 0, None, A, 256, 4, None, A, None, 0.0, None) == INVALID
    assert kp.lib().kvpool_pages_status(None, None) == INVALID
    assert kp.lib().kvpool_pages_status(by(pages(kp)), None) == INVALID


def test_scales_past_float32_are_refused(kp):
    f = kp.lib().kvpool_pages_attend
    by = ctypes.byref
    for cap, scale in ((0.0, 3e38), (1e-40, 0.0), (1e-38, 10.0), (5.0, 2.9e38)):
        sc = kp.Score(cap=cap)
        assert f(by(pages(kp)), 0, by(seqs(kp)), A, 256, 4, by(sc), A, None, scale, None) == INVALID, (cap, scale)


def test_oracle_attend_is_a_softmax_over_what_is_seen():
    """The restatement itself, against a row written out by hand."""
    r = np.random.default_rng(0)
    K, V = (r.standard_normal((1, 3, 1, 16, 64)) for _ in range(2))
    Q = r.standard_normal((2, 1, 64))
    table = np.array([[2, 0]])
    o, z, mag, err = paged.attend(K, V, 0, Q, table, [20], [0, 2], window=5, prefix=[3], cap=2.0, slopes=np.array([0.1]))
    for i, p in enumerate((18, 19)):
        js = [0, 1, 2] + list(range(p - 4, p + 1))
        x = []
        for j in js:
            s = float(Q[i, 0] @ K[0, table[0, j // 16], 0, j % 16]) / 8
            x.append(2 * np.tanh(s / 2) - 0.1 * (p - j))
        w = np.exp(x)
        v = np.stack([V[0, table[0, j // 16], 0, j % 16] for j in js])
        assert np.allclose(o[i, 0], w @ v / w.sum(), rtol=1e-12)
        assert np.isclose(z[i, 0], np.log(w.sum()), rtol=1e-12)
        assert (mag[i, 0] >= np.abs(o[i, 0]) - 1e-12).all() and 0 < err[i, 0] < 1e-4
