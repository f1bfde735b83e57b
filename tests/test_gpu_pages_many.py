"""Attention over paged caches by the kernel for many rows, at small sizes: its
row tiles (one per block, two), its split over clusters, every score modifier,
masked places that hold NaN, tables and lengths that lie, streams and graphs.
(The library gives small calls to the kernel for few rows; tables with room for
many tokens, or many blocks of rows, bring them here.)"""

import ctypes

import numpy as np
import pytest

from oracle import attention, codec, paged
from shared_quantized_kv_gb300 import workloads as wl

from paged_util import Batch, bf16, check_attend, reads
from parity_util import TOL, to_dev
from test_gpu_attend_pages import OneCache, reference
from test_gpu_pages import SCORES, kp, run, scores  # noqa: F401 (kp: a fixture)

pytestmark = pytest.mark.gpu

HEADS = [(2, 8, 128), (2, 2, 64), (1, 7, 128), (3, 9, 64)]
SPLIT = [0, 1 << 16]  # no clusters; clusters of 8 where there are few blocks


def hint(b, room):
    """max_kv of a call without clusters (tiles of 8 or fewer are not split), or of a widened table."""
    if room:
        b.many(room)
        return None
    assert reads(b, b.tokens, 1024) >= 1 << 27
    return 1024


@pytest.mark.parametrize("room", SPLIT)
@pytest.mark.parametrize("hk,hq,d", HEADS)
@pytest.mark.parametrize("P", [16, 32, 64, 128])
def test_ragged_batch(kp, hk, hq, d, P, room):
    """Blocks of one row tile and of two, empty and single-token sequences, whole
    prompts, and lengths on both sides of what a cluster splits. (Without
    clusters the long ones exceed the hint.)"""
    q = [0, 1, 5, 130, 0, 1, 77, 16, 0, 300, 20, 128, 200, 33, 40, 1]
    kv = [9, 200, 5, 131, 0, 1, 400, 1024, 40, 300, 1025, 1200, 2100, 2049, 127, 3000]
    b = Batch(hk, hq, d, P, q, kv, seed=hq).many(2048)
    if room:
        run(kp, b.many(room))
    else:
        run(kp, b, max_kv=hint(b, 0))


@pytest.mark.parametrize("hk,seqs", [(1, 12), (4, 7), (4, 17), (8, 20)])
def test_cluster_sizes(kp, hk, seqs):
    """Between 12 and 160 blocks: splits in 8, 4 and 2."""
    r = np.random.default_rng(seqs)
    q = [int(x) for x in r.integers(1, 60, seqs)]
    kv = [n + int(x) for n, x in zip(q, r.integers(1000, 2600, seqs))]
    run(kp, Batch(hk, 4 * hk, 64, 64, q, kv, seed=seqs).many(4096))


@pytest.mark.parametrize("room", SPLIT)
@pytest.mark.parametrize("name", sorted(SCORES))
@pytest.mark.parametrize("hk,hq,d", [(2, 8, 128), (1, 7, 128), (2, 2, 64)])
def test_scores(kp, name, hk, hq, d, room):
    q = [1, 0, 150, 3, 20, 300, 128, 40, 90]
    kv = [1, 50, 160, 700, 1500, 300, 2000, 1100, 90]
    b = Batch(hk, hq, d, 32, q, kv, seed=7)
    if room:
        run(kp, b.many(room), **scores(b, **SCORES[name]))
    else:
        run(kp, b.many(2048), max_kv=1024, **scores(b, **SCORES[name]))


@pytest.mark.parametrize("T", [400, 1900])
@pytest.mark.parametrize("chunk", [20, 100])
@pytest.mark.parametrize("score", [dict(), dict(window=150), dict(cap=9.0, slopes=True, window=150)])
def test_masked_keys_may_hold_anything(kp, T, chunk, score):
    """NaN and infinities where no row sees them, and in a chunk's last token,
    which only its own row sees; in blocks of one row tile and of two, with
    their keys split and not."""
    b = Batch(1, 4, 128, 16, [chunk, 1], [T, 60], seed=17).many()
    sc = scores(b, **score)
    if score:
        page, slot = paged.token_slots(b.table[0], 0, T - chunk - 149, b.P)
        b.K[0, page[::3], :, slot[::3]] = np.nan
        b.V[0, page[::3], :, slot[::3]] = np.inf
        b.V[0, page[1::3], :, slot[1::3]] = np.nan
        run(kp, b, **sc)
    page, slot = paged.token_slots(b.table[0], T - 1, 1, b.P)
    b.K[0, page, :, slot] = np.nan
    b.V[0, page, :, slot] = np.inf
    K, V, layer, Q, table, kv_len, q_start = b.dev()
    import torch

    dev = {k: torch.from_numpy(v).cuda() if isinstance(v, np.ndarray) else v for k, v in sc.items()}
    out, lse = kp.pages_attend(K, V, layer, Q, table, kv_len, q_start, return_lse=True, **dev)
    out, lse = out.float().cpu().numpy(), lse.cpu().numpy()
    assert np.isnan(out[chunk - 1]).all()
    ref = [x.copy() for x in b.ref(**sc)]
    for x in ref:
        x[chunk - 1] = np.nan
    check_attend(out, lse, ref, T)


@pytest.mark.parametrize("room", [0, 1 << 16])  # (the kernel for few rows, that for many)
@pytest.mark.parametrize("chunk,T", [(20, 900), (100, 900), (100, 2500)])
@pytest.mark.parametrize("rise,jump", [(0.02, 0), (0.3, 0), (0.02, 300), (-0.3, 0)])
@pytest.mark.parametrize("score", [dict(), dict(window=600)])
def test_scores_that_rise(kp, rise, jump, score, chunk, T, room):
    """Maxima that move on with every tile, by a little and by much, and one that
    jumps by more than float32 weights have room for."""
    b = Batch(1, 4, 64, 16, [chunk, 1], [T, 70], seed=22)
    if room:
        b.many(room)
    u = np.zeros(64, np.float32)
    u[:16] = 1
    at = np.arange(T)
    level = rise * at + jump * (at >= 2 * T // 3)
    page, slot = paged.token_slots(b.table[0], 0, T, b.P)
    K = b.K[0, page, 0, slot] * 0.1
    K[:, :16] = (level / 2)[:, None]  # <u, k> / sqrt(64) = level
    b.K[0, page, 0, slot] = bf16(K)
    b.Q = bf16(b.Q * 0.1 * (u == 0) + u)
    run(kp, b, **score)


@pytest.mark.parametrize("room", [0, 1 << 16])
@pytest.mark.parametrize("cap", [1e-30, 0.01, 1.0, 3.0, 1e6, 1e30])
def test_caps(kp, cap, room):
    """Caps that leave every score at the cap, between, and untouched; a zero row of Q."""
    b = Batch(1, 4, 64, 32, [100, 20], [1300, 900], seed=24)
    b.Q[5] = 0
    if room:
        b.many(room)
    if cap < 1e6:
        run(kp, b, cap=cap)
        return
    # tanh(z) is z within z^3 / 3, 1e-10 of a score here: the bound of plain scores holds
    K, V, layer, Q, table, kv_len, q_start = b.dev()
    out, lse = kp.pages_attend(K, V, layer, Q, table, kv_len, q_start, cap=cap, return_lse=True)
    check_attend(out.float().cpu().numpy(), lse.cpu().numpy(), b.ref(), 1300)


@pytest.mark.parametrize("room", [0, 1 << 16])
@pytest.mark.parametrize("top", [0.004, 0.2, 2.0, -0.05])
@pytest.mark.parametrize("score", [dict(), dict(cap=20.0), dict(prefix=True, window=90)])
def test_slopes(kp, top, score, room):
    """A bias by distance from flat to one that leaves the nearest keys alone, in
    heads side by side."""
    b = Batch(1, 4, 128, 32, [100, 20], [2100, 900], seed=23)
    if room:
        b.many(room)
    run(kp, b, slopes=np.array([0.0, 0.3, 0.7, 1.0], np.float32) * np.float32(top), **scores(b, **score))


@pytest.mark.parametrize("room", [0, 1 << 17])  # (the kernel for few rows, that for many)
@pytest.mark.parametrize("chunk", [1, 20, 100])
@pytest.mark.parametrize("T,window,prefix", [(1900, 150, 130), (5001, 1, 3), (6000, 1500, 700), (700, 500, 200)])
def test_between_prefix_and_window(kp, T, window, prefix, chunk, room):
    """Keys behind the prefix and before every window hold NaN and are passed
    over; with a chunk, so does its last token, which its own row alone sees."""
    import torch

    b = Batch(1, 4, 128, 32, [chunk, 1], [T, T - 40], seed=21)
    if room:
        b.many(room)
    pre = np.array([prefix, prefix // 2], np.int32)
    for s in range(2):
        gap = max(0, T - 40 * s - b.q[s] - window + 1 - pre[s])
        page, slot = paged.token_slots(b.table[s], pre[s], gap, b.P)
        b.K[0, page, :, slot] = np.nan
        b.V[0, page, :, slot] = np.inf
    run(kp, b, window=window, prefix=pre)
    if chunk == 1:
        return
    page, slot = paged.token_slots(b.table[0], T - 1, 1, b.P)
    b.V[0, page, :, slot] = np.nan
    K, V, layer, Q, table, kv_len, q_start = b.dev()
    out, lse = kp.pages_attend(K, V, layer, Q, table, kv_len, q_start, return_lse=True, window=window,
                               prefix=torch.from_numpy(pre).cuda())
    out, lse = out.float().cpu().numpy(), lse.cpu().numpy()
    assert np.isnan(out[chunk - 1]).all()
    ref = [x.copy() for x in b.ref(window=window, prefix=pre)]
    for x in ref:
        x[chunk - 1] = np.nan
    check_attend(out, lse, ref, T)


@pytest.mark.parametrize("d", [64, 128])
def test_many_sequences(kp, d):
    """More sequences than a warp's lanes, most of one token, some empty."""
    r = np.random.default_rng(15)
    q = [int(x) for x in r.choice([0, 1, 1, 1, 2, 9], 131)]
    kv = [n + int(r.integers(0, 60)) for n in q]
    run(kp, Batch(2, 4, d, 16, q, kv, seed=15).many(4096))


@pytest.mark.parametrize("hk,hq,d,q", [(1, 64, 128, 5), (1, 300, 64, 3), (1, 33, 128, 12), (2, 600, 64, 2)])
def test_wide_groups(kp, hk, hq, d, q):
    """Groups of query heads as large as a row tile, and larger than a block."""
    run(kp, Batch(hk, hq, d, 16, [q, 1, q], [200, 70, 1700], seed=hq).many())


def test_rows_behind_the_last_sequence_stay(kp):
    import torch

    for q in ([1, 33], [1, 90]):
        b = Batch(2, 8, 128, 16, q, [40, 1460], seed=9, extra_rows=50).many()
        K, V, layer, Q, table, kv_len, q_start = b.dev()
        out = torch.full((b.tokens, b.hq, b.d), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((b.tokens, b.hq), 7.0, device="cuda")
        kp.pages_attend(K, V, layer, Q, table, kv_len, q_start, out=out, lse=lse)
        n = sum(q)
        assert (out[n:] == 7).all() and (lse[n:] == 7).all()
        check_attend(out.float().cpu().numpy(), lse.cpu().numpy(), b.ref(), 1460)


@pytest.mark.parametrize("T", [70, 1400])
def test_page_numbers_out_of_range(kp, T):
    """They read as zeros and are recorded."""
    import torch

    make = lambda: Batch(2, 8, 64, 16, [1, 60], [100, T], seed=10).many()
    b, b2 = make(), make()
    b.table[0, 2], b.table[1, 1] = 1 << 20, -1
    for X in (b2.K, b2.V):
        np.nan_to_num(X, copy=False)
        X[0, b2.table[0, 2]] = X[0, b2.table[1, 1]] = 0
    K, V, layer, Q, table, kv_len, q_start = b.dev()
    K, V = torch.nan_to_num(K), torch.nan_to_num(V)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pg = kp._pages(K, V, status)
    out, lse = kp.pages_attend(K, V, layer, Q, table, kv_len, q_start, return_lse=True, status=status)
    assert kp.lib().kvpool_pages_status(ctypes.byref(pg), None) == -1
    assert kp.lib().kvpool_pages_status(ctypes.byref(pg), None) == 0
    check_attend(out.float().cpu().numpy(), lse.cpu().numpy(), b2.ref(), T)


@pytest.mark.parametrize("room", [0, 1 << 16])
def test_lengths_that_do_not_fit(kp, room):
    """More new rows than held tokens: rows before the first token see nothing.
    Held tokens beyond the table's room or below 0, row starts beyond the rows:
    an outcome, whatever it is. (In both kernels.)"""
    import torch

    kv = [60, 40, 50]
    make = lambda: Batch(2, 8, 128, 16, [60, 2, 1], kv, seed=16)
    b, c = make(), make()
    if room:
        b.many(room)
    K, V, layer, Q, table, kv_len, q_start = b.dev()
    K, V = torch.nan_to_num(K), torch.nan_to_num(V)
    table = table.clamp(min=0)
    short = kv_len.clone()
    short[0] = 25
    out, lse = kp.pages_attend(K, V, 0, Q, table, short, q_start, return_lse=True)
    assert (out[:35] == 0).all() and torch.isneginf(lse[:35]).all()
    c.q, c.kv, c.kv_len = [25, 2, 1], [25, 40, 50], np.array([25, 40, 50], np.int32)
    c.Q, c.q_start = c.Q[35:], np.array([0, 25, 27, 28], np.int32)
    check_attend(out[35:].float().cpu().numpy(), lse[35:].cpu().numpy(), c.ref(), 60)
    new = torch.ones(63, 2, 128, dtype=torch.bfloat16, device="cuda")
    for lens, starts in (([1 << 30, -5, 1 << 20], [0, 60, 62, 63]), ([60, 40, 50], [0, 1 << 30, 5, -7]),
                         ([-(1 << 31), 0, 50], [0, 60, 62, 1 << 20])):
        lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        starts = torch.tensor(starts, dtype=torch.int32, device="cuda")
        kp.pages_attend(K, V, 0, Q, table, lens, starts)
        kp.pages_append(K.clone(), V.clone(), 0, new, new, table, lens, starts)
        torch.cuda.synchronize()


def test_two_streams_at_once(kp):
    """Calls of both kernels on two streams, many times; the same bits each time."""
    import torch

    small = Batch(2, 8, 128, 16, [1, 1, 2], [700, 30, 900], seed=18)
    big = Batch(2, 8, 128, 16, [300, 50], [1900, 400], seed=19).many()
    streams = [torch.cuda.Stream(), torch.cuda.Stream(), torch.cuda.Stream()]
    args = [small.dev(), big.dev(), big.dev()]
    torch.cuda.synchronize()
    got = [[], [], []]
    for i in range(10):
        for st, a, g, q in zip(streams, args, got, (2, 300, 350)):
            K, V, layer, Q, table, kv_len, q_start = a
            g.append(kp.pages_attend(K, V, layer, Q, table, kv_len, q_start, max_q=q, return_lse=True, stream=st))
    torch.cuda.synchronize()
    for b, g in zip((small, big, big), got):
        check_attend(g[0][0].float().cpu().numpy(), g[0][1].cpu().numpy(), b.ref(), 1900)
        for o, z in g[1:]:
            assert torch.equal(o, g[0][0]) and torch.equal(z, g[0][1])


@pytest.mark.parametrize("score", [dict(), dict(window=50), dict(cap=8.0), dict(cap=30.0, slopes=True, window=40)])
def test_same_bits_whatever_lay_in_shared_memory(kp, score):
    """Short sequences leave most of a tile to what an earlier call left there."""
    import torch

    q = [1, 3, 40, 130, 1, 2, 77, 20, 5, 1]
    b = Batch(2, 8, 128, 16, q, [n + 3 * i for i, n in enumerate(q)], seed=25).many()
    K, V, layer, Q, table, kv_len, q_start = b.dev()
    dev = {k: torch.from_numpy(v).cuda() if isinstance(v, np.ndarray) else v for k, v in scores(b, **score).items()}
    other = Batch(2, 8, 128, 16, [300, 200], [1300, 900], seed=26).many()
    runs = []
    for scale in (0.01, 1.0, 100.0, -100.0):
        Ko, Vo, lo, Qo, to, ko, qo = other.dev()
        kp.pages_attend(Ko * scale, Vo * scale, lo, Qo, to, ko, qo)
        runs.append(kp.pages_attend(K, V, layer, Q, table, kv_len, q_start, return_lse=True, **dev))
    for o, z in runs[1:]:
        assert torch.equal(o, runs[0][0]) and torch.equal(z, runs[0][1])


@pytest.mark.parametrize("hk,hq", [(1, 4), (1, 2)])
def test_captured_graph(kp, hk, hq):
    """The first call in a capture; lengths change between replays."""
    import torch

    b = Batch(hk, hq, 64, 32, [70, 9], [1500, 300], seed=20).many()
    K, V, layer, Q, table, kv_len, q_start = b.dev()
    out = torch.empty(79, hq, 64, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(79, hq, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kp.pages_attend(K, V, layer, Q, table, kv_len, q_start, out=out, lse=lse)
    for t0, t1 in ((1500, 300), (80, 9), (70, 250)):
        b.kv, b.kv_len = [t0, t1], np.array([t0, t1], np.int32)
        kv_len.copy_(torch.from_numpy(b.kv_len))
        np.nan_to_num(b.K, copy=False), np.nan_to_num(b.V, copy=False)
        graph.replay()
        check_attend(out.float().cpu().numpy(), lse.cpu().numpy(), b.ref(), 1500)


@pytest.mark.parametrize("hk,hq,d,ctx,bits,P,q,kv,max_rows", [
    (2, 8, 128, 700, 4, 32, [1, 100, 0, 7], [500, 1400, 9, 300], 0),   # two row tiles, split and not
    (4, 4, 64, 1000, 2, 64, [50, 100], [130, 2000], 0),                 # one row tile
    (1, 7, 128, 260, 3, 128, [45, 1], [200, 1977], 64),                 # slices of 9 tokens
    (2, 4, 64, 130, 3, 16, [290, 1, 1], [900, 2, 50], 16),              # many slices
])
@pytest.mark.parametrize("bad", [False, True])
def test_pool_and_pages_in_one_softmax(kp, hk, hq, d, ctx, bits, P, q, kv, max_rows, bad):
    """As in test_gpu_attend_pages, the rows' states by the kernel for many rows;
    bad: NaN in the last token of a chunk, which its own row alone sees."""
    import torch

    w = wl.custom("pages_many", 1, hk, hq, d, ctx, 1, "lognormal", bits=(bits,))
    K, V = wl.layer_kv(w, 0)
    pool = kp.KVPool(1, hk, d, ctx, [bits], max_rows=max_rows)
    pool.compress(0, to_dev(K), to_dev(V))
    enc = codec.encode_layer(K, V, bits)
    b = Batch(hk, hq, d, P, q, kv, seed=ctx, layers=2, layer=1, extra_rows=3).many()
    ref = reference(enc, b.Q, b.K, b.V, 1, b.table, b.kv_len, b.q_start)
    longest = int(np.argmax(q))
    last = int(b.q_start[longest + 1]) - 1
    if bad:
        page, slot = paged.token_slots(b.table[longest], kv[longest] - 1, 1, P)
        b.V[1, page, :, slot] = np.nan
    c = OneCache(b)
    c.max_q, c.max_kv = b.tokens, 1 << 16
    out = torch.full((b.tokens, hq, d), float("nan"), device="cuda")
    got = pool.attend_pages(0, c.Q, c, c, page_layer=1, out=out).cpu().numpy()
    assert pool.status() == 0 and int(c.status_word.cpu()[0]) == 0
    keep = np.ones(b.tokens, bool)
    if bad:
        assert np.isnan(got[last]).all()
        keep[last] = False
    err = attention.row_rel_error(got[keep].astype(np.float64), ref[keep])
    assert err <= TOL, err
    pool.close()
