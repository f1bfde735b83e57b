"""Attention over paged caches in 4 bits by the kernel for many rows, at small
sizes: its row tiles (one per block, two), its split over clusters, every score
modifier, scales far apart or not finite, scores that rise and jump, tables and
lengths that lie, streams. (The library gives small calls to the kernel for few
rows; tables with room for many tokens bring them here.)"""

import numpy as np
import pytest

from oracle import paged, paged4

from paged4_util import Batch4, check4
from paged_util import bf16
from test_gpu_pages4 import SCORES, kp, run, scores  # noqa: F401 (kp: a fixture)

pytestmark = pytest.mark.gpu

HEADS = [(2, 8, 128), (2, 2, 64), (1, 7, 128), (3, 9, 64)]
SPLIT = [1024, 1 << 16]  # max_kv: no clusters (tiles of 8 or fewer are not split); clusters of 8 where there are few blocks


def many(b, room):
    """Room for `room` tokens in every row of the table: the kernel for many rows takes the call."""
    b.table = np.pad(b.table, ((0, 0), (0, max(0, room // b.P - b.table.shape[1]))), constant_values=-9)
    rows = b.tokens * (b.hq // b.hk)
    assert rows > 32 and len(b.q) * -(-rows // 32) * b.hk * room >= 1 << 17
    return b


@pytest.mark.parametrize("room", SPLIT)
@pytest.mark.parametrize("hk,hq,d", HEADS)
@pytest.mark.parametrize("P", [16, 32, 64, 128])
def test_ragged_batch(kp, hk, hq, d, P, room):
    """Blocks of one row tile and of two, empty and single-token sequences, whole
    prompts, and lengths on both sides of what a cluster splits. (Without
    clusters the long ones exceed the hint.)"""
    q = [0, 1, 5, 130, 0, 1, 77, 16, 0, 300, 20, 128, 200, 33, 40, 1]
    kv = [9, 200, 5, 131, 0, 1, 400, 1024, 40, 300, 1025, 1200, 2100, 2049, 127, 3000]
    run(kp, many(Batch4(hk, hq, d, P, q, kv, seed=hq), 1 << 16), max_kv=room)


@pytest.mark.parametrize("tiles", [0, 1, 3, 8, 100])
@pytest.mark.parametrize("hk,hq,d", [(2, 8, 128), (1, 5, 64)])
def test_workspaces_of_any_size(kp, hk, hq, d, tiles):
    """None, room for the shorter sequences, room for all: the same results."""
    import torch

    q, kv = [300, 1, 0, 150, 90, 257], [300, 40, 90, 1024, 1025, 700]
    b = many(Batch4(hk, hq, d, 32, q, kv, seed=41), 1 << 16)
    dev = b.dev4(kp)
    n = kp.pages4_attend_ws_bytes(*dev[:1], *dev[3:], b.tokens, hq)
    each = len(q) * hk * (4 * 128 * d + 1024)
    assert n == each * ((1 << 16) // 128)
    ws = torch.full((tiles * each + 64,), 255, dtype=torch.uint8, device="cuda")
    out, lse = kp.pages4_attend(*dev, return_lse=True, workspace=ws if tiles else ws[:0], max_kv=None if tiles < 100 else 1025)
    check4(out.float().cpu().numpy(), lse.cpu().numpy(), b.ref4())
    same = kp.pages4_attend(*dev, return_lse=True, workspace=ws if tiles else ws[:0], max_kv=None if tiles < 100 else 1025)
    assert torch.equal(out, same[0]) and torch.equal(lse, same[1])


@pytest.mark.parametrize("hk,seqs", [(1, 12), (4, 7), (4, 17), (8, 20)])
def test_cluster_sizes(kp, hk, seqs):
    """Between 12 and 160 blocks: splits in 8, 4 and 2."""
    r = np.random.default_rng(seqs)
    q = [int(x) for x in r.integers(1, 60, seqs)]
    kv = [n + int(x) for n, x in zip(q, r.integers(1000, 2600, seqs))]
    run(kp, many(Batch4(hk, 4 * hk, 64, 64, q, kv, seed=seqs), 4096))


@pytest.mark.parametrize("room", SPLIT)
@pytest.mark.parametrize("name", sorted(SCORES))
@pytest.mark.parametrize("hk,hq,d", [(2, 8, 128), (1, 7, 128), (2, 2, 64)])
def test_scores(kp, name, hk, hq, d, room):
    q = [1, 0, 150, 3, 20, 300, 128, 40, 90]
    kv = [1, 50, 160, 700, 1500, 300, 2000, 1100, 90]
    b = many(Batch4(hk, hq, d, 32, q, kv, seed=7), 1 << 16)
    run(kp, b, max_kv=room, **scores(b, **SCORES[name]))


@pytest.mark.parametrize("T", [400, 1900])
@pytest.mark.parametrize("chunk", [20, 100])
@pytest.mark.parametrize("score", [dict(), dict(window=150), dict(cap=9.0, slopes=True, window=150)])
def test_masked_keys_may_hold_anything(kp, T, chunk, score):
    """NaN, infinities and huge scales where no row sees them, and in a chunk's last
    token, which only its own row sees; in blocks of one row tile and of two, with
    their keys split and not."""
    b = many(Batch4(1, 4, 128, 16, [chunk, 1], [T, 60], seed=17), 1 << 16)
    sc = scores(b, **score)
    if score:
        page, slot = paged.token_slots(b.table[0], 0, T - chunk - 149, b.P)
        for x, (i, j, k) in zip(b.scale, ((0, 1, 2), (1, 2, 0))):
            x[0, page[i::5], :, slot[i::5]] = np.nan
            x[0, page[j::5], :, slot[j::5]] = np.inf
            x[0, page[k::5], :, slot[k::5]] = 1e30
        run(kp, b, **sc)
    page, slot = paged.token_slots(b.table[0], T - 1, 1, b.P)
    b.scale[0][0, page, :, slot] = np.nan
    b.scale[1][0, page, :, slot] = np.inf
    import torch

    dev = {k: torch.from_numpy(v).cuda() if isinstance(v, np.ndarray) else v for k, v in sc.items()}
    out, lse = kp.pages4_attend(*b.dev4(kp), return_lse=True, **dev)
    out, lse = out.float().cpu().numpy(), lse.cpu().numpy()
    assert np.isnan(out[chunk - 1]).all()
    ref = [x.copy() for x in b.ref4(**sc)]
    for x in ref:
        x[chunk - 1] = np.nan
    check4(out, lse, ref)


@pytest.mark.parametrize("chunk,T", [(20, 900), (100, 900), (100, 2500)])
@pytest.mark.parametrize("score", [dict(), dict(window=600), dict(cap=40.0)])
@pytest.mark.parametrize("k,v", [((-3, 3), (-3, 3)), ((-30, 0), (-2, 2)), ((0, 0), (-40, 40)), ((-14, 2), (-20, 20))])
def test_scales_far_apart(kp, chunk, T, score, k, v):
    """Keys and values of very different norms, next to one another and from tile to
    tile, whole tiles of zeros among them (the first one too)."""
    b = many(Batch4(1, 4, 128, 16, [chunk, 1], [T, 70], seed=23), 1 << 16)
    r = np.random.default_rng(4)
    for x, (lo, hi) in zip(b.scale, (k, v)):
        x *= np.exp2(r.integers(lo, hi + 1, x.shape)).astype(np.float32)
    for x in b.scale:
        for a, n in ((0, 128), (300, 40)):
            page, slot = paged.token_slots(b.table[0], a, n, b.P)
            x[0, page, :, slot] = 0
    run(kp, b, **score)


def rising(chunk, T, level, d=64, seed=22):
    """A sequence whose scores are about level[t] at key t: the codes' own noise apart."""
    b = many(Batch4(1, 4, d, 16, [chunk, 1], [T, 70], seed=seed), 1 << 16)
    # q = 0.5 u, u a row of H times 1: <q, k> / sqrt(d) = level for k = level * c u
    u = paged4.hadamard(d)[5].astype(np.float32)
    b.Q = bf16(b.Q * 0.05 + 0.5 * u)
    rows = np.random.default_rng(5).standard_normal((T, 1, d)).astype(np.float32) * 0.1
    k = rows + (np.asarray(level, np.float32) * 2 * d ** 0.5 / d)[:, None, None] * u
    page, slot = paged.token_slots(b.table[0], 0, T, b.P)
    b.codes[0][0, page, :, slot], b.scale[0][0, page, :, slot] = paged4.encode(k)
    return b


@pytest.mark.parametrize("room", [0, 1 << 16])  # (the kernel for few rows, that for many)
@pytest.mark.parametrize("chunk,T", [(20, 900), (100, 900), (100, 2500)])
@pytest.mark.parametrize("rise,jump", [(0.02, 0), (0.3, 0), (0.02, 300), (-0.3, 0)])
@pytest.mark.parametrize("score", [dict(), dict(window=600), dict(slopes=True)])
def test_scores_that_rise(kp, rise, jump, score, chunk, T, room):
    """Maxima that move on with every tile, by a little and by much, and one that
    jumps by more than float32 weights have room for. (A vector along one row of H
    is one coordinate of its transform, which the outermost level holds: what the
    codes stand for rises as much, about.)"""
    at = np.arange(T)
    b = rising(chunk, T, rise * at + jump * (at >= 2 * T // 3))
    sc = scores(b, **score)
    run(kp, b, **sc) if room else run(kp, b, max_q=1, max_kv=64, **sc)


@pytest.mark.parametrize("chunk,T,jumps", [
    (20, 900, {2 * 128 + 100: 60.0}), (100, 900, {2 * 128 + 100: 85.0}), (100, 2500, {2 * 128 + 100: 200.0}),
    (20, 900, {6 * 128 + 2: 85.0, 128 + 5: 86.0}), (20, 2500, {5 * 128 + 70: 80.0, 9 * 128 + 5: 84.0}),
    (100, 2500, {5 * 128 + 70: 300.0, 9 * 128 + 5: 310.0}), (100, 2500, {0: 100.0}), (100, 2500, {2300: 100.0})])
@pytest.mark.parametrize("score", [dict(), dict(window=2400)])
def test_keys_that_stand_out(kp, chunk, T, jumps, score):
    """Single keys far above what came before them, early and late, in one state of a row and in several."""
    level = np.zeros(T)
    for t, x in jumps.items():
        level[t] = x / 2.5  # (the outermost level holds 2.51 of sqrt(d))
    run(kp, rising(chunk, T, level * 2.5), **score)


@pytest.mark.parametrize("d", [64, 128])
def test_infinite_and_nan_keys_that_are_seen(kp, d):
    """Rows that see a NaN are NaN, and no others."""
    b = many(Batch4(1, 4, d, 16, [60, 1], [600, 70], seed=29), 1 << 16)
    page, slot = paged.token_slots(b.table[0], 570, 1, b.P)
    for x in b.scale:
        x[0, page, :, slot] = np.nan
    out, lse = kp.pages4_attend(*b.dev4(kp), return_lse=True)
    out, lse = out.float().cpu().numpy(), lse.cpu().numpy()
    first = 570 - 540  # the row at position 570
    assert np.isnan(out[first: 60]).all() and np.isnan(lse[first: 60]).all()
    ref = [x.copy() for x in b.ref4()]
    for x in ref:
        x[first: 60] = np.nan
    check4(out, lse, ref)


def test_page_numbers_out_of_range(kp):
    import torch

    b = many(Batch4(2, 4, 64, 16, [1, 50], [100, 370], seed=10), 1 << 16)
    good = b.table.copy()
    b.table[0, 2], b.table[1, 1], b.table[1, 20] = 1 << 20, -1, 1 << 30
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = kp.pages4_attend(*b.dev4(kp), return_lse=True, status=status)
    assert int(status) == 1
    b2 = Batch4(2, 4, 64, 16, [1, 50], [100, 370], seed=10)
    for s, i in ((0, 2), (1, 1), (1, 20)):
        for x in b2.scale:
            x[0, good[s, i]] = 0
    check4(out.float().cpu().numpy(), lse.cpu().numpy(), b2.ref4())


def test_rows_behind_the_last_sequence_and_streams(kp):
    import torch

    b = many(Batch4(2, 8, 128, 16, [1, 90], [40, 600], seed=9, extra_rows=50), 1 << 16)
    dev = b.dev4(kp)
    out = torch.full((b.tokens, b.hq, b.d), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((b.tokens, b.hq), 7.0, device="cuda")
    other = [torch.empty_like(x) for x in (out, lse)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for st, (o, z) in zip(streams, ((out, lse), other)):  # two calls at once
        st.wait_stream(torch.cuda.current_stream())
        kp.pages4_attend(*dev, out=o, lse=z, stream=st)
    for st in streams:
        st.synchronize()
    assert (out[91:] == 7).all() and (lse[91:] == 7).all()
    assert torch.equal(out[:91], other[0][:91]) and torch.equal(lse[:91], other[1][:91])
    check4(out.float().cpu().numpy(), lse.cpu().numpy(), b.ref4())


def test_captured_graph(kp):
    """Replayed with other lengths than it was captured with."""
    import torch

    b = many(Batch4(2, 8, 64, 32, [40, 30], [700, 400], seed=31), 1 << 16)
    pages, layer, Q, table, kv_len, q_start = b.dev4(kp)
    out = torch.empty(b.tokens, b.hq, b.d, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(b.tokens, b.hq, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        kp.pages4_attend(pages, layer, Q, table, kv_len, q_start, out=out, lse=lse)
    for lens in ((700, 400), (41, 390), (699, 30)):
        b.kv, b.kv_len = list(lens), np.array(lens, np.int32)
        kv_len.copy_(torch.from_numpy(b.kv_len))
        graph.replay()
        check4(out.float().cpu().numpy(), lse.cpu().numpy(), b.ref4())
