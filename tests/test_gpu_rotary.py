"""New tokens turned by position on their way into the pages, bf16 and 4 bits,
against the plain restatement (oracle/paged4.py). The rotation's float32 steps
are part of its definition, so K, Q and codes are equal bit for bit."""

import ctypes

import numpy as np
import pytest

from oracle import paged, paged4

from paged4_util import Batch4, bf16, new_rows, place, rotation, token_positions

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kp():
    import torch

    from shared_quantized_kv_gb300 import build, kvpool

    assert torch.cuda.is_available()
    build.build()
    return kvpool


def up(x):
    import torch

    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def fused(b, hq, seed=5):
    """Q, K and V of new tokens, rows of one projection: host parts and device views."""
    import torch

    rows = new_rows(b, seed, hq + 2 * b.hk)
    dev = up(rows).to(torch.bfloat16)
    cut = lambda x: (x[:, :hq], x[:, hq: hq + b.hk], x[:, hq + b.hk:])
    return cut(rows), cut(dev)


def turned(b, x, cos, sin, at, interleaved):
    """x of all rows, turned where a position is given (rows at -1 stay)."""
    out = np.array(x, np.float32)
    out[at >= 0] = paged4.turn(x[at >= 0], cos[at[at >= 0]], sin[at[at >= 0]], interleaved)
    return out


CASES = [  # new tokens, held tokens
    ([1, 1, 1], [1, 16, 200]),
    ([0, 40, 1, 0, 300], [5, 55, 64, 200, 301]),
    ([17], [17]),
]
TURNS = [(1.0, False), (1.0, True), (0.5, False), (0.5, True), (0.25, False), (0.75, False), (0.75, True)]


@pytest.mark.parametrize("part,interleaved", TURNS)
@pytest.mark.parametrize("hk,hq,d,P", [(2, 4, 64, 16), (8, 32, 128, 64), (3, 21, 128, 32), (32, 32, 64, 128)])
@pytest.mark.parametrize("q,kv", CASES)
def test_append(kp, hk, hq, d, P, q, kv, part, interleaved):
    import torch

    b = Batch4(hk, hq, d, P, q, kv, seed=len(q), layers=3, layer=1, extra_rows=5)
    (hq_rows, hk_rows, hv_rows), (Q, K, V) = fused(b, hq)
    offset = 1000
    R = int(d * part)
    cos, sin = rotation(offset + 301, R)
    turn = kp.Rotary(up(cos), up(sin), interleaved, offset)
    at = token_positions(b)
    at = np.where(at >= 0, at + offset, -1)
    want_k, want_q = turned(b, hk_rows, cos, sin, at, interleaved), turned(b, hq_rows, cos, sin, at, interleaved)
    # bf16
    Kp, Vp, layer, _, table, kv_len, q_start = b.dev()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full(Q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    got = kp.pages_append_rotary(Kp, Vp, layer, K, V, table, kv_len, q_start, turn, Q=Q, Q_out=out, status=status)
    assert got is out and int(status) == 0
    rows = at >= 0
    assert np.array_equal(out.float().cpu().numpy()[rows], bf16(want_q)[rows])
    assert (out[torch.from_numpy(~rows).cuda()] == 7).all()
    place(b.K, layer, bf16(want_k), b)
    place(b.V, layer, hv_rows, b)
    assert np.array_equal(Kp.float().cpu().numpy(), b.K, equal_nan=True)
    assert np.array_equal(Vp.float().cpu().numpy(), b.V, equal_nan=True)
    # 4 bits
    pages = b.pages4(kp)
    got = kp.pages4_append(pages, layer, K, V, table, kv_len, q_start, rotary=turn, Q=Q, status=status)
    assert int(status) == 0 and np.array_equal(got.float().cpu().numpy()[rows], bf16(want_q)[rows])
    for x, codes, scale, rows in zip((want_k, hv_rows), b.codes, b.scale, range(2)):
        u, t = paged4.encode(x)
        place(codes, layer, u, b)
        place(scale, layer, t, b)
        assert np.array_equal(pages[rows].cpu().numpy(), paged4.pack(codes))
        assert np.array_equal(pages[2 + rows].cpu().numpy(), scale, equal_nan=True)


@pytest.mark.parametrize("d", [64, 128])
def test_without_rotation_and_read_back(kp, d):
    """Codes of vectors as they are, and what they stand for: t times an exact sum, rounded twice."""
    import torch

    b = Batch4(3, 3, d, 16, [30, 0, 1, 64], [30, 7, 90, 80], seed=4, layers=2, layer=1, extra_rows=3)
    (_, hk_rows, hv_rows), (_, K, V) = fused(b, 3)
    pages, layer, _, table, kv_len, q_start = b.dev4(kp)
    assert kp.pages4_append(pages, layer, K, V, table, kv_len, q_start) is None
    for x, n in ((hk_rows, 0), (hv_rows, 1)):
        u, t = paged4.encode(x)
        place(b.codes[n], layer, u, b)
        place(b.scale[n], layer, t, b)
        assert np.array_equal(pages[n].cpu().numpy(), paged4.pack(b.codes[n]))
    out = [torch.full((b.tokens, 3, d), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    kp.pages4_read(pages, layer, table, kv_len, q_start, b.tokens, *out)
    H = paged4.hadamard(d)
    for x, got in ((hk_rows, out[0]), (hv_rows, out[1])):
        u, t = paged4.encode(x)
        want = bf16(((u - 7.5) @ H).astype(np.float32) * t[..., None])
        n = b.q_start[-1]
        assert np.array_equal(got.float().cpu().numpy()[:n], want[:n])
        assert (got[n:] == 7).all()
        # and it is near what was written: mean square error of the quantiser
        err = ((want[:n] - x[:n]) ** 2).sum() / (x[:n] ** 2).sum()
        assert err < 0.3352 ** 2 / 4
    # whole sequences, from another layer's view of the same table: all tokens held
    start = torch.tensor(np.concatenate([[0], np.cumsum(b.kv)]), dtype=torch.int32, device="cuda")
    Kr, Vr = kp.pages4_read(pages, layer, table, kv_len, start, int(start[-1]))
    r = 0
    for s, n in enumerate(b.kv):
        page, slot = paged.token_slots(b.table[s], 0, n, b.P)
        for got, u, t in ((Kr, b.codes[0], b.scale[0]), (Vr, b.codes[1], b.scale[1])):
            want = bf16(((u[layer, page, :, slot] - 7.5) @ H).astype(np.float32) * t[layer, page, :, slot][..., None])
            assert np.array_equal(got[r: r + n].float().cpu().numpy(), want)
        r += n


@pytest.mark.parametrize("part,interleaved", TURNS)
def test_positions_and_q_in_place(kp, part, interleaved):
    """Each token's row of the tables given; Q turned where it is."""
    import torch

    d, hq = 128, 5
    b = Batch4(2, hq, d, 32, [3, 50], [40, 50], seed=6, extra_rows=2)
    (hq_rows, hk_rows, _), (Q, K, V) = fused(b, hq)
    cos, sin = rotation(77, int(d * part))
    at = np.random.default_rng(0).integers(0, 77, b.tokens).astype(np.int32)
    want_q = bf16(paged4.turn(hq_rows, cos[at], sin[at], interleaved))
    want_k = bf16(paged4.turn(hk_rows, cos[at], sin[at], interleaved))
    for four in (False, True):
        q = torch.empty_strided(Q.shape, Q.stride(), dtype=Q.dtype, device="cuda").copy_(Q)
        turn = kp.Rotary(up(cos), up(sin), interleaved)
        Kp, Vp, layer, _, table, kv_len, q_start = b.dev()
        if four:
            got = kp.pages4_append(b.pages4(kp), 0, K, V, table, kv_len, q_start, turn, Q=q, Q_out=q, positions=up(at))
        else:
            got = kp.pages_append_rotary(Kp, Vp, 0, K, V, table, kv_len, q_start, turn, Q=q, Q_out=q, positions=up(at))
            page, slot = paged.token_slots(b.table[1], 0, 50, b.P)
            assert np.array_equal(Kp[0].float().cpu().numpy()[page, :, slot], want_k[3:53])
        assert got is q
        assert np.array_equal(q.float().cpu().numpy()[:53], want_q[:53])
        assert np.array_equal(q.float().cpu().numpy()[53:], hq_rows[53:])


@pytest.mark.parametrize("four", [False, True])
def test_positions_outside_the_tables(kp, four):
    """Nothing is written for such a token, its Q neither, and it is recorded; the others are not touched by it."""
    import torch

    d, hq, hk = 64, 4, 2
    b = Batch4(hk, hq, d, 16, [1, 20], [30, 33], seed=7)
    (hq_rows, hk_rows, _), (Q, K, V) = fused(b, hq)
    cos, sin = rotation(33, d)
    at = token_positions(b).astype(np.int32)
    at[3], at[8], at[0] = -1, 33, 1 << 30
    ok = (at >= 0) & (at < 33)
    Kp, Vp, layer, _, table, kv_len, q_start = b.dev()
    pages = b.pages4(kp)
    before = Kp.clone(), pages.K.clone()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((b.tokens, hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
    turn = kp.Rotary(up(cos), up(sin))
    args = 0, K, V, table, kv_len, q_start, turn
    if four:
        kp.pages4_append(pages, *args, Q=Q, Q_out=out, positions=up(at), status=status)
        pg, read = kp._pages4(pages, status), kp.lib().kvpool_pages4_status
    else:
        kp.pages_append_rotary(Kp, Vp, *args, Q=Q, Q_out=out, positions=up(at), status=status)
        pg, read = kp._pages(Kp, Vp, status), kp.lib().kvpool_pages_status
    assert read(ctypes.byref(pg), None) == -1 and read(ctypes.byref(pg), None) == 0
    want = paged4.turn(hq_rows[ok], cos[at[ok]], sin[at[ok]])
    assert np.array_equal(out.float().cpu().numpy()[ok], bf16(want))
    assert (out[torch.from_numpy(~ok).cuda()] == 7).all()
    for i in range(b.tokens):
        s = 0 if i < 1 else 1
        p = int(b.kv[s] - b.q[s] + i - b.q_start[s])
        page, slot = b.table[s, p // 16], p % 16
        old, new = (before[1], pages.K) if four else (before[0], Kp)
        same = torch.equal(old[0, page, :, slot], new[0, page, :, slot])
        assert same == (not ok[i]), i
    # an offset that leaves the tables, and one whose sum passes 32 bits
    for offset in (33, (1 << 31) - 1, -34):
        status.zero_()
        kp.pages_append_rotary(Kp, Vp, 0, K, V, table, kv_len, q_start, kp.Rotary(up(cos), up(sin), False, offset),
                               status=status)
        assert int(status) == 4


@pytest.mark.parametrize("four", [False, True])
def test_pages_out_of_range_and_no_room(kp, four):
    """K and V are dropped and recorded, Q is turned all the same; positions before 0 get nothing."""
    import torch

    d, hk = 64, 2
    b = Batch4(hk, 2, d, 16, [2, 3, 5], [40, 50, 5], seed=8)
    (hq_rows, _, _), (Q, K, V) = fused(b, 2)
    table, kv_len, q_start = up(b.table), up(b.kv_len), up(b.q_start)
    table[0, 2] = 1 << 20          # tokens 38, 39
    kv_len[1] = 16 * b.table.shape[1] + 2  # tokens 2 ... behind the table's room: one fits
    kv_len[2] = 3                  # two positions before 0
    Kp, Vp, _, _, _, _, _ = b.dev()
    pages = b.pages4(kp)
    table[1, :] = int(b.table[1, 0])
    cos, sin = rotation(200, d)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((b.tokens, 2, d), 7.0, dtype=torch.bfloat16, device="cuda")
    before = (pages.K if four else Kp).clone()
    f = (lambda *a, **k: kp.pages4_append(pages, *a, **k)) if four else (lambda *a, **k: kp.pages_append_rotary(Kp, Vp, *a, **k))
    f(0, K, V, table, kv_len, q_start, kp.Rotary(up(cos), up(sin)), Q=Q, Q_out=out, status=status)
    assert int(status) == 1
    room = 16 * b.table.shape[1]
    at = np.array([38, 39, room - 1, room, room + 1, -1, -1, 0, 1, 2])
    at[5:7] = [-1, -1]
    rows = at >= 0
    assert np.array_equal(out.float().cpu().numpy()[rows], bf16(paged4.turn(hq_rows[rows], cos[at[rows]], sin[at[rows]])))
    assert (out[5:7] == 7).all()
    after = pages.K if four else Kp
    changed = [(int(a), int(c)) for a, c in (after != before).view(after.shape[1], hk, 16, -1).any(-1).any(1).nonzero()
               if four or not torch.isnan(before[0, a, 0, c]).all() or not torch.isnan(after[0, a, 0, c]).all()]
    want = sorted([(int(b.table[1, 0]), 15)] + [(int(b.table[2, 0]), i) for i in range(3)])
    assert sorted(changed) == want


@pytest.mark.parametrize("d", [64, 128])
def test_vectors_of_all_sizes(kp, d):
    """Zeros, infinities, NaN, the largest and the smallest bf16 values."""
    import torch

    hk, n = 2, 40
    b = Batch4(hk, hk, d, 16, [n], [n], seed=9)
    r = np.random.default_rng(1)
    x = bf16(r.standard_normal((n, hk, d)).astype(np.float32))
    x[1], x[2] = 0, bf16(np.float32(2.0) ** 120 * x[2])
    x[3, 0, 5], x[4, 1, 0], x[5, 0, d - 1] = np.inf, -np.inf, np.nan
    x[6, 0], x[7, 1, 1:] = bf16(np.float32(3.3e38) * np.sign(x[6, 0])), 0
    x[8] = bf16(x[8] * np.float32(2.0) ** -100)
    x[9] = 1.0  # one coordinate of H x alone
    dev = up(x).to(torch.bfloat16)
    pages, _, _, table, kv_len, q_start = b.dev4(kp)
    kp.pages4_append(pages, 0, dev, dev, table, kv_len, q_start)
    u, t = paged4.encode(x)
    for i in range(2):
        place(b.scale[i], 0, t, b)
        assert np.array_equal(pages[2 + i].cpu().numpy(), b.scale[i], equal_nan=True)
        place(b.codes[i], 0, u, b)
        got = paged4.unpack(pages[i].cpu().numpy())
        known = ~np.isnan(b.scale[i])
        assert np.array_equal(got[known], b.codes[i][known])
    K, V = kp.pages4_read(pages, 0, table, kv_len, q_start, n)
    assert torch.equal(K.view(torch.int16), V.view(torch.int16))
    K = K.float().cpu().numpy()
    assert (K[1] == 0).all() and np.isnan(K[3, 0]).all() and np.isnan(K[4, 1]).all() and np.isnan(K[5, 0]).all()
    fine = [i for i in range(n) if i not in (3, 4, 5, 6)]
    assert np.isfinite(K[fine]).all() and np.isfinite(K[3, 1]).all()


def test_graph_and_stream(kp):
    """Captured on another stream, replayed with other lengths, tables and rows."""
    import torch

    d, hk, hq = 128, 2, 8
    b = Batch4(hk, hq, d, 16, [1, 1], [40, 33], seed=10)
    (hq_rows, hk_rows, hv_rows), (Q, K, V) = fused(b, hq)
    pages, _, _, table, kv_len, q_start = b.dev4(kp)
    cos, sin = rotation(100, d)
    turn = kp.Rotary(up(cos), up(sin))
    out = torch.empty(2, hq, d, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        kp.pages4_append(pages, 0, K, V, table, kv_len, q_start, turn, Q=Q, Q_out=out)
    for lens in ((40, 33), (47, 20)):
        b.kv = list(lens)
        kv_len.copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        at = np.array([n - 1 for n in lens])
        u, t = paged4.encode(paged4.turn(hk_rows, cos[at], sin[at]))
        place(b.codes[0], 0, u, b)
        assert np.array_equal(pages.K.cpu().numpy(), paged4.pack(b.codes[0]))
        assert np.array_equal(out.float().cpu().numpy(), bf16(paged4.turn(hq_rows, cos[at], sin[at])))
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = kp.pages_append_rotary(*b.dev()[:2], 0, K, V, table, kv_len, q_start, turn, Q=Q, stream=st)
    st.synchronize()
    assert torch.equal(got, out)
