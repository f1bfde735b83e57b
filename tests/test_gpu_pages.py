"""Paged private caches on the GPU: append, copy and attention against the
plain float64 restatement (oracle/paged.py). Slots behind a sequence's last
token hold NaN in every test, unused table entries numbers out of range."""

import numpy as np
import pytest

from oracle import paged

from paged_util import Batch, bf16, check_attend

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kp():
    import torch

    from shared_quantized_kv_gb300 import build, kvpool

    assert torch.cuda.is_available()
    build.build()
    return kvpool


def run(kp, b, max_q=None, max_kv=None, **score):
    """pages_attend of a Batch, host results, checked against the reference."""
    import torch

    K, V, layer, Q, table, kv_len, q_start = b.dev()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    dev = {}
    for k, v in score.items():
        dev[k] = torch.from_numpy(v).cuda() if isinstance(v, np.ndarray) else v
    dev["softmax_scale"] = dev.pop("scale", 0.0)
    out, lse = kp.pages_attend(K, V, layer, Q, table, kv_len, q_start, max_q=max_q, max_kv=max_kv, return_lse=True,
                               status=status, **dev)
    assert int(status.cpu()[0]) == 0
    out, lse = out.float().cpu().numpy(), lse.cpu().numpy()
    check_attend(out, lse, b.ref(**score), max(b.kv + [1]))
    return out, lse


HEADS = [(2, 4, 64), (3, 3, 64), (2, 8, 128), (1, 7, 128), (2, 16, 128), (1, 20, 64)]


@pytest.mark.parametrize("hk,hq,d", HEADS)
@pytest.mark.parametrize("P", [16, 32, 64, 128])
def test_decode(kp, hk, hq, d, P):
    """One new token per sequence, lengths around page and unit borders."""
    kv = [1, 2, 15, 16, 17, 63, 64, 65, 128, 129, 300]
    run(kp, Batch(hk, hq, d, P, [1] * len(kv), kv, seed=P), max_q=1, max_kv=300)


@pytest.mark.parametrize("hk,hq,d", HEADS)
@pytest.mark.parametrize("P", [16, 128])
def test_ragged_batch(kp, hk, hq, d, P):
    """Empty, single-token and chunk sequences, whole prompts among them."""
    q = [0, 1, 5, 130, 0, 1, 77, 16, 0]
    kv = [9, 200, 5, 131, 0, 1, 400, 333, 40]
    run(kp, Batch(hk, hq, d, P, q, kv, seed=hq), max_q=130, max_kv=400)


@pytest.mark.parametrize("hk,hq,d", [(1, 4, 128), (2, 2, 64)])
def test_long_context_is_split(kp, hk, hq, d):
    """Few sequences over long contexts: the keys are split and merged."""
    run(kp, Batch(hk, hq, d, 64, [1, 2], [9001, 12345], seed=3), max_q=2)
    run(kp, Batch(hk, hq, d, 32, [40], [7777], seed=4))


def test_hints_do_not_change_results(kp):
    """max_q and max_kv below the real ones give right results too."""
    b = Batch(2, 8, 128, 16, [3, 70, 1], [500, 90, 2000], seed=5)
    for hint in (dict(), dict(max_q=1, max_kv=16), dict(max_q=4, max_kv=2000), dict(max_q=70, max_kv=64)):
        run(kp, b, **hint)


SCORES = {
    "cap": dict(cap=5.0),
    "slopes": dict(slopes=True),
    "window": dict(window=33),
    "window1": dict(window=1),
    "scale": dict(scale=0.5),
    "cap_slopes_window": dict(cap=20.0, slopes=True, window=100),
    "documents": dict(first=True),
    "prefix": dict(prefix=True),
    "prefix_window": dict(prefix=True, window=20),
    "prefix_window_documents_cap": dict(prefix=True, window=20, first=True, cap=30.0, slopes=True),
}


def scores(b, cap=0.0, slopes=False, window=0, first=False, prefix=False, scale=None, seed=0):
    r = np.random.default_rng(seed)
    sc = {}
    if cap:
        sc["cap"] = cap
    if scale:
        sc["scale"] = scale
    if slopes:
        sc["slopes"] = r.uniform(0.0, 0.2, b.hq).astype(np.float32)
    if window:
        sc["window"] = window
    if first:
        # documents of 29 tokens; some rows' document begins behind the row (they see nothing of their own)
        f = np.zeros(b.tokens, np.int32)
        for s in range(len(b.q)):
            for i in range(b.q[s]):
                p = b.kv[s] - b.q[s] + i
                f[b.q_start[s] + i] = p // 29 * 29 if i % 11 else p + 1
        sc["first"] = f
    if prefix:
        sc["prefix"] = np.array([(0, 3, 45, 1000, -5)[i % 5] for i in range(len(b.q))], np.int32)
    return sc


@pytest.mark.parametrize("name", sorted(SCORES))
@pytest.mark.parametrize("hk,hq,d,chunk", [(2, 4, 64, 1), (1, 7, 128, 1), (2, 8, 128, 90), (2, 2, 64, 150)])
def test_scores(kp, name, hk, hq, d, chunk):
    q = [1, 0, chunk, min(chunk, 3), chunk]
    kv = [1, 50, max(chunk, 160), 700, max(chunk, 300)]
    b = Batch(hk, hq, d, 32, q, kv, seed=7)
    run(kp, b, max_q=chunk, **scores(b, **SCORES[name]))


@pytest.mark.parametrize("chunk", [1, 100])
def test_masked_keys_may_hold_anything(kp, chunk):
    """Infinities and NaN in keys that a row does not see (behind it, before
    its document, outside its window) leave it as it is."""
    import torch

    b = Batch(2, 8, 128, 32, [chunk, chunk], [400, 350], seed=8)
    run(kp, b, max_q=chunk, window=150)
    # tokens that no row's window reaches
    for s, t in ((0, 400), (1, 350)):
        page, slot = paged.token_slots(b.table[s], 0, t - chunk - 149, b.P)
        b.K[0, page[::3], :, slot[::3]] = np.nan
        b.V[0, page[::3], :, slot[::3]] = np.inf
        b.V[0, page[1::3], :, slot[1::3]] = np.nan
    # (bounded against the reference, as base is: rows that are recomputed because a masked NaN met
    # a weight of 0 keep float32 weights, rows that are not round them to bf16)
    run(kp, b, max_q=chunk, window=150)
    if chunk > 1:
        # the last token of a chunk: every row before it must not see it
        page, slot = paged.token_slots(b.table[0], 399, 1, b.P)
        b.K[0, page, :, slot] = np.nan
        b.V[0, page, :, slot] = np.nan
        K, V, layer, Q, table, kv_len, q_start = b.dev()
        out, lse = kp.pages_attend(K, V, layer, Q, table, kv_len, q_start, max_q=chunk, window=150, return_lse=True)
        out, lse = out.float().cpu().numpy(), lse.cpu().numpy()
        assert np.isnan(out[chunk - 1]).all()
        ref = [x.copy() for x in b.ref(window=150)]
        for x in ref:
            x[chunk - 1] = np.nan
        check_attend(out, lse, ref, 400)


def test_rows_behind_the_last_sequence_stay(kp):
    import torch

    b = Batch(2, 8, 128, 16, [1, 33], [40, 60], seed=9, extra_rows=50)
    K, V, layer, Q, table, kv_len, q_start = b.dev()
    for max_q in (1, 33):
        out = torch.full((b.tokens, b.hq, b.d), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((b.tokens, b.hq), 7.0, device="cuda")
        kp.pages_attend(K, V, layer, Q, table, kv_len, q_start, max_q=max_q, out=out, lse=lse)
        assert (out[34:] == 7).all() and (lse[34:] == 7).all()
        check_attend(out.float().cpu().numpy(), lse.cpu().numpy(), b.ref(), 60)


def test_page_numbers_out_of_range(kp):
    """They read as zeros, write nothing, and are recorded."""
    import torch

    b = Batch(2, 4, 64, 16, [1, 20], [100, 70], seed=10)
    good = b.table.copy()
    b.table[0, 2], b.table[1, 1] = 1 << 20, -1
    K, V, layer, Q, table, kv_len, q_start = b.dev()
    K, V = torch.nan_to_num(K), torch.nan_to_num(V)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pg = kp._pages(K, V, status)
    import ctypes

    for max_q in (1, 20):
        out, lse = kp.pages_attend(K, V, layer, Q, table, kv_len, q_start, max_q=max_q, return_lse=True, status=status)
        assert kp.lib().kvpool_pages_status(ctypes.byref(pg), None) == -1
        assert kp.lib().kvpool_pages_status(ctypes.byref(pg), None) == 0
        b2 = Batch(2, 4, 64, 16, [1, 20], [100, 70], seed=10)
        for s, i in ((0, 2), (1, 1)):
            b2.K[0, good[s, i]] = 0
            b2.V[0, good[s, i]] = 0
        check_attend(out.float().cpu().numpy(), lse.cpu().numpy(), b2.ref(), 100)
    before = K.clone(), V.clone()
    b.table[0, 6] = -3
    new = torch.ones(21, 2, 64, dtype=torch.bfloat16, device="cuda")
    kp.pages_append(K, V, 0, new[:1], new[:1], torch.from_numpy(b.table[:1]).cuda(), kv_len[:1], q_start[:2],
                    status=status)
    assert kp.lib().kvpool_pages_status(ctypes.byref(pg), None) == -1
    assert torch.equal(K, before[0]) and torch.equal(V, before[1])


@pytest.mark.parametrize("hk,d,P", [(2, 64, 16), (8, 128, 64), (32, 64, 32), (5, 128, 128)])
@pytest.mark.parametrize("q", [[1, 1, 1], [0, 40, 1, 0, 300], [17]])
def test_append(kp, hk, d, P, q):
    """New tokens land in their slots of the layer and nothing else changes;
    K and V are rows of one fused projection."""
    import torch

    kv = [n + (0, 15, 63, 200, 1)[i] for i, n in enumerate(q)]
    b = Batch(hk, hk, d, P, q, kv, seed=len(q), layers=3, layer=1, extra_rows=5)
    K, V, layer, Q, table, kv_len, q_start = b.dev()
    r = np.random.default_rng(1)
    rows = bf16(r.standard_normal((b.tokens, 4 * hk, d), dtype=np.float32))
    fused = torch.from_numpy(rows).cuda().to(torch.bfloat16)
    kp.pages_append(K, V, layer, fused[:, hk: 2 * hk], fused[:, 3 * hk:], table, kv_len, q_start)
    paged.append(b.K, layer, rows[:, hk: 2 * hk], b.table, b.kv_len, b.q_start)
    paged.append(b.V, layer, rows[:, 3 * hk:], b.table, b.kv_len, b.q_start)
    assert np.array_equal(K.float().cpu().numpy(), b.K, equal_nan=True)
    assert np.array_equal(V.float().cpu().numpy(), b.V, equal_nan=True)


@pytest.mark.parametrize("n", [0, 1, 3, 64, 65, 200, 4000])
def test_copy(kp, n):
    """Whole pages of every layer; sources may repeat."""
    import torch

    pages = 2 * n + 7
    g = torch.Generator(device="cuda")
    g.manual_seed(n)
    K, V = (torch.randn(3, pages, 2, 16, 64, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    order = np.random.default_rng(n).permutation(pages)
    src, dst = order[:n].tolist(), order[n: 2 * n].tolist()
    if n > 2:
        src[1] = src[0]
    Kr, Vr = K.clone(), V.clone()
    if n:
        Kr[:, dst], Vr[:, dst] = Kr[:, src], Vr[:, src]
    kp.pages_copy(K, V, src, dst)
    assert torch.equal(K, Kr) and torch.equal(V, Vr)


def test_large_pages_copy(kp):
    """Pages larger than a CTA's piece, odd numbers of heads."""
    import torch

    K, V = (torch.randn(2, 9, 5, 128, 128, device="cuda").to(torch.bfloat16) for _ in range(2))
    Kr, Vr = K.clone(), V.clone()
    Kr[:, [8, 2]], Vr[:, [8, 2]] = Kr[:, [0, 5]], Vr[:, [0, 5]]
    kp.pages_copy(K, V, [0, 5], [8, 2])
    assert torch.equal(K, Kr) and torch.equal(V, Vr)


def test_strided_queries_and_other_stream(kp):
    """Q as rows of a fused projection, everything on a stream of its own."""
    import torch

    b = Batch(2, 8, 128, 16, [1, 40], [100, 70], seed=11)
    K, V, layer, Q, table, kv_len, q_start = b.dev()
    fused = torch.cat([torch.full_like(Q[:, :2], float("nan")), Q, torch.full_like(Q[:, :2], float("nan"))], 1)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    out, lse = kp.pages_attend(K, V, layer, fused[:, 2:10], table, kv_len, q_start, return_lse=True, stream=st)
    st.synchronize()
    check_attend(out.float().cpu().numpy(), lse.cpu().numpy(), b.ref(), 100)


def test_offsets_past_32_bits(kp):
    """A cache of more than 2^32 bytes per layer, the sequence in its last pages."""
    import torch

    pages, hk, P, d = 70000, 4, 64, 128  # 70000 x 64 KiB = 4.6e9 bytes per layer
    K, V = (torch.zeros(1, pages, hk, P, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    b = Batch(hk, 8, d, P, [1, 70], [100, 300], seed=12)
    Kb, Vb, layer, Q, table, kv_len, q_start = b.dev()
    n = b.K.shape[1]
    K[0, -n:], V[0, -n:] = Kb[0], Vb[0]
    table = torch.where(table >= 0, table + (pages - n), table)
    for max_q in (1, 70):
        out, lse = kp.pages_attend(K, V, 0, Q, table, kv_len, q_start, max_q=max_q, return_lse=True)
        check_attend(out.float().cpu().numpy(), lse.cpu().numpy(), b.ref(), 300)
    new = torch.full((2, hk, d), 3.0, dtype=torch.bfloat16, device="cuda")
    kp.pages_append(K, V, 0, new, new, table, kv_len, torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda"))
    for s in range(2):
        t = int(kv_len[s]) - 1
        assert (K[0, int(table[s, t // P]), :, t % P] == 3).all()
    kp.pages_copy(K, V, [pages - 1, pages - 2], [0, 1])
    bits = lambda x: x.view(torch.int16)  # unused slots hold NaN, which equals nothing
    assert torch.equal(bits(K[0, 0]), bits(K[0, -1])) and torch.equal(bits(V[0, 1]), bits(V[0, -2]))


def test_captured_graph_reads_the_tables_of_its_replay(kp):
    """append and attend in a graph; between replays lengths, tables and tokens change."""
    import torch

    b = Batch(2, 8, 128, 16, [1, 1], [40, 33], seed=13)
    K, V, layer, Q, table, kv_len, q_start = b.dev()
    nk = torch.zeros(2, 2, 128, dtype=torch.bfloat16, device="cuda")
    nv = torch.zeros_like(nk)
    out = torch.empty(2, 8, 128, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(2, 8, device="cuda")

    def step():
        kp.pages_append(K, V, 0, nk, nv, table, kv_len, q_start)
        kp.pages_attend(K, V, 0, Q, table, kv_len, q_start, max_q=1, out=out, lse=lse)

    step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    r = np.random.default_rng(2)
    free = sorted(set(range(b.K.shape[1])) - set(b.table[b.table >= 0].tolist()))
    b.table[0, 3], b.table[1, 3] = free[0], free[1]
    table.copy_(torch.from_numpy(b.table))
    for t0, t1 in ((40, 33), (49, 60), (52, 61)):
        new = [bf16(r.standard_normal((2, 2, 128), dtype=np.float32)) for _ in range(2)]
        b.kv, b.kv_len = [t0, t1], np.array([t0, t1], np.int32)
        for X in (b.K, b.V):
            np.nan_to_num(X, copy=False)
        K.copy_(torch.from_numpy(b.K)), V.copy_(torch.from_numpy(b.V))
        paged.append(b.K, 0, new[0], b.table, b.kv_len, b.q_start)
        paged.append(b.V, 0, new[1], b.table, b.kv_len, b.q_start)
        nk.copy_(torch.from_numpy(new[0]))
        nv.copy_(torch.from_numpy(new[1]))
        kv_len.copy_(torch.from_numpy(b.kv_len))
        graph.replay()
        assert np.array_equal(K.float().cpu().numpy(), b.K)
        check_attend(out.float().cpu().numpy(), lse.cpu().numpy(), b.ref(), 61)


def test_same_call_same_bits(kp):
    b = Batch(2, 8, 128, 16, [1, 40, 3], [5000, 300, 64], seed=14)
    x, y = run(kp, b), run(kp, b)
    assert np.array_equal(x[0], y[0]) and np.array_equal(x[1], y[1])
