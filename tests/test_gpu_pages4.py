"""Attention over paged caches in 4 bits, page copies and the cache's life, against
the plain float64 restatement (oracle/paged4.py). Slots behind a sequence's last
token have NaN scales in every test, unused table entries numbers out of range."""

import ctypes

import numpy as np
import pytest

from oracle import paged, paged4

from paged4_util import Batch4, bf16, check4, new_rows, place, rotation

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kp():
    import torch

    from shared_quantized_kv_gb300 import build, kvpool

    assert torch.cuda.is_available()
    build.build()
    return kvpool


def run(kp, b, max_q=None, max_kv=None, **score):
    """pages4_attend of a Batch4, host results, checked against the reference."""
    import torch

    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    dev = {k: torch.from_numpy(v).cuda() if isinstance(v, np.ndarray) else v for k, v in score.items()}
    dev["softmax_scale"] = dev.pop("scale", 0.0)
    out, lse = kp.pages4_attend(*b.dev4(kp), max_q=max_q, max_kv=max_kv, return_lse=True, status=status, **dev)
    assert int(status.cpu()[0]) == 0
    out, lse = out.float().cpu().numpy(), lse.cpu().numpy()
    check4(out, lse, b.ref4(**score))
    return out, lse


HEADS = [(2, 4, 64), (3, 3, 64), (2, 8, 128), (1, 7, 128), (2, 16, 128), (1, 20, 64)]


@pytest.mark.parametrize("hk,hq,d", HEADS)
@pytest.mark.parametrize("P", [16, 32, 64, 128])
def test_decode(kp, hk, hq, d, P):
    """One new token per sequence, lengths around page and unit borders."""
    kv = [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 128, 129, 300]
    run(kp, Batch4(hk, hq, d, P, [1] * len(kv), kv, seed=P), max_q=1, max_kv=300)


@pytest.mark.parametrize("hk,hq,d", HEADS)
@pytest.mark.parametrize("P", [16, 128])
def test_ragged_batch(kp, hk, hq, d, P):
    """Empty, single-token and chunk sequences, whole prompts among them."""
    q = [0, 1, 5, 130, 0, 1, 77, 16, 0]
    kv = [9, 200, 5, 131, 0, 1, 400, 333, 40]
    run(kp, Batch4(hk, hq, d, P, q, kv, seed=hq), max_q=130, max_kv=400)


@pytest.mark.parametrize("hk,hq,d", [(1, 4, 128), (2, 2, 64)])
def test_long_context_is_split(kp, hk, hq, d):
    """Few sequences over long contexts: the keys are split and merged."""
    run(kp, Batch4(hk, hq, d, 64, [1, 2], [9001, 12345], seed=3), max_q=2)
    run(kp, Batch4(hk, hq, d, 32, [40], [7777], seed=4))
    run(kp, Batch4(hk, hq, d, 16, [3, 1], [8000, 1], seed=5), max_q=3)


def test_hints_do_not_change_results(kp):
    """max_q and max_kv below the real ones give right results too."""
    b = Batch4(2, 8, 128, 16, [3, 70, 1], [500, 90, 2000], seed=5)
    for hint in (dict(), dict(max_q=1, max_kv=16), dict(max_q=4, max_kv=2000), dict(max_q=70, max_kv=64),
                 dict(max_q=8, max_kv=1)):
        run(kp, b, **hint)


SCORES = {
    "cap": dict(cap=5.0),
    "wide_cap": dict(cap=100.0),
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
@pytest.mark.parametrize("hk,hq,d,chunk", [(2, 4, 64, 1), (1, 7, 128, 1), (2, 8, 128, 90), (2, 2, 64, 150), (1, 3, 128, 4)])
def test_scores(kp, name, hk, hq, d, chunk):
    q = [1, 0, chunk, min(chunk, 3), chunk]
    kv = [1, 50, max(chunk, 160), 700, max(chunk, 300)]
    b = Batch4(hk, hq, d, 32, q, kv, seed=7)
    run(kp, b, max_q=chunk, **scores(b, **SCORES[name]))


@pytest.mark.parametrize("chunk", [1, 5, 100])
def test_masked_keys_may_hold_anything(kp, chunk):
    """Infinite and NaN scales of keys that a row does not see (behind it, before
    its document, outside its window) leave it as it is."""
    b = Batch4(2, 8, 128, 32, [chunk, chunk], [400, 350], seed=8)
    run(kp, b, max_q=chunk, window=150)
    for s, t in ((0, 400), (1, 350)):  # tokens that no row's window reaches
        page, slot = paged.token_slots(b.table[s], 0, t - chunk - 149, b.P)
        for X in b.scale:
            X[0, page[::3], :, slot[::3]] = np.nan
            X[0, page[1::3], :, slot[1::3]] = np.inf
    run(kp, b, max_q=chunk, window=150)
    if chunk > 1:
        # the last token of a chunk: every row before it must not see it
        page, slot = paged.token_slots(b.table[0], 399, 1, b.P)
        for X in b.scale:
            X[0, page, :, slot] = np.nan
        out, lse = kp.pages4_attend(*b.dev4(kp), max_q=chunk, window=150, return_lse=True)
        out, lse = out.float().cpu().numpy(), lse.cpu().numpy()
        assert np.isnan(out[chunk - 1]).all() and np.isnan(lse[chunk - 1]).all()
        ref = [x.copy() for x in b.ref4(window=150)]
        for x in ref:
            x[chunk - 1] = np.nan
        check4(out, lse, ref)


@pytest.mark.parametrize("chunk", [1, 4, 70])
@pytest.mark.parametrize("d", [64, 128])
def test_far_scores(kp, chunk, d):
    """Queries of any size (one row's scores 2^8 larger than another's), keys and
    values of very different norms, and the largest score last."""
    b = Batch4(2, 4, d, 16, [chunk, 1], [300, 200], seed=11)
    r = np.random.default_rng(3)
    b.Q *= np.exp2(r.integers(-8, 5, b.Q.shape[:2]))[..., None].astype(np.float32)
    b.scale[0] *= np.exp2(r.integers(-6, 3, b.scale[0].shape)).astype(np.float32)
    b.scale[1] *= np.exp2(r.integers(-40, 40, b.scale[1].shape)).astype(np.float32)
    page, slot = paged.token_slots(b.table[0], 290, 1, b.P)
    b.scale[0][0, page, :, slot] *= 16
    run(kp, b, max_q=chunk)


@pytest.mark.parametrize("chunk", [1, 40])
def test_zero_rows_and_keys(kp, chunk):
    """A query of zeros weighs all keys alike; keys of zeros score 0; one huge and one tiny channel."""
    b = Batch4(2, 4, 64, 32, [chunk], [100], seed=12)
    b.Q[0, 0] = 0
    b.Q[chunk - 1, 1] = 0
    b.Q[chunk - 1, 1, 3], b.Q[chunk - 1, 2, 5] = bf16(np.array([1e-30, 1e4]))
    page, slot = paged.token_slots(b.table[0], 10, 30, b.P)
    b.scale[0][0, page, :, slot] = 0
    b.scale[1][0, page[::2], :, slot[::2]] = 0
    run(kp, b, max_q=chunk)


def test_rows_behind_the_last_sequence_stay(kp):
    import torch

    b = Batch4(2, 8, 128, 16, [1, 33], [40, 60], seed=9, extra_rows=50)
    for max_q in (1, 33):
        out = torch.full((b.tokens, b.hq, b.d), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((b.tokens, b.hq), 7.0, device="cuda")
        kp.pages4_attend(*b.dev4(kp), max_q=max_q, out=out, lse=lse)
        assert (out[34:] == 7).all() and (lse[34:] == 7).all()
        check4(out.float().cpu().numpy(), lse.cpu().numpy(), b.ref4())


def test_page_numbers_out_of_range(kp):
    """They read as zeros and are recorded; so are sequences longer than their table."""
    import torch

    b = Batch4(2, 4, 64, 16, [1, 20], [100, 70], seed=10)
    good = b.table.copy()
    b.table[0, 2], b.table[1, 1] = 1 << 20, -1
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for max_q in (1, 20):
        dev = b.dev4(kp)
        pg = kp._pages4(dev[0], status)
        out, lse = kp.pages4_attend(*dev, max_q=max_q, return_lse=True, status=status)
        assert kp.lib().kvpool_pages4_status(ctypes.byref(pg), None) == -1
        assert kp.lib().kvpool_pages4_status(ctypes.byref(pg), None) == 0
        b2 = Batch4(2, 4, 64, 16, [1, 20], [100, 70], seed=10)
        for s, i in ((0, 2), (1, 1)):
            for X in b2.scale:
                X[0, good[s, i]] = 0
        check4(out.float().cpu().numpy(), lse.cpu().numpy(), b2.ref4())
    K, V = kp.pages4_read(dev[0], 0, dev[3], dev[4], torch.tensor([0, 100, 170], dtype=torch.int32, device="cuda"), 170,
                          status=status)
    assert kp.lib().kvpool_pages4_status(ctypes.byref(pg), None) == -1
    for X in (K, V):
        assert (X[32:48] == 0).all() and (X[116:132] == 0).all() and torch.isfinite(X).all()


def test_more_tokens_than_the_table_has_room_for(kp):
    """Tokens behind the table's room are seen by no row, rows of them see all before."""
    import torch

    b = Batch4(2, 4, 64, 16, [3], [48], seed=13)
    b.table = b.table[:, :3].copy()
    pages, layer, Q, table, kv_len, q_start = b.dev4(kp)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = kp.pages4_attend(pages, layer, Q, table, kv_len + 2, q_start, return_lse=True, status=status)
    assert int(status) == 1
    # row 0 is at position 47, rows 1 and 2 behind the room: all see the 48 tokens
    ref = b.ref4()
    Q1 = Q.clone()
    for i in range(3):
        Q1[2] = Q[i]
        o, z = kp.pages4_attend(pages, layer, Q1, table, kv_len, q_start, return_lse=True)
        assert torch.equal(o[2], out[i]) and torch.equal(z[2], lse[i])
    assert np.isfinite(ref[1]).all()


def test_strided_queries_and_other_stream(kp):
    """Q as rows of a fused projection, everything on a stream of its own."""
    import torch

    b = Batch4(2, 8, 128, 16, [1, 40], [100, 70], seed=11)
    pages, layer, Q, table, kv_len, q_start = b.dev4(kp)
    fused = torch.cat([torch.full_like(Q[:, :2], float("nan")), Q, torch.full_like(Q[:, :2], float("nan"))], 1)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    out, lse = kp.pages4_attend(pages, layer, fused[:, 2:10], table, kv_len, q_start, return_lse=True, stream=st)
    st.synchronize()
    check4(out.float().cpu().numpy(), lse.cpu().numpy(), b.ref4())


def test_offsets_past_32_bits(kp):
    """Codes of more than 2^32 bytes per layer, the sequence in its last pages."""
    import torch

    pages, hk, P, d = 270000, 4, 64, 128  # 270000 x 16 KiB = 4.4e9 bytes of K codes
    big = kp.Pages4(*(torch.zeros(1, pages, hk, P, d // 2, dtype=torch.uint8, device="cuda") for _ in range(2)),
                    *(torch.zeros(1, pages, hk, P, device="cuda") for _ in range(2)))
    b = Batch4(hk, 8, d, P, [1, 70], [100, 300], seed=12)
    small, layer, Q, table, kv_len, q_start = b.dev4(kp)
    n = b.K.shape[1]
    for X, Y in zip(big, small):
        X[0, -n:] = Y[0]
    table = torch.where(table >= 0, table + (pages - n), table)
    for max_q in (1, 70):
        out, lse = kp.pages4_attend(big, 0, Q, table, kv_len, q_start, max_q=max_q, return_lse=True)
        check4(out.float().cpu().numpy(), lse.cpu().numpy(), b.ref4())
    new = torch.full((2, hk, d), 3.0, dtype=torch.bfloat16, device="cuda")
    start = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    kp.pages4_append(big, 0, new, new, table, kv_len, start)
    for K in kp.pages4_read(big, 0, table, kv_len, start, 2):
        # a constant vector is one coordinate of H x, beyond the outermost level: 7.5 steps of it, and half a step of the rest
        u, t = paged4.encode(np.full((d,), 3.0, np.float32))
        assert np.array_equal(K.float().cpu().numpy(), np.broadcast_to(bf16(paged4.values(u, t)), (2, hk, d)))
    kp.pages4_copy(big, [pages - 1, pages - 2], [0, 1])
    for X in big:
        x = X if X.dtype == torch.uint8 else X.view(torch.int32)
        assert torch.equal(x[0, 0], x[0, -1]) and torch.equal(x[0, 1], x[0, -2])


@pytest.mark.parametrize("n", [0, 1, 3, 64, 65, 200])
def test_copy(kp, n):
    """Whole pages of every layer, codes and scales; sources may repeat."""
    import torch

    pages = 2 * n + 7
    g = torch.Generator(device="cuda")
    g.manual_seed(n)
    cache = kp.pages4_empty(3, pages, 2, 16, 64)
    for X in cache[:2]:
        X.random_(0, 256, generator=g)
    for X in cache[2:]:
        X.normal_(generator=g)
    order = np.random.default_rng(n).permutation(pages)
    src, dst = order[:n].tolist(), order[n: 2 * n].tolist()
    if n > 2:
        src[1] = src[0]
    ref = [X.clone() for X in cache]
    for X in ref:
        if n:
            X[:, dst] = X[:, src]
    kp.pages4_copy(cache, src, dst)
    assert all(torch.equal(X, Y) for X, Y in zip(cache, ref))


def test_captured_graph_reads_the_tables_of_its_replay(kp):
    """append and attend in a graph; between replays lengths, tables and tokens change."""
    import torch

    b = Batch4(2, 8, 128, 16, [1, 1], [40, 33], seed=13)
    pages, layer, Q, table, kv_len, q_start = b.dev4(kp)
    nk = torch.zeros(2, 2, 128, dtype=torch.bfloat16, device="cuda")
    nv = torch.zeros_like(nk)
    out = torch.empty(2, 8, 128, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(2, 8, device="cuda")

    def step():
        kp.pages4_append(pages, 0, nk, nv, table, kv_len, q_start)
        kp.pages4_attend(pages, 0, Q, table, kv_len, q_start, max_q=1, out=out, lse=lse)

    step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    free = sorted(set(range(b.K.shape[1])) - set(b.table[b.table >= 0].tolist()))
    b.table[0, 3], b.table[1, 3] = free[0], free[1]
    table.copy_(torch.from_numpy(b.table))
    for X in b.scale:
        np.nan_to_num(X, copy=False)
    for i, (t0, t1) in enumerate(((40, 33), (49, 60), (52, 61))):
        new = [bf16(np.random.default_rng((i, j)).standard_normal((2, 2, 128), dtype=np.float32)) for j in range(2)]
        b.kv, b.kv_len = [t0, t1], np.array([t0, t1], np.int32)
        for X, Y in zip(pages, b.pages4(kp)):
            X.copy_(Y)
        for j in range(2):
            u, t = paged4.encode(new[j])
            place(b.codes[j], 0, u, b)
            place(b.scale[j], 0, t, b)
        nk.copy_(torch.from_numpy(new[0]))
        nv.copy_(torch.from_numpy(new[1]))
        kv_len.copy_(torch.from_numpy(b.kv_len))
        graph.replay()
        assert np.array_equal(pages.K.cpu().numpy(), paged4.pack(b.codes[0]))
        check4(out.float().cpu().numpy(), lse.cpu().numpy(), b.ref4())


def test_same_call_same_bits(kp):
    b = Batch4(2, 8, 128, 16, [1, 40, 3], [5000, 300, 64], seed=14)
    x, y = run(kp, b), run(kp, b)
    assert np.array_equal(x[0], y[0]) and np.array_equal(x[1], y[1])


@pytest.mark.parametrize("bits", [4, 16])
def test_agents_lives(kp, bits):
    """A cache as agents use it: prompts, decode steps, forks, drafts taken back,
    ends, a compaction, several layers, a rotation; every step's attention against
    the restatement of the same tokens, and the cache read back."""
    import torch

    layers, hk, hq, d, P = 2, 2, 8, 64, 16
    cache = kp.PagedCache(layers, hk, d, 40, P, bits=bits)
    cos, sin = rotation(400, d)
    turn = kp.Rotary(torch.from_numpy(cos).cuda(), torch.from_numpy(sin).cuda(), False, 30)
    r = np.random.default_rng(5)
    held = {}  # per sequence and layer: rotated keys and values, as they went in

    def step(seqs, counts, padding=0):
        batch = cache.grow(seqs, counts)
        n = sum(counts)
        at = np.concatenate([len(held[s][0][0]) + np.arange(c) for s, c in zip(seqs, counts)] or [[]]).astype(int) + 30
        for layer in range(layers):
            rows = bf16(r.standard_normal((n + padding, hq + 2 * hk, d)).astype(np.float32))
            dev = torch.from_numpy(rows).cuda().to(torch.bfloat16)
            Q = cache.append(layer, dev[:, hq: hq + hk], dev[:, hq + hk:], batch, rotary=turn, Q=dev[:, :hq])
            out, lse = cache.attend(layer, Q, batch, return_lse=True)
            k = paged4.turn(rows[:n, hq: hq + hk], cos[at], sin[at])
            q = bf16(paged4.turn(rows[:n, :hq], cos[at], sin[at]))
            i = 0
            for s, c in zip(seqs, counts):
                held[s][layer] = [np.concatenate([a, x[i: i + c]]) for a, x in zip(held[s][layer], (k, rows[:n, hq + hk:]))]
                K, V = held[s][layer]
                T = len(K)
                # one sequence, its tokens in pages of their own
                pages = -(-T // P)
                b = Batch4.__new__(Batch4)
                full = [np.zeros((pages * P, hk, d), np.float32) for _ in range(2)]
                full[0][:T], full[1][:T] = K, V
                coded = [paged4.encode(x) for x in full]
                shaped = [x.reshape(pages, P, *x.shape[1:]).swapaxes(1, 2) for c in coded for x in c]
                args = q[i: i + c], np.arange(pages)[None], [T], [0, c]
                if c and bits == 4:
                    ref = paged4.attend(shaped[0], shaped[1], shaped[2], shaped[3], *args, P)
                    check4(out[i: i + c].float().cpu().numpy(), lse[i: i + c].cpu().numpy(), ref)
                elif c:
                    from paged_util import check_attend

                    kv = [bf16(x).reshape(pages, P, hk, d).swapaxes(1, 2)[None] for x in full]
                    check_attend(out[i: i + c].float().cpu().numpy(), lse[i: i + c].cpu().numpy(),
                                 paged.attend(*kv, 0, *args), T)
                i += c
        assert cache.status() == 0

    def new():
        s = cache.new()
        held[s] = [[np.zeros((0, hk, d), np.float32)] * 2 for _ in range(layers)]
        return s

    a, b = new(), new()
    step([a, b], [37, 5])
    step([a, b], [1, 1], padding=3)
    c = cache.fork(a)
    held[c] = [list(x) for x in held[a]]
    step([c, a, b], [4, 1, 60])
    cache.truncate(c, 39)  # drafts taken back
    held[c] = [[x[:39] for x in kv] for kv in held[c]]
    step([c, b], [2, 1])
    cache.free(a)
    assert cache.compact() >= 0
    step([b, c], [1, 17])
    if bits == 4:
        for layer in range(layers):
            for s, (K, V) in zip((b, c), cache.read(layer, [b, c])):
                for got, x in zip((K, V), held[s][layer]):
                    u, t = paged4.encode(x)
                    want = bf16(((u - 7.5) @ paged4.hadamard(d)).astype(np.float32) * t[..., None])
                    assert np.array_equal(got.float().cpu().numpy(), want)
        assert cache.read(0, [cache.new()])[0][0].shape == (0, hk, d)
    else:
        with pytest.raises(ValueError):
            cache.read(0, [b])
    assert cache.status() == 0
    cache.close()


def test_joint_softmax_takes_bf16_pages(kp):
    """A 4-bit cache is refused there, by name."""
    import torch

    cache = kp.PagedCache(1, 2, 64, 4, 16, bits=4)
    batch = cache.grow([cache.new()], [3])
    pool = kp.KVPool(1, 2, 64, 130, [4])
    Q = torch.zeros(3, 4, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="16 bits"):
        pool.attend_pages(0, Q, cache, batch)
    with pytest.raises(ValueError):
        kp.pages4_attend(cache.pages4._replace(K=cache.pages4.K.view(torch.int8)), 0, Q, batch.table, batch.kv_len, batch.q_start)
    with pytest.raises(ValueError):
        kp.pages4_attend(cache.pages4._replace(V_scale=cache.pages4.V_scale[:, :2]), 0, Q, batch.table, batch.kv_len, batch.q_start)
    with pytest.raises(ValueError):
        kp.pages4_attend(cache.pages4, 0, Q.float(), batch.table, batch.kv_len, batch.q_start)
    with pytest.raises(ValueError):
        cache.append(0, Q[:, :2], Q[:, :2], batch, Q=Q)
    with pytest.raises(ValueError):
        cache.append(0, Q[:2, :2], Q[:2, :2], batch)
    pool.close()
    cache.close()


@pytest.mark.parametrize("rows", [1, 90])
def test_two_graphs_and_an_eager_call_at_once(kp, rows):
    """Two captured calls over one cache (each with a workspace of its own) and an eager one, replayed side by side."""
    import torch

    b = Batch4(2, 16, 64, 16, [rows, 1], [700, 300], seed=51)
    b.table = np.pad(b.table, ((0, 0), (0, 4096 - b.table.shape[1])), constant_values=-9)
    dev = b.dev4(kp)
    outs = [(torch.empty(b.tokens, b.hq, b.d, dtype=torch.bfloat16, device="cuda"), torch.empty(b.tokens, b.hq, device="cuda"))
            for _ in range(3)]
    streams = [torch.cuda.Stream() for _ in range(3)]
    graphs = []
    for st, (o, z) in zip(streams[:2], outs):
        st.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            kp.pages4_attend(*dev, out=o, lse=z)
        graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(5):
        for st, g in zip(streams, graphs):
            with torch.cuda.stream(st):
                g.replay()
        kp.pages4_attend(*dev, out=outs[2][0], lse=outs[2][1], stream=streams[2])
    torch.cuda.synchronize()
    for o, z in outs:
        assert torch.equal(o, outs[0][0]) and torch.equal(z, outs[0][1])
    check4(outs[0][0].float().cpu().numpy(), outs[0][1].cpu().numpy(), b.ref4())
