"""The shared pool and paged private caches together: attention over both in
one softmax against the oracle's float64 attention over the dequantised pool
and each row's own tokens, and a life of a few agents (chunks, single tokens,
forks, rejected drafts, compaction, ends) step by step."""

import ctypes

import numpy as np
import pytest

from oracle import attention, codec, paged
from shared_quantized_kv_gb300 import workloads as wl

from paged_util import Batch, bf16, check_attend
from parity_util import TOL, to_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kp():
    import torch

    from shared_quantized_kv_gb300 import build, kvpool

    assert torch.cuda.is_available()
    build.build()
    return kvpool


def own_tokens(table_row, K, V, layer, T, P):
    """K, V [kv_heads, T, d] of one sequence."""
    page, slot = paged.token_slots(table_row, 0, T, P)
    return K[layer, page, :, slot].transpose(1, 0, 2), V[layer, page, :, slot].transpose(1, 0, 2)


def reference(enc, Q, K, V, layer, table, kv_len, q_start):
    """float64 [tokens, q_heads, d]: every row an agent of its own whose tail is
    what it sees of its sequence; rows of no sequence have no tail."""
    P, d = K.shape[3:]
    Kh, Vh = attention.dequantise_f64(enc)
    n = Q.shape[0]
    most = max([1] + [int(t) for t in kv_len])
    Kt = np.zeros((n, K.shape[2], most, d), np.float32)
    Vt = Kt.copy()
    lens = np.zeros(n, np.int64)
    for s in range(len(kv_len)):
        a, b, T = int(q_start[s]), int(q_start[s + 1]), int(kv_len[s])
        k, v = own_tokens(table[s], K, V, layer, T, P)
        for i in range(b - a):
            lens[a + i] = T - (b - a) + i + 1
            Kt[a + i, :, :lens[a + i]] = k[:, :lens[a + i]]
            Vt[a + i, :, :lens[a + i]] = v[:, :lens[a + i]]
    bits = lambda x: wl.f32_to_bf16_bits(x)
    return attention.attend_f64(Kh, Vh, bits(Q), (bits(Kt), bits(Vt), lens))


class OneCache:
    """A Batch as pool.attend_pages takes a cache and its batch."""

    def __init__(self, b):
        import torch

        self.K, self.V, self.layer, Q, self.table, self.kv_len, self.q_start = b.dev()
        self.status_word = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.tokens, self.max_q, self.max_kv = b.tokens, max(b.q), max(b.kv)
        self.Q = Q


@pytest.mark.parametrize("hk,hq,d,ctx,bits,k_block,P,q,kv,max_rows", [
    (2, 8, 128, 300, 3, 0, 16, [1, 1, 1], [40, 1, 333], 0),            # a decode step
    (2, 8, 128, 700, 4, 32, 32, [1, 30, 0, 7], [500, 30, 9, 300], 0),   # chunks, block-scaled K
    (4, 4, 64, 1000, 2, 0, 64, [50, 100], [130, 100], 0),
    (1, 7, 128, 260, 3, 0, 128, [25, 1], [200, 77], 64),                # slices of 9 tokens, the last of 8
    (2, 4, 64, 130, 3, 32, 16, [90, 1, 1], [900, 2, 50], 16),           # many slices
    (1, 2, 64, 4000, 3, 0, 32, [1], [3000], 0),                          # one row, long contexts
])
def test_pool_and_pages_in_one_softmax(kp, hk, hq, d, ctx, bits, k_block, P, q, kv, max_rows):
    import torch

    w = wl.custom("pages", 1, hk, hq, d, ctx, 1, "lognormal", bits=(bits,))
    K, V = wl.layer_kv(w, 0)
    pool = kp.KVPool(1, hk, d, ctx, [bits], max_rows=max_rows, k_block=k_block)
    pool.compress(0, to_dev(K), to_dev(V))
    enc = codec.encode_layer(K, V, bits, k_block=k_block)
    b = Batch(hk, hq, d, P, q, kv, seed=ctx, layers=2, layer=1, extra_rows=3)
    c = OneCache(b)
    out = torch.full((b.tokens, hq, d), float("nan"), device="cuda")
    got = pool.attend_pages(0, c.Q, c, c, page_layer=1, out=out).cpu().numpy()
    assert pool.status() == 0 and int(c.status_word.cpu()[0]) == 0
    ref = reference(enc, b.Q, b.K, b.V, 1, b.table, b.kv_len, b.q_start)
    err = attention.row_rel_error(got.astype(np.float64), ref)
    assert err <= TOL, err
    # the rows of no sequence are the pool's alone
    alone = pool.attend(0, c.Q[-3:].contiguous()).cpu().numpy()
    assert attention.row_rel_error(got[-3:].astype(np.float64), alone.astype(np.float64)) <= TOL
    pool.close()


def test_attend_pages_refusals(kp):
    import torch

    lib = kp.lib()
    by = ctypes.byref
    w = wl.custom("pages_ref", 1, 2, 4, 64, 130, 1, "lognormal")
    pool = kp.KVPool(2, 2, 64, 130, [3, 3], max_rows=64)
    K, V = wl.layer_kv(w, 0)
    pool.compress(0, to_dev(K), to_dev(V))
    b = Batch(2, 4, 64, 16, [1, 20], [30, 40], seed=1)
    c = OneCache(b)
    out = torch.empty(21, 4, 64, device="cuda")
    need = pool.attend_pages_ws_bytes(21, 4)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    assert need > 0
    assert pool.attend_pages_ws_bytes(0, 4) == 0 and pool.attend_pages_ws_bytes(21, 3) == 0

    def call(layer=0, page_layer=0, out_=None, ws_bytes=need, ws_=None, hq=4, scale=0.0, **pg_change):
        pg = kp._pages(c.K, c.V, c.status_word)
        for k, v in pg_change.items():
            setattr(pg, k, v)
        sq = kp._seqs(c.table, c.kv_len, c.q_start, 21, 20, 40)
        return lib.kvpool_attend_pages(pool.handle, layer, by(pg), page_layer, by(sq), c.Q.data_ptr(), hq,
                                       out.data_ptr() if out_ is None else out_, scale,
                                       ws.data_ptr() if ws_ is None else ws_, ws_bytes, None)

    assert call() == 0
    assert call(layer=1) == -2  # not compressed
    for bad in (dict(layer=2), dict(page_layer=1), dict(page_layer=-1), dict(ws_bytes=need - 1), dict(ws_=ws.data_ptr() + 4),
                dict(out_=out.data_ptr() + 4), dict(hq=3), dict(hq=2 * 65), dict(scale=-1.0), dict(kv_heads=1),
                dict(head_dim=128), dict(page_tokens=24)):
        assert call(**bad) == -1, bad
    torch.cuda.synchronize()
    pool.close()


def test_python_refusals(kp):
    import torch

    b = Batch(2, 4, 64, 16, [1, 20], [30, 40], seed=2)
    K, V, layer, Q, table, kv_len, q_start = b.dev()
    ok = dict(K_pages=K, V_pages=V, layer=0, Q=Q, table=table, kv_len=kv_len, q_start=q_start)
    for bad in (dict(Q=Q.float()), dict(Q=Q[:, :, :32]), dict(Q=Q.cpu()), dict(Q=Q.transpose(0, 1)), dict(kv_len=kv_len[:1]),
                dict(q_start=q_start[:2]), dict(table=table.long()), dict(table=table[:, ::2]), dict(K_pages=K[0]),
                dict(V_pages=V[:, :-1]), dict(K_pages=K.float()), dict(first=kv_len), dict(prefix=q_start),
                dict(slopes=torch.ones(3, device="cuda")), dict(slopes=torch.ones(4)), dict(out=Q.float()),
                dict(out=Q[:3]), dict(lse=torch.ones(21, 4, device="cuda").double()), dict(table=table.cpu())):
        with pytest.raises(ValueError):
            kp.pages_attend(**{**ok, **bad})
    with pytest.raises(kp.KVPoolError):
        kp.pages_attend(**ok, window=-1)
    for bad in (dict(window=(1 << 32) + 1), dict(max_q=1 << 32), dict(max_kv=1 << 31)):
        with pytest.raises(ValueError):
            kp.pages_attend(**ok, **bad)
    for src, dst in (([1 << 32], [1]), ([0], [(1 << 32) + 1]), ([0, -(1 << 32)], [1, 2]), ([0], [])):
        with pytest.raises(ValueError):
            kp.pages_copy(K, V, src, dst)
    with pytest.raises(kp.KVPoolError):
        kp.pages_attend(**{**ok, "layer": 1})
    new = torch.zeros(21, 2, 64, dtype=torch.bfloat16, device="cuda")
    for kv in ((new[:5], new), (new.float(), new.float()), (new[:, :1], new[:, :1]), (new.cpu(), new.cpu())):
        with pytest.raises(ValueError):
            kp.pages_append(K, V, 0, *kv, table, kv_len, q_start)
    with pytest.raises(ValueError):
        kp.pages_copy(K, V, [0], [1, 2])
    with pytest.raises(kp.KVPoolError):
        kp.pages_copy(K, V, [0], [0])


def test_a_life_of_agents(kp):
    """Three layers, a pool and a cache of few pages: every step's attention of
    every layer against the tokens that each agent should have."""
    import torch

    L, hk, hq, d, P, ctx = 3, 2, 8, 128, 16, 200
    w = wl.custom("life", L, hk, hq, d, ctx, 1, "lognormal")
    pool = kp.KVPool(L, hk, d, ctx, [3] * L, max_rows=64)
    encs = []
    for l in range(L):
        K, V = wl.layer_kv(w, l)
        pool.compress(l, to_dev(K), to_dev(V))
        encs.append(codec.encode_layer(K, V, 3))
    cache = kp.PagedCache(L, hk, d, pages=24, page_tokens=P)
    r = np.random.default_rng(0)
    held = {}  # agent -> K, V [L, tokens, hk, d]

    def step(agents, counts):
        batch = cache.grow(agents, counts)
        n = sum(counts)
        new = [bf16(r.standard_normal((L, n, hk, d), dtype=np.float32)) for _ in range(2)]
        Q = bf16(r.standard_normal((L, n, hq, d), dtype=np.float32))
        a = 0
        for s, c in zip(agents, counts):
            held[s] = [np.concatenate([x, y[:, a: a + c]], 1) for x, y in zip(held[s], new)]
            a += c
        dev = lambda x: torch.from_numpy(x).cuda().to(torch.bfloat16)
        lens = [held[s][0].shape[1] for s in agents]
        start = np.concatenate([[0], np.cumsum(counts)])
        for l in range(L):
            cache.append(l, dev(new[0][l]), dev(new[1][l]), batch)
            own, lse = cache.attend(l, dev(Q[l]), batch, return_lse=True)
            both = pool.attend_pages(l, dev(Q[l]), cache, batch)
            # the agents' tokens in pages of their own, for the restatement
            pages = sum(-(-t // P) for t in lens)
            Kp = np.zeros((1, pages, hk, P, d), np.float32)
            Vp, table, at = Kp.copy(), np.zeros((len(agents), max(-(-t // P) for t in lens)), np.int64), 0
            for i, s in enumerate(agents):
                m = -(-lens[i] // P)
                table[i, :m] = np.arange(at, at + m)
                at += m
                page, slot = paged.token_slots(table[i], 0, lens[i], P)
                Kp[0, page, :, slot], Vp[0, page, :, slot] = held[s][0][l], held[s][1][l]
            check_attend(own.float().cpu().numpy(), lse.cpu().numpy(),
                         paged.attend(Kp, Vp, 0, Q[l], table, lens, start), max(lens))
            err = attention.row_rel_error(both.cpu().numpy().astype(np.float64),
                                          reference(encs[l], Q[l], Kp, Vp, 0, table, lens, start))
            assert err <= TOL, err
        assert cache.status() == 0 and pool.status() == 0

    empty = lambda: [np.zeros((L, 0, hk, d), np.float32) for _ in range(2)]
    a, b = cache.new(), cache.new()
    held[a], held[b] = empty(), empty()
    step([a, b], [37, 1])            # a prompt and a single token
    step([b, a], [1, 1])
    c = cache.fork(a)                # two agents that share 38 tokens, the last page partly filled
    held[c] = [x.copy() for x in held[a]]
    step([a, b, c], [1, 1, 1])       # each writes its own
    step([c], [30])
    cache.truncate(c, 45)            # drafts rejected
    held[c] = [x[:, :45] for x in held[c]]
    e = cache.fork(c)
    held[e] = [x.copy() for x in held[c]]
    step([c, e], [5, 2])
    cache.free(a)
    del held[a]
    assert cache.compact() > 0
    used = {p for s in held for p in cache.pager.table(s)}
    assert used == set(range(len(used)))
    step([b, c, e], [40, 1, 17])
    before = {s: cache.pager.length(s) for s in held}
    with pytest.raises(kp.KVPoolError) as err:  # more than there is: nobody has grown
        cache.grow([b, e], [10, 1000])
    assert err.value.code == -4 and before == {s: cache.pager.length(s) for s in held}
    step([b, c, e], [1, 1, 1])
    for s in list(held):
        cache.free(s)
    assert cache.pager.free_pages() == 24
    cache.close()
    pool.close()
