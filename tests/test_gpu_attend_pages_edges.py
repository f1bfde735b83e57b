"""Attention over the pool and pages together, where it is easily wrong: rows of
no sequence beside a pool of scores far below 0, many KV heads, one workspace
for several calls, other streams, captured graphs."""

import numpy as np
import pytest

from oracle import attention, codec
from shared_quantized_kv_gb300 import workloads as wl

from paged_util import Batch, bf16
from parity_util import TOL, to_dev
from test_gpu_attend_pages import OneCache, reference
from test_gpu_pages import kp  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu


def filled(kp, w, layers=1, scale=None, **options):
    """A pool of w's shape and the oracle's encoding of each layer; scale: a factor of K and what is added to it."""
    pool = kp.KVPool(layers, w.kv_heads, w.head_dim, w.ctx, list(w.bits)[:1] * layers, **options)
    encs = []
    for l in range(layers):
        K, V = wl.layer_kv(w, l)
        if scale is not None:
            K = wl.f32_to_bf16_bits(wl.bf16_bits_to_f32(K) * scale[0] + scale[1])
        pool.compress(l, to_dev(K), to_dev(V))
        encs.append(codec.encode_layer(K, V, w.bits[0]))
    return pool, encs


def close(got, ref):
    err = attention.row_rel_error(got.cpu().numpy().astype(np.float64), ref)
    assert err <= TOL, err


@pytest.mark.parametrize("d,level", [(64, 5.0), (64, 11.0), (64, 12.0), (64, 13.5), (64, 16.0), (128, 10.0), (128, 40.0)])
def test_rows_of_no_sequence_and_a_pool_far_below_0(kp, d, level):
    """Scores of about -level * sqrt(d) nats: the pool's largest lies below what
    float32 weights reach from 0 (-87 nats)."""
    w = wl.custom("below", 1, 2, 8, d, 300, 1, "lognormal", bits=(4,))
    pool, encs = filled(kp, w, scale=(0.05, 1.0))
    b = Batch(2, 8, d, 16, [1, 5], [40, 33], seed=d, extra_rows=4)
    b.Q = bf16(0.05 * b.Q - np.float32(level))
    c = OneCache(b)
    got = pool.attend_pages(0, c.Q, c, c)
    assert pool.status() == 0
    close(got, reference(encs[0], b.Q, b.K, b.V, 0, b.table, b.kv_len, b.q_start))
    pool.close()
@pytest.mark.parametrize("hk,hq,max_rows,tokens", [(40, 40, 0, 400), (32, 32, 1024, 700), (20, 40, 1024, 513)])
def test_more_rows_than_one_wave_of_the_pool(kp, hk, hq, max_rows, tokens):
    """max_rows admits more rows at once than the pool's attention has CTAs for."""
    w = wl.custom("wave", 1, hk, hq, 64, 130, 1, "lognormal", bits=(3,))
    pool, encs = filled(kp, w, max_rows=max_rows)
    b = Batch(hk, hq, 64, 64, [tokens - 3, 1, 2], [tokens - 3, 50, 70], seed=hk)
    c = OneCache(b)
    got = pool.attend_pages(0, c.Q, c, c)
    assert pool.status() == 0 and int(c.status_word.cpu()[0]) == 0
    ref = reference(encs[0], b.Q[-40:], b.K, b.V, 0, b.table, b.kv_len, np.array([0, 37, 38, 40]))
    close(got[-40:], ref)
    few = Batch(hk, hq, 64, 64, [40], [40], seed=hk)  # the first rows, alone
    few.K, few.V, few.table, few.Q = b.K, b.V, b.table[:1], b.Q[:40]
    close(got[:40], reference(encs[0], few.Q, few.K, few.V, 0, few.table, few.kv_len, few.q_start))
    pool.close()


def test_more_kv_heads_than_the_gpu_has_sms_is_refused(kp):
    import torch

    sms = torch.cuda.get_device_properties(0).multi_processor_count
    pool = kp.KVPool(1, sms + 1, 64, 130, [3])
    assert pool.attend_pages_ws_bytes(5, sms + 1) == 0 and pool.attend_ws_bytes(5, sms + 1) == 0
    pool.close()


def test_one_workspace_for_calls_in_turn_and_a_graph(kp):
    """Two layers' calls share a workspace on a stream of their own, then in a
    graph whose replays see other lengths."""
    import torch

    w = wl.custom("turn", 2, 2, 8, 128, 500, 1, "lognormal", bits=(3,))
    pool, encs = filled(kp, w, layers=2, max_rows=64)
    b = Batch(2, 8, 128, 16, [30, 1, 7], [200, 90, 7], seed=31, layers=2, layer=0, extra_rows=2)
    b.K[1], b.V[1] = -b.K[0], 2 * b.V[0]
    c = OneCache(b)
    st = torch.cuda.Stream()
    ws = torch.empty(pool.attend_pages_ws_bytes(b.tokens, 8), dtype=torch.uint8, device="cuda")
    out = torch.empty(2, b.tokens, 8, 128, device="cuda")

    def refs():
        return [reference(encs[l], b.Q, np.nan_to_num(b.K), np.nan_to_num(b.V), l, b.table, b.kv_len, b.q_start)
                for l in range(2)]

    def both(stream):
        for l in range(2):
            pool.attend_pages(l, c.Q, c, c, workspace=ws, out=out[l], stream=stream)

    torch.cuda.synchronize()
    for _ in range(3):
        both(st)
    st.synchronize()
    for l, ref in enumerate(refs()):
        close(out[l], ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both(None)
    for kv in ([200, 90, 7], [60, 33, 50], [30, 1, 96]):
        need = [-(-t // b.P) for t in kv]
        order = np.random.default_rng(sum(kv)).permutation(b.K.shape[1])
        if sum(need) > len(order):
            order = np.resize(order, sum(need))
        b.table[:] = -7
        at = 0
        for s, n in enumerate(need):
            b.table[s, :n] = order[at: at + n]
            at += n
        b.kv, b.kv_len = kv, np.array(kv, np.int32)
        for X in (b.K, b.V):
            np.nan_to_num(X, copy=False)
        c.K.copy_(torch.from_numpy(b.K)), c.V.copy_(torch.from_numpy(b.V))
        c.table.copy_(torch.from_numpy(b.table)), c.kv_len.copy_(torch.from_numpy(b.kv_len))
        out.fill_(float("nan"))
        graph.replay()
        for l, ref in enumerate(refs()):
            close(out[l], ref)
    assert pool.status() == 0 and int(c.status_word.cpu()[0]) == 0
    pool.close()


def test_two_streams_at_once(kp):
    """Calls on two streams, each with a workspace of its own, many times: the same bits each time."""
    import torch

    w = wl.custom("streams", 1, 2, 8, 128, 700, 1, "lognormal", bits=(3,))
    pool, encs = filled(kp, w, max_rows=128)
    bs = [Batch(2, 8, 128, 16, [1, 1, 2], [700, 30, 300], seed=32, extra_rows=1),
          Batch(2, 8, 128, 16, [120, 50], [600, 400], seed=33).many()]
    cs = [OneCache(b) for b in bs]
    cs[1].max_q, cs[1].max_kv = bs[1].tokens, 1 << 16
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for st, c, g in zip(streams, cs, got):
            g.append(pool.attend_pages(0, c.Q, c, c, stream=st))
    torch.cuda.synchronize()
    for b, g in zip(bs, got):
        close(g[0], reference(encs[0], b.Q, b.K, b.V, 0, b.table, b.kv_len, b.q_start))
        for x in g[1:]:
            assert torch.equal(x, g[0])
    assert pool.status() == 0
    pool.close()
