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
