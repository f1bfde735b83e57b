"""Paged attention by the kernel for many rows where scores lie far apart: single
keys that stand out from what came before them by almost what a float32 weight
has room for (2^128, 88.7 nats), early and late in a row's keys."""

import numpy as np
import pytest

from oracle import attention, codec, paged
from shared_quantized_kv_gb300 import workloads as wl

from paged_util import Batch, bf16, check_attend
from parity_util import TOL, to_dev
from test_gpu_attend_pages import OneCache, reference
from test_gpu_pages import kp, run  # noqa: F401 (kp: a fixture)

pytestmark = pytest.mark.gpu


def standing_out(chunk, T, jumps, seed=27):
    """A sequence whose scores are about 0, but jumps[t] (nats, in steps of a half) at key t."""
    b = Batch(1, 4, 64, 16, [chunk, 1], [T, 70], seed=seed).many()
    u = np.zeros(64, np.float32)
    u[:16] = 1
    level = np.zeros(T, np.float32)
    for t, jump in jumps.items():
        assert t < T - chunk
        level[t] = jump
    page, slot = paged.token_slots(b.table[0], 0, T, b.P)
    K = b.K[0, page, 0, slot] * 0.1
    K[:, :16] = (level / 2)[:, None]  # <u, k> / sqrt(64) = level
    b.K[0, page, 0, slot] = bf16(K)
    b.Q = bf16(b.Q * 0.1 * (u == 0) + u)
    return b


@pytest.mark.parametrize("chunk,T", [(20, 900), (100, 900), (20, 2500), (100, 2500)])
@pytest.mark.parametrize("jump", [80.0, 86.5, 87.0, 87.5, 88.0, 88.5, 89.0, 90.0])
@pytest.mark.parametrize("score", [dict(), dict(window=2400)])
def test_one_key_stands_out(kp, chunk, T, jump, score):
    """In the second half of a tile in the middle: the reference follows before the next tile."""
    run(kp, standing_out(chunk, T, {2 * 128 + 100: jump}), **score)


@pytest.mark.parametrize("chunk,T,a,b", [(20, 900, 6 * 128 + 2, 128 + 5),            # one CTA: the last tile of a slot, the first of the other
                                         (20, 2500, 5 * 128 + 70, 9 * 128 + 5),      # CTAs of a cluster
                                         (100, 2500, 5 * 128 + 70, 9 * 128 + 5)])
@pytest.mark.parametrize("ja,jb", [(87.0, 88.5), (86.0, 88.0), (88.5, 88.5), (85.0, 95.0)])
@pytest.mark.parametrize("score", [dict(), dict(window=2400)])
def test_states_that_lag_are_merged(kp, chunk, T, a, b, ja, jb, score):
    """Two keys of about the same weight in different states of a row: one as the
    state's first reference, one so late that its reference never followed."""
    run(kp, standing_out(chunk, T, {a: ja, b: jb}), **score)


@pytest.mark.parametrize("chunk,T", [(20, 900), (100, 900), (100, 2500)])
@pytest.mark.parametrize("jump", [60.0, 87.0, 88.5, 95.0])
def test_states_that_lag_join_the_pool(kp, chunk, T, jump):
    """A late key that stands out, in a row's own tokens, and a pool whose scores are as far up."""
    import torch

    b = standing_out(chunk, T, {T - chunk - 3: jump, T - chunk - 200: jump - 1})
    w = wl.custom("far", 1, 1, 4, 64, 130, 1, "lognormal", bits=(4,))
    K, V = wl.layer_kv(w, 0)
    K = wl.bf16_bits_to_f32(K) * 0.1
    K[..., :16] += jump / 2  # scores about as large as the late key's
    K = wl.f32_to_bf16_bits(K)
    pool = kp.KVPool(1, 1, 64, 130, [4])
    pool.compress(0, to_dev(K), to_dev(V))
    enc = codec.encode_layer(K, V, 4)
    c = OneCache(b)
    c.max_q, c.max_kv = b.tokens, 1 << 16
    got = pool.attend_pages(0, c.Q, c, c).cpu().numpy()
    assert pool.status() == 0 and int(c.status_word.cpu()[0]) == 0
    err = attention.row_rel_error(got.astype(np.float64), reference(enc, b.Q, b.K, b.V, 0, b.table, b.kv_len, b.q_start))
    assert err <= TOL, err
    pool.close()


@pytest.mark.parametrize("chunk,T", [(20, 900), (100, 900), (100, 2500)])
@pytest.mark.parametrize("level", [0.0, 40.0, -100.0])
@pytest.mark.parametrize("low", [64, 100, 460])
@pytest.mark.parametrize("score", [dict(), dict(window=2400), dict(slopes=np.array([0, 0.001, 0.002, 0.003], np.float32))])
@pytest.mark.parametrize("own", [False, True])  # (the chunk's own tokens too lie at the level, or at 0)
def test_first_keys_of_the_lowest_value(kp, chunk, T, level, low, score, own):
    """Keys whose products overflow to minus infinity weigh nothing, wherever the
    row's other scores lie: as if they were not seen."""
    import torch

    b = standing_out(chunk, T, {t: level for t in range(T - chunk)})
    page, slot = paged.token_slots(b.table[0], 0, low, b.P)
    b.K[0, page, 0, slot, :16] = bf16(np.float32(-3e38))
    if own:
        page, slot = paged.token_slots(b.table[0], T - chunk, chunk, b.P)
        b.K[0, page, 0, slot, :16] = level / 2
    K, V, layer, Q, table, kv_len, q_start = b.dev()
    dev = {k: torch.from_numpy(v).cuda() if isinstance(v, np.ndarray) else v for k, v in score.items()}
    out, lse = kp.pages_attend(K, V, layer, Q, table, kv_len, q_start, return_lse=True, **dev)
    first = np.full(b.tokens, low, np.int32)
    first[b.q_start[1]:] = 0
    check_attend(out.float().cpu().numpy(), lse.cpu().numpy(), b.ref(first=first, **score), T)
