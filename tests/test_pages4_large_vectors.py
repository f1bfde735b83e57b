"""Vectors near the types' largest value in 4 bits: codes and a finite scale as for
any other, by the restatement and by the kernels."""

import numpy as np
import pytest

from oracle import paged, paged4

from paged4_util import Batch4, check4, new_rows
from paged_util import bf16
from test_gpu_pages4 import kp  # noqa: F401 (a fixture)

LARGE, TOP = (float(x) for x in bf16(np.array([1.2e38, 3.38e38])))


def rows(shape, size, seed=0):
    """Channels between half of `size` and `size`, of either sign."""
    r = np.random.default_rng(seed)
    return bf16((r.uniform(0.5, 1.0, shape) * np.where(r.random(shape) < 0.5, -1, 1) * size).astype(np.float32))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("size", [LARGE, TOP])
def test_restatement(d, size):
    """A power of two less of everything: the same codes, the scale that much smaller."""
    x = rows((50, d), size)
    x[0] = size  # one coordinate of the transform
    u, t = paged4.encode(x)
    u2, t2 = paged4.encode(x * np.float32(2.0 ** -100))
    assert (u == u2).all() and (t == t2 * np.float32(2.0) ** 100).all() and np.isfinite(t).all()
    err = ((paged4.values(u[1:], t[1:]) / size - x[1:] / size) ** 2).sum() / ((x[1:] / size).astype(np.float64) ** 2).sum()
    assert err < 0.3352 ** 2 / 4


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("size", [LARGE, TOP])
def test_append_and_read(kp, d, size):
    import torch

    b = Batch4(2, 2, d, 16, [20, 1], [20, 30], seed=3)
    pages, layer, _, table, kv_len, q_start = b.dev4(kp)
    new = rows((b.tokens, 2, d), size)
    new[0, 0] = size
    dev = torch.from_numpy(new).cuda().to(torch.bfloat16)
    kp.pages4_append(pages, 0, dev, dev, table, kv_len, q_start)
    u, t = paged4.encode(new)
    K, V = kp.pages4_read(pages, 0, table, kv_len, q_start, b.tokens)
    page, slot = paged.token_slots(b.table[0], 0, 20, b.P)
    assert np.array_equal(pages.K_scale.cpu().numpy()[0, page, :, slot], t[:20]) and np.isfinite(t).all()
    with np.errstate(over="ignore"):
        want = bf16(((u - 7.5) @ paged4.hadamard(d)).astype(np.float32) * t[..., None])
    for X in (K, V):
        assert np.array_equal(X.float().cpu().numpy(), want)
    if size < TOP:
        assert np.isfinite(want).all()


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("q,T,max_kv", [(1, 300, 0), (5, 300, 0), (90, 300, 1 << 18)])
def test_attention(kp, d, q, T, max_kv):
    """Large keys under small queries (whose scores are ordinary): appended, then attended."""
    import torch

    b = Batch4(1, 4, d, 16, [T], [T], seed=4)
    b.table = np.pad(b.table, ((0, 0), (0, (1 << 14) - b.table.shape[1])), constant_values=-9)
    pages, layer, Q, table, kv_len, q_start = b.dev4(kp)
    k, v = rows((T, 1, d), LARGE), new_rows(b, 5, 1)
    kp.pages4_append(pages, 0, *(torch.from_numpy(x).cuda().to(torch.bfloat16) for x in (k, v)), table, kv_len, q_start)
    page, slot = paged.token_slots(b.table[0], 0, T, b.P)
    for i, x in enumerate((k, v)):
        b.codes[i][0, page, :, slot], b.scale[i][0, page, :, slot] = paged4.encode(x)
    b.Q = bf16(b.Q[:q] * np.float32(2.0 ** -124))
    b.tokens, b.q, b.q_start = q, [q], np.array([0, q], np.int32)
    out, lse = kp.pages4_attend(pages, 0, torch.from_numpy(b.Q).cuda().to(torch.bfloat16), table, kv_len,
                                torch.from_numpy(b.q_start).cuda(), max_kv=max_kv, return_lse=True)
    check4(out.float().cpu().numpy(), lse.cpu().numpy(), b.ref4())
