"""Caps far above most scores, in a batch where one head reaches them: the other
heads' scores keep float32's relative precision."""

import numpy as np
import pytest

from paged_util import Batch, bf16, check_attend
from test_gpu_pages import kp  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("room", [0, 1 << 16])  # (the kernel for few rows, that for many)
@pytest.mark.parametrize("cap", [1e3, 1e4, 1e5, 1e7])
@pytest.mark.parametrize("slopes", [False, True])
def test_one_head_reaches_the_cap(kp, cap, slopes, room):
    import torch

    b = Batch(1, 4, 64, 32, [100, 20], [1300, 900], seed=34)
    b.Q[:, 3] = bf16(b.Q[:, 3] * np.float32(cap / 2))
    if room:
        b.many(room)
    K, V, layer, Q, table, kv_len, q_start = b.dev()
    sl = np.array([0.0, 0.01, 0.05, 0.002], np.float32)
    dev = dict(slopes=torch.from_numpy(sl).cuda()) if slopes else {}
    sc = dict(slopes=sl) if slopes else {}
    out, lse = kp.pages_attend(K, V, layer, Q, table, kv_len, q_start, cap=cap, return_lse=True, **dev)
    out, lse = out.float().cpu().numpy(), lse.cpu().numpy()
    # tanh(z) is z within z^3 / 3: below 2e-5 of a score of 8 for the smallest cap, so these take the
    # cap's own reference, in which only that head's error has to count the cap's
    ref, flat = b.ref(cap=cap, **sc), b.ref(**sc)
    assert np.abs(flat[1][:, :3] - ref[1][:, :3]).max() < 1e-3
    err = ref[3].copy()
    err[:, :3] = flat[3][:, :3] + 2.0 ** -22 * np.abs(flat[1][:, :3]).max()
    check_attend(out, lse, (ref[0], ref[1], ref[2], err), 1300)
