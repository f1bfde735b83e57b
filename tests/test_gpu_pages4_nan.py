"""A value that is NaN and seen makes a row NaN however small its weight, in
whole units of keys and in those that end inside, by both attention kernels."""

import numpy as np
import pytest

from oracle import paged, paged4

from paged4_util import Batch4
from test_gpu_pages4 import kp  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("max_kv", [0, 1 << 18])
@pytest.mark.parametrize("q,T,at", [(1, 40, 35), (1, 64, 35), (1, 300, 5), (3, 40, 33), (50, 90, 20), (50, 300, 140)])
@pytest.mark.parametrize("score", [dict(), dict(window=250)])
def test_nan_values_of_no_weight(kp, q, T, at, max_kv, score):
    b = Batch4(1, 1, 128, 16, [q], [T], seed=91)
    b.table = np.pad(b.table, ((0, 0), (0, (1 << 14) - b.table.shape[1])), constant_values=-9)
    b.Q[:] = b.Q[0]
    u, t = paged4.encode(-60 * b.Q[0, 0])  # a score of about -600 in every row
    page, slot = paged.token_slots(b.table[0], at, 1, b.P)
    b.codes[0][0, page, :, slot], b.scale[0][0, page, :, slot] = u, t
    b.scale[1][0, page, :, slot] = np.nan
    out, lse = kp.pages4_attend(*b.dev4(kp), max_kv=max_kv, return_lse=True, **score)
    behind = np.arange(T - q, T) - at
    sees = (behind >= 0) & (behind < score.get("window", T))
    out = out.float().cpu().numpy()
    assert np.isnan(out[sees]).all() and np.isfinite(out[~sees]).all()
