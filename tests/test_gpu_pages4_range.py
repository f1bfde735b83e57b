"""Attention over 4-bit caches at the far ends of the types' range: queries and
keys of very different sizes whose scores are ordinary."""

import numpy as np
import pytest

from paged4_util import Batch4
from paged_util import bf16
from test_gpu_pages4 import kp, run, scores  # noqa: F401 (kp: a fixture)

pytestmark = pytest.mark.gpu

FAR = [(122, -116), (118, -118), (60, -60), (-60, 60), (-118, 118), (-122, 122)]  # powers of two of queries and of keys
SCORES = [dict(), dict(window=150), dict(cap=9.0, slopes=True)]


def far(b, q, k):
    b.Q = bf16(b.Q * np.float32(2.0 ** q))
    b.scale[0] *= np.float32(2.0 ** k)
    return b


@pytest.mark.parametrize("q,k", FAR)
@pytest.mark.parametrize("score", SCORES)
@pytest.mark.parametrize("d,chunk", [(128, 1), (64, 3), (128, 5)])
def test_few_rows(kp, d, chunk, score, q, k):
    b = far(Batch4(2, 8, d, 16, [chunk, 1], [300, 40], seed=71), q, k)
    run(kp, b, max_q=chunk, **scores(b, **score))


@pytest.mark.parametrize("q,k", FAR)
@pytest.mark.parametrize("score", SCORES)
@pytest.mark.parametrize("d,n,T", [(128, 100, 100), (64, 100, 100), (128, 90, 1500), (64, 30, 400)])
def test_many_rows(kp, d, n, T, score, q, k):
    """Prompts, whose first rows see few keys, and chunks."""
    b = far(Batch4(1, 8, d, 16, [n, 1], [T, 60], seed=72), q, k)
    b.table = np.pad(b.table, ((0, 0), (0, 4096 - b.table.shape[1])), constant_values=-9)
    run(kp, b, **scores(b, **score))
