"""Attention of few rows over 4-bit caches of many keys: the log of the sum as
precise for rows whose weights lie on few keys (a window, a document that begins
late, keys that stand out, large queries) as for flat ones, at every length."""

import numpy as np
import pytest

from oracle import paged, paged4

from paged4_util import Batch4
from paged_util import bf16
from test_gpu_pages4 import kp, run  # noqa: F401 (kp: a fixture)

pytestmark = pytest.mark.gpu

ROOM = 1 << 20  # with a max_kv of that, blocks of 16 rows where there are more than 8


def batch(hk, hq, d, q, T, seed):
    b = Batch4(hk, hq, d, 128, [q], [T], seed=seed)
    b.table = np.pad(b.table, ((0, 0), (0, ROOM // 128 - b.table.shape[1])), constant_values=-9)
    return b


@pytest.mark.parametrize("T", [16383, 16384, 20011])
@pytest.mark.parametrize("hk,hq,d,q,max_kv", [(1, 4, 128, 1, 0), (1, 8, 64, 2, 0), (1, 16, 128, 1, ROOM), (1, 10, 64, 1, ROOM),
                                              (1, 6, 128, 5, 256)])
@pytest.mark.parametrize("form", ["flat", "large", "peak", "window", "window1", "document", "cap"])
def test_scores_keep_their_bits(kp, form, hk, hq, d, q, max_kv, T):
    b = batch(hk, hq, d, q, T, seed=T % 7)
    score = {}
    if form == "large":
        b.Q = bf16(b.Q * 8)
    elif form == "peak":
        # one key with a part of every query in it stands out
        r = np.random.default_rng(3)
        b.Q = bf16(b.Q[:1, :1] + 0.3 * b.Q)
        u, t = paged4.encode((1.5 * b.Q[0, 0] + 4 * r.standard_normal(d)).astype(np.float32))
        page, slot = paged.token_slots(b.table[0], T // 3, 1, b.P)
        b.codes[0][0, page, :, slot], b.scale[0][0, page, :, slot] = u, t
    elif form == "window":
        score["window"] = 16
    elif form == "window1":
        score["window"] = 1
    elif form == "document":
        score["first"] = np.full(b.tokens, T - 20, np.int32)
    elif form == "cap":
        score["cap"] = 30.0
    run(kp, b, max_q=q, max_kv=max_kv, **score)
