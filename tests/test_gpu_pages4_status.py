"""Attention of many rows over 4-bit caches with a workspace and without one: the
same results and the same status word, whatever the tables hold where no row looks."""

import numpy as np
import pytest

from paged4_util import Batch4, check4
from test_gpu_pages4 import kp  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu


def both(kp, b, **score):
    """(out, lse, status) with a workspace of the call's own choice, with room for one tile, with none."""
    import torch

    dev = b.dev4(kp)
    more = {k: torch.from_numpy(v).cuda() if isinstance(v, np.ndarray) else v for k, v in score.items()}
    assert kp.pages4_attend_ws_bytes(dev[0], *dev[3:], b.tokens, b.hq) > 0
    for ws in (None, torch.empty(1 << 20, dtype=torch.uint8, device="cuda"), torch.empty(0, dtype=torch.uint8, device="cuda")):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, lse = kp.pages4_attend(*dev, return_lse=True, status=status, workspace=ws, **more)
        yield out.float().cpu().numpy(), lse.cpu().numpy(), int(status)


def batch(q, kv, d=64, hk=2, hq=4, P=32):
    b = Batch4(hk, hq, d, P, q, kv, seed=81)
    b.table = np.pad(b.table, ((0, 0), (0, (1 << 16) // P - b.table.shape[1])), constant_values=-9)
    return b


CASES = {
    # windows of 200 end behind tile 17: entries of the tiles before it
    "window": (dict(window=200), lambda b: b.table[0, : 17 * 4]),
    # between a prefix of 300 tokens (tiles 0 to 2) and the windows
    "prefix": (dict(window=200, prefix=np.array([300, 0], np.int32)), lambda b: b.table[0, 3 * 4: 17 * 4]),
    # documents that begin with the chunk
    "documents": (dict(first=np.full(301, 2700, np.int32)), lambda b: b.table[0, : 21 * 4]),
    # a block of rows that see nothing between blocks that do
    "hole": (dict(window=100, first=np.where(np.arange(301) // 128 == 1, 5000, 0).astype(np.int32)),
             lambda b: b.table[0, : 20 * 4]),
}


@pytest.mark.parametrize("bad", [-1, 1 << 30])
@pytest.mark.parametrize("name", sorted(CASES))
def test_entries_that_no_row_sees(kp, name, bad):
    b = batch([300, 1], [3000, 40])
    score, where = CASES[name]
    ref = b.ref4(**score)
    where(b)[:] = bad
    for out, lse, status in both(kp, b, **score):
        assert status == 0
        check4(out, lse, ref)


@pytest.mark.parametrize("d,P", [(64, 16), (128, 128), (128, 32)])
@pytest.mark.parametrize("where", ["first", "middle", "last"])
def test_entries_that_rows_see(kp, d, P, where):
    """One of them is recorded, in a tile's first page or its last, and reads as zeros."""
    b = batch([300, 1], [3000, 40], d=d, P=P)
    at = {"first": 0, "middle": 1100 // P, "last": 2999 // P}[where]
    for x in b.scale:
        x[0, b.table[0, at]] = 0
    ref = b.ref4()
    b.table[0, at] = -1
    for out, lse, status in both(kp, b):
        assert status == 1
        check4(out, lse, ref)
