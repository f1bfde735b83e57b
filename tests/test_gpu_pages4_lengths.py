"""4-bit caches whose lengths lie: more new tokens than held ones, none held,
more held than the table has room for (nothing beyond it is written, read or
seen, and it is recorded); by the kernels for few rows and for many."""

import numpy as np
import pytest

from oracle import paged4

from paged4_util import Batch4, bf16, check4, new_rows, place, rotation
from test_gpu_pages4 import kp  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu


def attend(kp, b, **more):
    import torch

    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = kp.pages4_attend(*b.dev4(kp), return_lse=True, status=status, **more)
    return out.float().cpu().numpy(), lse.cpu().numpy(), int(status)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("room", [0, 1 << 16])  # (few rows; many: a table with room, or many rows)
@pytest.mark.parametrize("q,kv", [([5, 1], [3, 0]), ([300, 2, 70], [299, 1, 0]), ([300, 40], [10, 400]), ([1, 1], [0, 30])])
def test_positions_before_zero_see_nothing(kp, d, room, q, kv):
    b = Batch4(2, 8, d, 16, q, kv, seed=61)
    b.table = np.pad(b.table, ((0, 0), (0, max(0, room // 16 - b.table.shape[1]))), constant_values=-9)
    out, lse, status = attend(kp, b)
    assert status == 0
    check4(out, lse, b.ref4())
    if sum(q) * 4 > 256:
        import torch

        out, lse, status = attend(kp, b, workspace=torch.empty(0, dtype=torch.uint8, device="cuda"))
        assert status == 0
        check4(out, lse, b.ref4())


@pytest.mark.parametrize("hq,room,q,far", [(4, 256, 3, 0), (4, 256, 3, 7), (4, 1024, 90, 0), (64, 2048, 30, 100), (64, 4096, 90, 1 << 30),
                                           (4, 64, 1, (1 << 31) - 70)])
def test_more_than_the_table_has_room_for(kp, hq, room, q, far):
    """Every row lies at the room's end or behind it and sees all that fits."""
    b = Batch4(1, hq, 64, 16, [3, q], [40, room], seed=62)
    b.table = np.ascontiguousarray(b.table[:, : room // 16])
    ref = b.ref4(prefix=np.array([0, room], np.int32))
    b.kv_len[1] = room + q - 1 + far
    out, lse, status = attend(kp, b)
    assert status == (1 if b.kv_len[1] > room else 0)
    check4(out, lse, ref)


@pytest.mark.parametrize("kv,q", [(65, 1), (70, 10), (100, 64), ((1 << 31) - 1, 5), (3, 5)])
@pytest.mark.parametrize("d", [64, 128])
def test_append_and_read(kp, d, kv, q):
    import torch

    b = Batch4(2, 2, d, 16, [1, q], [20, 64], seed=28)
    b.table = np.ascontiguousarray(b.table[:, :4])  # room for 64 tokens
    b.kv_len[1] = kv
    pages, layer, _, table, kv_len, q_start = b.dev4(kp)
    rows = new_rows(b, 2, 2)
    dev = torch.from_numpy(rows).cuda().to(torch.bfloat16)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kp.pages4_append(pages, 0, dev, dev, table, kv_len, q_start, status=status)
    assert int(status) == (1 if kv > 64 else 0)
    u, t = paged4.encode(rows)
    held = [(0, 19)] + [(1, kv - q + i) for i in range(q)]
    for i, (s, p) in enumerate(held):
        if 0 <= p < 64:
            page, slot = b.table[s, p // 16], p % 16
            b.codes[0][0, page, :, slot], b.scale[0][0, page, :, slot] = u[i], t[i]
    assert np.array_equal(pages.K.cpu().numpy(), paged4.pack(b.codes[0]))
    assert np.array_equal(pages.K_scale.cpu().numpy(), b.scale[0], equal_nan=True)
    out = [torch.full((q + 1, 2, d), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    kp.pages4_read(pages, 0, table, kv_len, q_start, q + 1, *out, status=status)
    H = paged4.hadamard(d)
    for i, (s, p) in enumerate(held):
        got = out[0][i].float().cpu().numpy()
        if p < 0:
            assert (got == 7).all()
        elif p >= 64:
            assert (got == 0).all()
        else:
            assert np.array_equal(got, bf16(((u[i] - 7.5) @ H).astype(np.float32) * t[i][:, None]))
