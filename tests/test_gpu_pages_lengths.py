"""Sequences longer than their row of the table has room for: what does not fit
is neither written nor seen, and is recorded; positions are the real ones."""

import ctypes

import numpy as np
import pytest

from oracle import paged

from paged_util import Batch, bf16, check_attend, reads
from test_gpu_pages import kp  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu


def status_of(kp, K, V, word):
    pg = kp._pages(K, V, word)
    return kp.lib().kvpool_pages_status(ctypes.byref(pg), None)


@pytest.mark.parametrize("kv,q", [(65, 1), (70, 10), (100, 10), (100, 64), (1 << 30, 3), ((1 << 31) - 1, 5)])
def test_append(kp, kv, q):
    import torch

    b = Batch(2, 2, 64, 16, [1, q], [20, 64], seed=28)
    b.table = np.ascontiguousarray(b.table[:, :4])  # room for 64 tokens
    b.kv_len[1] = kv
    K, V, layer, _, table, kv_len, q_start = b.dev()
    r = np.random.default_rng(2)
    new = [bf16(r.standard_normal((q + 1, 2, 64), dtype=np.float32)) for _ in range(2)]
    dev = [torch.from_numpy(x).cuda().to(torch.bfloat16) for x in new]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kp.pages_append(K, V, 0, *dev, table, kv_len, q_start, status=status)
    assert status_of(kp, K, V, status) == -1
    for X, x in ((b.K, new[0]), (b.V, new[1])):
        X[0, b.table[0, 1], :, 19 - 16] = x[0]
        for i in range(q):
            p = kv - q + i
            if p < 64:
                X[0, b.table[1, p // 16], :, p % 16] = x[1 + i]
    assert np.array_equal(K.float().cpu().numpy(), b.K, equal_nan=True)
    assert np.array_equal(V.float().cpu().numpy(), b.V, equal_nan=True)


def plain(b, room, window=0, slopes=None):
    """What paged.attend returns, of a batch with one KV head whose table has
    room for `room` tokens of a sequence: rows at their positions, keys from
    the room on seen by none."""
    parts = []
    for s in range(len(b.q)):
        kv, T = int(b.kv_len[s]), min(int(b.kv_len[s]), room)
        page, slot = paged.token_slots(b.table[s], 0, T, b.P)
        k, v = (X[0, page, 0, slot].astype(np.float64) for X in (b.K, b.V))
        for i in range(b.q[s]):
            p = kv - b.q[s] + i
            lo, hi = max(0, p - window + 1) if window else 0, min(p + 1, T)
            q = b.Q[b.q_start[s] + i].astype(np.float64)
            x = q @ k[lo:hi].T / 8
            err = (64 + 2) * 2.0 ** -24 / 8 * (np.abs(q) @ np.abs(k[lo:hi]).T) + 2.0 ** -23 * np.abs(x)
            if slopes is not None:
                far = slopes[:, None].astype(np.float64) * (p - np.arange(lo, hi))
                x, err = x - far, err + 2.0 ** -22 * far
            if lo >= hi:
                parts.append((np.zeros((b.hq, 64)), np.full(b.hq, -np.inf), np.zeros((b.hq, 64)), np.zeros(b.hq)))
                continue
            w = np.exp(x - x.max(1, keepdims=True))
            total = w.sum(1, keepdims=True)
            parts.append((w @ v[lo:hi] / total, x.max(1) + np.log(total[:, 0]), w @ np.abs(v[lo:hi]) / total,
                          err.max(1) + 2.0 ** -23 * np.abs(x).max(1)))
    return [np.stack(x) for x in zip(*parts)]


@pytest.mark.parametrize("hq,room,kv,q", [(4, 1024, 1025, 1), (4, 1024, 1040, 20), (4, 1024, 1100, 20), (4, 1024, 1400, 100),
                                          (64, 4096, 4100, 20), (64, 4096, 4200, 60), (64, 4096, 9000, 60)])
@pytest.mark.parametrize("score", [dict(), dict(window=60), dict(slopes=True)])
def test_attend(kp, hq, room, kv, q, score):
    """By the kernel for few rows (4 heads) and that for many (64)."""
    import torch

    b = Batch(1, hq, 64, 16, [3, q], [40, room], seed=29)
    b.table = np.ascontiguousarray(b.table[:, :room // 16])
    b.kv_len[1] = kv
    assert (reads(b, b.tokens, room) >= 1 << 27) == (hq == 64)
    slopes = np.linspace(0.0, 0.02, hq).astype(np.float32) if score.get("slopes") else None
    K, V, layer, Q, table, kv_len, q_start = b.dev()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = kp.pages_attend(K, V, layer, Q, table, kv_len, q_start, return_lse=True, status=status,
                               window=score.get("window", 0), slopes=None if slopes is None else torch.from_numpy(slopes).cuda())
    assert status_of(kp, K, V, status) == -1
    check_attend(out.float().cpu().numpy(), lse.cpu().numpy(), plain(b, room, score.get("window", 0), slopes), room)


def test_a_length_that_fits_is_not_recorded(kp):
    import torch

    b = Batch(1, 4, 64, 16, [3, 20], [64, 64], seed=30)
    b.table = np.ascontiguousarray(b.table[:, :4])
    K, V, layer, Q, table, kv_len, q_start = b.dev()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = kp.pages_attend(K, V, layer, Q, table, kv_len, q_start, return_lse=True, status=status)
    kp.pages_append(K, V, 0, Q[:, :1], Q[:, 1:2], table, kv_len, q_start, status=status)
    assert status_of(kp, K, V, status) == 0
    check_attend(out.float().cpu().numpy(), lse.cpu().numpy(), b.ref(), 64)
