"""Which calls of 4-bit attention have use for a workspace (host only)."""

import ctypes

import pytest

A = 1 << 20  # an aligned address, never used


@pytest.fixture(scope="module")
def kp():
    from shared_quantized_kv_gb300 import build, kvpool

    build.build()
    return kvpool


@pytest.mark.parametrize("seqs,used", [(1, True), (65535, True), (65536, False), (1 << 20, False)])
def test_more_sequences_than_a_grid_has_room_for(kp, seqs, used):
    """Their tiles are made without one, so none is asked for."""
    pg = kp.Pages4Arg(A, A, A, A, 1, 1000, 2, 64, 64, None)
    sq = kp.Seqs(seqs, 1000, A, A, A, max(seqs, 300), 300, 64000)
    n = kp.lib().kvpool_pages4_attend_ws_bytes(ctypes.byref(pg), ctypes.byref(sq), 4)
    assert n == (seqs * 2 * 500 * (2 * 128 * 64 * 2 + 1024) if used else 0)
