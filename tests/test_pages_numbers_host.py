"""Numbers past 32 bits are refused by every Python call of the paged caches
that takes one, not cut to their low bits; on a machine without a GPU."""

import pytest

FAR = (1 << 32, (1 << 32) + 1, -(1 << 32), 1 << 31, -(1 << 31) - 1)


@pytest.fixture(scope="module")
def kp():
    from shared_quantized_kv_gb300 import build, kvpool

    build.build()
    kvpool.lib()
    return kvpool


@pytest.mark.parametrize("far", FAR)
def test_pager(kp, far):
    p = kp.Pager(4, 16)
    for _ in range(2):
        p.extend(p.new(), 20)
    for f in (lambda: p.extend(far, 1), lambda: p.truncate(far, 0), lambda: p.fork(far), lambda: p.free(far),
              lambda: p.length(far), lambda: p.table(far), lambda: p.owners(far)):
        with pytest.raises(ValueError):
            f()
    assert [p.length(s) for s in (0, 1)] == [20, 20] and p.free_pages() == 0
    p.close()
    for args in ((far + 4, 16), (4, far + 16)):
        # (-2^31 - 1 + 4 fits 32 bits: the pager itself refuses that many pages)
        with pytest.raises((ValueError, kp.KVPoolError)):
            kp.Pager(*args)


@pytest.mark.parametrize("far", FAR)
def test_layers(kp, monkeypatch, far):
    """The layer is looked at first: nothing else is reached."""
    with pytest.raises(ValueError, match="layer"):
        kp.pages_append(None, None, far, None, None, None, None, None)
    with pytest.raises(ValueError, match="layer"):
        kp.pages_attend(None, None, far, None, None, None, None)
    pool = kp.KVPool.__new__(kp.KVPool)
    pool._h = None
    with pytest.raises(ValueError, match="layer"):
        pool.attend_pages(far, None, None, None)
    with pytest.raises(ValueError, match="page_layer"):
        pool.attend_pages(0, None, None, None, page_layer=far)
    with pytest.raises(ValueError, match="tokens"):
        pool.attend_pages_ws_bytes(far, 4)
    with pytest.raises(ValueError, match="q_heads"):
        pool.attend_pages_ws_bytes(4, far)
