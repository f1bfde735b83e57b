"""PagedCache and its batches where the arguments do not fit, on a machine
without a GPU: refused before anything changes."""

import pytest

from test_pages_grow_host import Recorded, kp  # noqa: F401 (kp: a fixture)


@pytest.mark.parametrize("what", ["_here", "_pages", "_raw_stream"])
def test_compact_on_another_device(kp, monkeypatch, what):
    """The tables of a cache whose pages cannot be copied stay as they are."""
    r = Recorded(kp, monkeypatch)
    cache = r.cache
    a, b = cache.new(), cache.new()
    cache.grow([a, b], [40, 30])
    cache.free(a)
    before = cache.pager.table(b)

    def refuse(*args, **kwargs):
        raise ValueError("another device")

    with monkeypatch.context() as m:
        m.setattr(kp, what, refuse)
        m.setattr(kp, "pages_copy", refuse)
        with pytest.raises(ValueError):
            cache.compact()
    assert cache.pager.table(b) == before
    assert cache.compact() == 2 and cache.pager.table(b) == [1, 0]
    assert r.copied == [(4, 0), (3, 1)]
    cache.close()
