"""PagedCache.grow when it cannot grow, on a machine without a GPU (the page
copies and the batch's upload are recorded, not made): no sequence has grown,
and every page that a sequence got of its own meanwhile is copied."""

import pytest


class Recorded:
    """A PagedCache of `pages` pages without device memory, and the page copies that it asked for."""

    def __init__(self, kp, monkeypatch, pages=8):
        self.cache = kp.PagedCache.__new__(kp.PagedCache)
        self.cache.pager, self.cache.page_tokens = kp.Pager(pages, 16), 16
        self.cache.K = self.cache.V = self.cache.status_word = None
        self.copied, self.upload = [], None

        def copy(K, V, src, dst, stream=None):
            self.copied += list(zip(src, dst))

        def batch(cache, seqs, counts, stream=None):
            if self.upload is not None:
                raise self.upload

        monkeypatch.setattr(kp, "pages_copy", copy)
        monkeypatch.setattr(kp, "PagedBatch", batch)
        monkeypatch.setattr(kp, "_here", lambda: 0)
        monkeypatch.setattr(kp, "_pages", lambda *a, **k: None)
        monkeypatch.setattr(kp, "_raw_stream", lambda *a, **k: None)


@pytest.fixture
def kp():
    from shared_quantized_kv_gb300 import build, kvpool

    build.build()
    kvpool.lib()
    return kvpool


def forked(kp, monkeypatch):
    """Agents a and b that share a partly filled page, and what each holds."""
    r = Recorded(kp, monkeypatch)
    a = r.cache.new()
    r.cache.grow([a], [20])
    b = r.cache.fork(a)
    return r, a, b


def check_nobody_has_grown(r, a, b):
    pager = r.cache.pager
    assert pager.length(a) == pager.length(b) == 20
    ta, tb = pager.table(a), pager.table(b)
    assert ta[0] == tb[0] == 0 and len(ta) == len(tb) == 2
    # b still has the page that both had; a too, or a copy of it
    assert tb[1] == 1 and (ta[1] == 1 or (1, ta[1]) in r.copied)
    used = {p for t in (ta, tb) for p in t}
    assert pager.free_pages() == 8 - len(used)


@pytest.mark.parametrize("count,error", [(1 << 31, ValueError), (1 << 32, ValueError), (-(1 << 40), ValueError), (1.5, TypeError),
                                         ("1", TypeError), (None, TypeError)])
def test_counts_that_are_no_int32(kp, monkeypatch, count, error):
    r, a, b = forked(kp, monkeypatch)
    for counts in ([1, count], [count, 1]):
        with pytest.raises(error):
            r.cache.grow([a, b], counts)
        check_nobody_has_grown(r, a, b)
    r.cache.close()


def test_counts_that_the_pager_refuses(kp, monkeypatch):
    r, a, b = forked(kp, monkeypatch)
    for count in (-1, (1 << 31) - 1, 1000):
        with pytest.raises(kp.KVPoolError):
            r.cache.grow([a, b], [1, count])
        check_nobody_has_grown(r, a, b)
    r.cache.close()


def test_a_batch_that_cannot_be_uploaded(kp, monkeypatch):
    for error in (RuntimeError("out of memory"), KeyboardInterrupt()):
        r, a, b = forked(kp, monkeypatch)
        r.upload = error
        with pytest.raises(type(error)):
            r.cache.grow([a, b], [1, 20])
        check_nobody_has_grown(r, a, b)
        r.upload = None
        r.cache.grow([a, b], [1, 20])
        assert r.cache.pager.length(a) == 21 and r.cache.pager.length(b) == 40
        r.cache.close()


@pytest.mark.parametrize("what", ["_here", "_pages", "_raw_stream"])
def test_another_device(kp, monkeypatch, what):
    r, a, b = forked(kp, monkeypatch)

    def refuse(*args, **kwargs):
        raise ValueError("another device")

    monkeypatch.setattr(kp, what, refuse)
    with pytest.raises(ValueError):
        r.cache.grow([a, b], [1, 20])
    check_nobody_has_grown(r, a, b)
    assert not r.copied
    r.cache.close()
