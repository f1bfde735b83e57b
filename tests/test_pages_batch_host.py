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


def test_fewer_rows_than_the_batch(kp, monkeypatch):
    """They would be taken for the last of their sequence: refused. More rows are padding."""
    import types

    import torch

    r = Recorded(kp, monkeypatch)
    calls = []
    monkeypatch.setattr(kp, "pages_append", lambda *a, **k: calls.append("append"))
    monkeypatch.setattr(kp, "pages_attend", lambda *a, **k: calls.append("attend"))
    batch = types.SimpleNamespace(tokens=3, table=None, kv_len=None, q_start=None, max_q=3, max_kv=20)
    pool = kp.KVPool.__new__(kp.KVPool)
    pool._h = None
    rows = lambda n: torch.zeros(n, 2, 64, dtype=torch.bfloat16)
    for f in (lambda: r.cache.append(0, rows(2), rows(2), batch), lambda: r.cache.attend(0, rows(2), batch),
              lambda: r.cache.attend(0, rows(0), batch), lambda: pool.attend_pages(0, rows(2), r.cache, batch)):
        with pytest.raises(ValueError, match="3 tokens"):
            f()
    assert not calls
    for n in (3, 5):
        r.cache.append(0, rows(n), rows(n), batch), r.cache.attend(0, rows(n), batch)
    assert calls == ["append", "attend"] * 2
    r.cache.close()
