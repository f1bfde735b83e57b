"""What the calls of the rotation and of the 4-bit caches refuse before they
touch a device (every call here is refused: the addresses are never used)."""

import ctypes

import pytest

INVALID = -1
A = 1 << 20  # an aligned address
FAR = (1 << 32, (1 << 32) + 1, -(1 << 32), 1 << 31)


@pytest.fixture(scope="module")
def kp():
    from shared_quantized_kv_gb300 import build, kvpool

    build.build()
    kvpool.lib()
    return kvpool


def pages4(kp, **other):
    a = dict(K=A, V=A, K_scale=A, V_scale=A, layers=2, pages=10, kv_heads=2, page_tokens=16, head_dim=64, status=None)
    return kp.Pages4Arg(**(a | other))


def pages(kp):
    return kp.Pages(A, A, 2, 10, 2, 16, 64, None)


def seqs(kp, **other):
    a = dict(seqs=1, table_stride=4, page_table=A, kv_len=A, q_start=A, tokens=3, max_q=0, max_kv=0)
    return kp.Seqs(**(a | other))


def rotary(kp, **other):
    return kp.RotaryArg(**(dict(cos=A, sin=A, positions=100, dim=64, interleaved=0, offset=0, at=None) | other))


ref = ctypes.byref

BAD_PAGES = [dict(K=None), dict(V=None), dict(K=A + 8), dict(K_scale=None), dict(V_scale=None), dict(K_scale=A + 4),
             dict(V_scale=A + 8), dict(layers=0), dict(pages=0), dict(kv_heads=0), dict(page_tokens=8),
             dict(page_tokens=48), dict(head_dim=32), dict(head_dim=96), dict(head_dim=256), dict(status=A + 1),
             dict(pages=1 << 30)]
BAD_SEQS = [dict(seqs=0), dict(table_stride=0), dict(tokens=0), dict(page_table=None), dict(kv_len=None),
            dict(q_start=None), dict(q_start=A + 2), dict(max_q=-1)]
BAD_ROTARY = [dict(cos=None), dict(sin=None), dict(cos=A + 4), dict(sin=A + 8), dict(positions=0), dict(dim=0),
              dict(dim=8), dict(dim=24), dict(dim=80), dict(dim=128), dict(at=A + 2)]
# K, k_stride, V, v_stride, Q, q_stride, q_heads, Q_out, q_out_stride
GOOD = dict(K=A, ks=128, V=A, vs=128, Q=A, qs=256, hq=4, out=A, os=256)
BAD_ROWS = [dict(K=None), dict(V=None), dict(K=A + 8), dict(V=A + 2), dict(ks=127), dict(ks=120), dict(vs=132), dict(Q=A + 8),
            dict(qs=255), dict(qs=248), dict(hq=0), dict(hq=5), dict(out=None), dict(out=A + 8), dict(os=248),
            dict(os=260), dict(Q=None)]


def append(kp, four, pg, sq, turn, rows, layer=0):
    call = kp.lib().kvpool_pages4_append if four else kp.lib().kvpool_pages_append_rotary
    return call(ref(pg), layer, ref(sq), turn, rows["K"], rows["ks"], rows["V"], rows["vs"], rows["Q"], rows["qs"],
                rows["hq"], rows["out"], rows["os"], None)


@pytest.mark.parametrize("four", [False, True])
def test_appends_refuse(kp, four):
    pg = pages4(kp) if four else pages(kp)
    for bad in BAD_ROTARY:
        assert append(kp, four, pg, seqs(kp), ref(rotary(kp, **bad)), GOOD) == INVALID, bad
    for bad in BAD_SEQS:
        assert append(kp, four, pg, seqs(kp, **bad), ref(rotary(kp)), GOOD) == INVALID, bad
    for bad in BAD_ROWS:
        assert append(kp, four, pg, seqs(kp), ref(rotary(kp)), GOOD | bad) == INVALID, bad
    for layer in (-1, 2):
        assert append(kp, four, pg, seqs(kp), ref(rotary(kp)), GOOD, layer) == INVALID
    # Q without a rotation; the bf16 append without one is kvpool_pages_append
    assert append(kp, four, pg, seqs(kp), None, GOOD) == INVALID
    if not four:
        assert append(kp, four, pg, seqs(kp), None, GOOD | dict(Q=None, out=None, hq=0)) == INVALID
    # what is well formed is refused for want of a device alone
    assert append(kp, four, pg, seqs(kp), ref(rotary(kp)), GOOD) not in (0, INVALID)


def test_pages4_calls_refuse(kp):
    lib = kp.lib()
    one = (ctypes.c_int32 * 1)(1)
    two = (ctypes.c_int32 * 1)(2)

    def calls(pg, sq):
        yield append(kp, True, pg, sq, ref(rotary(kp)), GOOD)
        yield lib.kvpool_pages4_read(ref(pg), 0, ref(sq), A, A, None)
        yield lib.kvpool_pages4_attend(ref(pg), 0, ref(sq), A, 256, 4, None, A, None, 0.0, None, 0, None)

    for bad in BAD_PAGES:
        for rc in calls(pages4(kp, **bad), seqs(kp)):
            assert rc == INVALID, bad
        assert lib.kvpool_pages4_copy(ref(pages4(kp, **bad)), one, two, 1, None) == INVALID
    for bad in BAD_SEQS:
        for rc in calls(pages4(kp), seqs(kp, **bad)):
            assert rc == INVALID, bad
    pg, sq = pages4(kp), seqs(kp)
    for rc in calls(pg, sq):
        assert rc not in (0, INVALID)
    for K, V in ((None, A), (A, None), (A + 8, A), (A, A + 2)):
        assert lib.kvpool_pages4_read(ref(pg), 0, ref(sq), K, V, None) == INVALID
    for Q, qs, hq, out, lse, scale in ((None, 256, 4, A, None, 0.0), (A + 8, 256, 4, A, None, 0.0), (A, 250, 4, A, None, 0.0),
                                       (A, 248, 4, A, None, 0.0), (A, 256, 3, A, None, 0.0), (A, 256, 1, A, None, 0.0),
                                       (A, 256, 4, None, None, 0.0), (A, 256, 4, A + 8, None, 0.0),
                                       (A, 256, 4, A, A + 2, 0.0), (A, 256, 4, A, None, -1.0),
                                       (A, 256, 4, A, None, float("inf")), (A, 256, 4, A, None, float("nan"))):
        assert lib.kvpool_pages4_attend(ref(pg), 0, ref(sq), Q, qs, hq, None, out, lse, scale, None, 0, None) == INVALID
    assert lib.kvpool_pages4_attend(ref(pg), 0, ref(sq), A, 256, 4, None, A, None, 0.0, A + 8, 100, None) == INVALID
    # a workspace where there is use for one: many rows over many keys
    big = seqs(kp, seqs=3, table_stride=1000, tokens=900)
    need = lib.kvpool_pages4_attend_ws_bytes(ref(pg), ref(big), 4)
    assert need == 3 * 2 * 125 * (2 * 128 * 64 * 2 + 1024)
    assert lib.kvpool_pages4_attend_ws_bytes(ref(pg), ref(seqs(kp, seqs=3, table_stride=1000, tokens=900, max_q=128)), 4) == 0
    assert lib.kvpool_pages4_attend_ws_bytes(ref(pg), ref(sq), 4) == 0
    assert lib.kvpool_pages4_attend_ws_bytes(ref(pg), ref(big), 3) == 0
    assert lib.kvpool_pages4_attend_ws_bytes(None, ref(big), 4) == 0
    assert lib.kvpool_pages4_attend(None, 0, ref(sq), A, 256, 4, None, A, None, 0.0, None, 0, None) == INVALID
    assert lib.kvpool_pages4_status(ref(pg), None) == INVALID and lib.kvpool_pages4_status(None, None) == INVALID
    for src, dst, n in ((one, one, 1), (one, two, -1), (one, two, 11), (None, two, 1)):
        assert lib.kvpool_pages4_copy(ref(pg), src, dst, n, None) == INVALID
    assert lib.kvpool_pages4_copy(ref(pg), None, None, 0, None) == 0


@pytest.mark.parametrize("far", FAR)
def test_python_refuses_numbers_past_32_bits(kp, far):
    """The layer is looked at first: nothing else is reached."""
    with pytest.raises(ValueError, match="layer"):
        kp.pages_append_rotary(None, None, far, None, None, None, None, None, kp.Rotary(None, None))
    with pytest.raises(ValueError, match="layer"):
        kp.pages4_append(None, far, None, None, None, None, None)
    with pytest.raises(ValueError, match="layer"):
        kp.pages4_read(None, far, None, None, None, 1)
    with pytest.raises(ValueError, match="tokens"):
        kp.pages4_read(None, 0, None, None, None, far)
    with pytest.raises(ValueError, match="layer"):
        kp.pages4_attend(None, far, None, None, None, None)
    with pytest.raises(ValueError, match="page"):
        kp.pages4_copy(None, [far], [0])


def test_python_refuses(kp):
    with pytest.raises(ValueError, match="rotary"):
        kp.pages_append_rotary(None, None, 0, None, None, None, None, None, None)
    with pytest.raises(ValueError, match="length"):
        kp.pages4_copy(None, [1, 2], [0])
    with pytest.raises(ValueError, match="bits"):
        kp.PagedCache(1, 2, 64, 4, 16, bits=8)
    for args in ((0, 64), (5, 0), (5, 63)):
        with pytest.raises(ValueError):
            kp.rotary_tables(*args, device="cpu")


def test_far_positions_of_the_tables():
    """Angles in 64 bits: a far position's cosine keeps float32's precision."""
    import math

    from shared_quantized_kv_gb300 import kvpool

    cos, sin = kvpool.rotary_tables(200001, 64, 10000.0, device="cpu")
    for p, i in ((200000, 0), (199999, 1), (131071, 31), (0, 5)):
        a = p * 10000.0 ** (-2 * i / 64)
        assert abs(float(cos[p, i]) - math.cos(a)) < 2.0 ** -24 + 1e-10
        assert abs(float(sin[p, i]) - math.sin(a)) < 2.0 ** -24 + 1e-10


def test_every_declared_call_is_bound(kp):
    import os
    import re

    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "kvpool.h")
    with open(path) as f:
        names = set(re.findall(r"\b(kvpool_[a-z0-9_]+)\s*\(", f.read()))
    assert {"kvpool_pages4_attend", "kvpool_pages_append_rotary"} <= names <= set(kp._SIGS)
