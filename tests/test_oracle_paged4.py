"""The plain restatement of the 4-bit cache, pinned to mathematics."""

import numpy as np
import pytest

from oracle import paged4


@pytest.mark.parametrize("d", [64, 128])
def test_transform(d):
    H = paged4.hadamard(d)
    assert (H @ H == d * np.eye(d)).all() and (H == H.T).all()
    e = np.eye(d, dtype=np.float32)
    u, t = paged4.encode(e)  # rows of H: every coordinate +-1 in units of the norm
    assert ((u == 10) | (u == 5)).all()  # floor(1 / 0.3352) + 8 = 10, floor(-1 / 0.3352) + 8 = 5
    assert np.allclose(t, 0.3352 / d, rtol=2 ** -22)


def test_packing_by_hand():
    u = np.arange(8, dtype=np.uint8)[None]
    # channels 0 2 4 6 in the low half's nibbles, 1 3 5 7 in the high half's
    assert paged4.pack(u)[0].tolist() == [0x20, 0x64, 0x31, 0x75]
    r = np.random.default_rng(0).integers(0, 16, (5, 3, 128), dtype=np.uint8)
    assert (paged4.unpack(paged4.pack(r)) == r).all()


@pytest.mark.parametrize("d", [64, 128])
def test_error_is_the_quantisers(d):
    """Mean square error of a normal variable: 0.01154 (J. Max, table II, N = 16), of which step^2 / 12 =
    0.00936 comes from inside the cells. Coordinates in units of their own vector's norm have lighter tails
    (excess kurtosis -6 / (d + 2)), so the error lies between the two (3 % for the sample). With a
    channel ten times larger, which the transform spreads over all, the coordinates are no longer normal
    (two bells around the channel's value), but all lie within the 16 cells or close behind, so that each
    is off by half a step at most: 0.3352^2 / 4 = 0.0281."""
    x = np.random.default_rng(1).standard_normal((4000, d)).astype(np.float32)
    for big in (1, 10):
        x[:, 3] *= big
        v = paged4.values(*paged4.encode(x))
        err = ((v - x) ** 2).sum() / (x.astype(np.float64) ** 2).sum()
        assert err < 0.3352 ** 2 / 4
        if big == 1:
            assert 0.97 * 0.3352 ** 2 / 12 < err < 1.03 * 0.01154, err


@pytest.mark.parametrize("d", [64, 128])
def test_scales(d):
    """Powers of two change the scale alone; zeros stand for zeros; what is not finite for NaN."""
    x = np.random.default_rng(2).standard_normal((50, d)).astype(np.float32)
    u, t = paged4.encode(x)
    for k in (-100, -30, 5, 120):
        u2, t2 = paged4.encode(x * np.float32(2.0) ** k)
        assert (u2 == u).all() and (t2 == t * np.float32(2.0) ** k).all()
    assert (paged4.values(*paged4.encode(np.zeros((1, d)))) == 0).all()
    x[0, 1], x[1, 2] = np.inf, np.nan
    t = paged4.encode(x)[1]
    assert np.isnan(t[:2]).all() and np.isfinite(t[2:]).all()


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation(interleaved):
    """A rotation by p then q is one by p + q, lengths stay, and scores depend on distances alone."""
    r = np.random.default_rng(3)
    x, y = (r.standard_normal((1, 2, 64)).astype(np.float32) for _ in range(2))
    angle = np.arange(40)[:, None] * 100.0 ** (-np.arange(0, 32, 2) / 32)
    c, s = np.cos(angle).astype(np.float32), np.sin(angle).astype(np.float32)
    at = lambda z, p: paged4.turn(z, c[p: p + 1], s[p: p + 1], interleaved)
    assert np.allclose(at(at(x, 5), 7), at(x, 12), atol=1e-5)
    assert np.allclose((at(x, 31) ** 2).sum(-1), (x ** 2).sum(-1), rtol=1e-5)
    assert (at(x, 9)[..., 32:] == x[..., 32:]).all() and (at(x, 0) == x).all()
    assert np.allclose((at(x, 3) * at(y, 10)).sum(-1), (at(x, 20) * at(y, 27)).sum(-1), atol=1e-4)


def test_attention_against_a_loop():
    """The attention of one row, written out with python floats."""
    import math

    r = np.random.default_rng(4)
    u = r.integers(0, 16, (2, 1, 16, 64), dtype=np.uint8)
    t = r.uniform(0.01, 0.02, (2, 1, 16)).astype(np.float32)
    Q = r.standard_normal((1, 2, 64)).astype(np.float32)
    table, T = np.array([[1, 0]]), 21
    out, lse, tol, _ = paged4.attend(u, t, u[::-1], t[::-1], Q, table, [T], [0, 1], 16, cap=3.0, window=20)
    for h in range(2):
        num, den = [0.0] * 64, 0.0
        for j in range(1, T):
            page, slot = (1, j) if j < 16 else (0, j - 16)
            k = paged4.values(u[page, 0, slot], t[page, 0, slot])
            v = paged4.values(u[1 - page, 0, slot], t[1 - page, 0, slot])
            w = math.exp(3 * math.tanh(sum(float(a) * float(b) for a, b in zip(k, Q[0, h])) / 8 / 3))
            den += w
            num = [n + w * float(x) for n, x in zip(num, v)]
        assert abs(lse[0, h] - math.log(den)) < 1e-12
        assert np.allclose(out[0, h], np.array(num) / den, atol=1e-12)
    assert (tol > 0).all()
