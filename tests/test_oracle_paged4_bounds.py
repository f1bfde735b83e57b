"""What the restatement's bounds on attention over 4-bit caches let pass and what
they do not: the steps of a kernel restated in float32 and fp16, as they should
be and with mistakes in them."""

import functools

import numpy as np
import pytest

from oracle import paged4

from paged4_util import check4
from paged_util import bf16

F = np.float32


def codes(T, d, seed, k_size=1.0):
    r = np.random.default_rng(seed)
    k, v = (r.standard_normal((T, d)).astype(F) for _ in range(2))
    return paged4.encode(k * F(k_size)), paged4.encode(v)


def transformed(q):
    """H q in float32, stage by stage."""
    y, h, d = q.astype(F), 1, q.shape[-1]
    while h < d:
        z = y.reshape(-1, d // (2 * h), 2, h)
        y = np.stack([z[:, :, 0] + z[:, :, 1], z[:, :, 0] - z[:, :, 1]], 2).reshape(-1, d)
        h *= 2
    return y


def restated(K, V, Q, seen, scores="two parts"):
    """Rows Q [R, d] over keys K, V (codes and scales), seen [R, T]: out (bf16 values), lse."""
    (uk, tk), (uv, tv) = K, V
    d = Q.shape[-1]
    e = np.frexp(np.abs(Q).max(-1, keepdims=True))[1]
    q = Q * np.ldexp(F(1), -e)
    y = transformed(q)
    c = (uk - 7.5).astype(F)
    if scores == "scaled keys":  # code times scale in fp16, one part
        k = (c * tk[:, None] * F(64)).astype(np.float16).astype(F)
        x = (y.astype(np.float16).astype(F) @ k.T) / F(64)
    else:
        hi = y.astype(np.float16)
        lo = (y - hi.astype(F)).astype(np.float16)
        acc = F(0.5) * y.sum(-1, keepdims=True) + hi.astype(F) @ (c - F(0.5)).T
        if scores == "one part":  # and the factor that makes the rounded row's product with the row exact
            g = hi.astype(F)
            acc = F(0.5) * g.sum(-1, keepdims=True) + g @ (c - F(0.5)).T
            acc = acc * ((y * y).sum(-1, keepdims=True) / (y * g).sum(-1, keepdims=True))
        else:
            acc = acc + lo.astype(F) @ (c - F(0.5)).T
        x = acc * tk
    x = x * np.ldexp(F(1), e) * F(d ** -0.5)
    x = np.where(seen, x, F(-np.inf))
    top = x.max(-1, keepdims=True)
    w = np.exp(x - top)
    l = w.sum(-1, keepdims=True)
    if scores == "weights in e4m3":  # (four bits: half a step is 2^-4)
        m, n = np.frexp(w)
        w = np.ldexp(np.round(m * 16) / 16, n).astype(F)
    o = bf16(w * tv) @ (uv - 7.5).astype(F)
    out = bf16(transformed(o) / l)
    return out[:, None], (top + np.log(l))


def reference(K, V, Q, seen, T):
    """attend's result of one head whose rows see the last keys of T."""
    P = 128
    pages = -(-T // P)
    shaped = []
    for u, t in (K, V):
        full = np.zeros((pages * P,) + u.shape[1:], u.dtype), np.zeros(pages * P, F)
        full[0][:T], full[1][:T] = u, t
        shaped += [full[0].reshape(pages, 1, P, -1), full[1].reshape(pages, 1, P)]
    R = len(Q)
    first = np.argmax(seen, -1).astype(np.int32)
    # every row the last of a sequence of its own over the same pages
    table = np.broadcast_to(np.arange(pages), (R, pages))
    return paged4.attend(*shaped, Q[:, None], table, [T] * R, np.arange(R + 1), P, first=first)


CASES = {  # keys, queries' size, keys seen, one that stands out
    "few": (300, 1, 300, False),
    "flat": (5000, 1, 5000, False),
    "long": (20000, 1, 20000, False),
    "large": (20000, 8, 20000, False),
    "peak": (20000, 1, 20000, True),
    "window16": (20000, 1, 16, False),
    "window1": (20000, 1, 1, False),
}


@functools.cache
def case(name, d):
    T, size, window, peak = CASES[name]
    K, V = codes(T, d, T)
    Q = bf16(np.random.default_rng(5).standard_normal((20, d)).astype(F) * F(size))
    if peak:
        r = np.random.default_rng(6)
        u, t = paged4.encode((1.5 * Q[0] + 4 * r.standard_normal(d)).astype(F)[None])
        K[0][T // 3], K[1][T // 3] = u[0], t[0]
        Q[:] = bf16(Q[0] + 0.3 * r.standard_normal(Q.shape).astype(F))
    seen = np.broadcast_to(np.arange(T) >= T - window, (20, T))
    return K, V, Q, seen, reference(K, V, Q, seen, T)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("name", sorted(CASES))
def test_what_is_right_passes(name, d):
    K, V, Q, seen, ref = case(name, d)
    out, lse = restated(K, V, Q, seen)
    assert check4(out, lse, ref) < 0.9  # (and not by much more than a rounding of the output)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("name,scores", [("large", "one part"), ("peak", "one part"), ("window16", "one part"),
                                         ("window1", "one part"), ("few", "scaled keys"), ("large", "scaled keys"),
                                         ("window16", "scaled keys"), ("peak", "scaled keys")])
def test_scores_in_fewer_bits_do_not(name, scores, d):
    K, V, Q, seen, ref = case(name, d)
    with pytest.raises(AssertionError, match="times its bound"):
        check4(*restated(K, V, Q, seen, scores), ref)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("name", ["few", "flat", "long", "window16"])
def test_wrong_outputs_do_not(name, d):
    K, V, Q, seen, ref = case(name, d)
    out, lse = restated(K, V, Q, seen)
    with pytest.raises(AssertionError, match="output"):
        check4(restated(K, V, Q, seen, "weights in e4m3")[0], lse, ref)
    # of an output of zeros few elements lie within their bounds
    o, _, tol, _ = ref
    assert np.mean(np.abs(o) <= tol) < 0.1
