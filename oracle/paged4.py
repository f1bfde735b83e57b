"""Paged private caches in 4 bits and the rotation by position, restated plainly
(tests only; shares no code with the library).

The codes are whole numbers decided by float32 arithmetic, so ``encode`` goes
through the same float32 steps as the definition states them (numpy rounds each
once). What codes stand for, and attention over it, is in float64; ``attend``
also returns what a bound on the kernels' error needs.
"""

from __future__ import annotations

import numpy as np

from oracle.paged import sees, token_slots

STEP = np.float32(0.3352)


def hadamard(d):
    """H[i, j] = (-1)^popcount(i & j)."""
    i = np.arange(d)
    both = i[:, None] & i[None, :]
    ones = np.zeros_like(both)
    while both.any():
        ones += both & 1
        both >>= 1
    return np.where(ones % 2, -1.0, 1.0)


def turn(x, cos, sin, interleaved=False):
    """Rows x [tokens, heads, d] (float32) rotated by cos, sin [tokens, R / 2]
    (float32): products and their sum, each rounded to float32 once."""
    x = np.asarray(x, np.float32)
    R = 2 * cos.shape[1]
    a, b = (np.arange(0, R, 2), np.arange(1, R, 2)) if interleaved else (np.arange(R // 2), np.arange(R // 2, R))
    c, s = cos[:, None].astype(np.float32), sin[:, None].astype(np.float32)
    out = x.copy()
    out[..., a] = x[..., a] * c - x[..., b] * s
    out[..., b] = x[..., b] * c + x[..., a] * s
    return out


def encode(x):
    """Codes uint8 [..., d] and scales float32 [...] of float32 vectors."""
    x = np.asarray(x, np.float32)
    d = x.shape[-1]
    with np.errstate(all="ignore"):
        top = np.abs(x).max(-1, keepdims=True)
        e = np.clip(np.frexp(np.where(np.isfinite(top), top, 0))[1], -126, 126)
        y = x * np.ldexp(np.float32(1), -e).astype(np.float32)
        sq = y * y
        while sq.shape[-1] > 1:
            sq = sq[..., 0::2] + sq[..., 1::2]
        step = STEP * np.sqrt(sq)
        h = 1
        while h < d:
            z = y.reshape(*x.shape[:-1], d // (2 * h), 2, h)
            y = np.stack([z[..., 0, :] + z[..., 1, :], z[..., 0, :] - z[..., 1, :]], -2).reshape(x.shape)
            h *= 2
        u = np.clip(np.floor(y * (np.float32(1) / step)) + 8, 0, 15)
        u = np.where(step > 0, u, 8)
        t = (step * np.float32(1 / d) * np.ldexp(np.float32(1), e).astype(np.float32))[..., 0]
        bad = ~np.isfinite(x).all(-1)
    return np.nan_to_num(u).astype(np.uint8), np.where(bad, np.float32(np.nan), t).astype(np.float32)


def pack(u):
    """Bytes [..., d / 2] of codes: per eight channels a little-endian word, channel
    2 k in bits 4 k, channel 2 k + 1 sixteen bits above."""
    w = np.zeros(u.shape[:-1] + (u.shape[-1] // 8,), np.uint32)
    for c in range(8):
        w |= u[..., c::8].astype(np.uint32) << (4 * (c // 2) + 16 * (c % 2))
    return w.astype("<u4").view(np.uint8)


def unpack(codes):
    w = np.ascontiguousarray(codes).view("<u4")
    u = np.empty(codes.shape[:-1] + (2 * codes.shape[-1],), np.uint8)
    for c in range(8):
        u[..., c::8] = w >> (4 * (c // 2) + 16 * (c % 2)) & 15
    return u


def values(u, t):
    """What codes stand for: float64 t H (u - 7.5)."""
    return (u.astype(np.float64) - 7.5) @ hadamard(u.shape[-1]) * np.asarray(t, np.float64)[..., None]


def attend(u_k, t_k, u_v, t_v, Q, table, kv_len, q_start, P, cap=0.0, slopes=None, window=0, first=None, prefix=None,
           scale=None):
    """Float64 attention over one layer's codes [pages, kv_heads, P, d] and
    scales [pages, kv_heads, P]: (out, lse, tol, tol_lse). The last two bound a
    kernel whose operands of the first product are exact, or H q in two fp16
    parts, and which rounds weights to bf16 once. Where many independent
    roundings meet, six standard deviations of their sum are taken (a rounding is
    uniform within half a step: 6 / sqrt(3) = 3.5 half steps), else the worst.

    Scores, of c = u - 7.5, y = H q, z = H c, t the key's scale:
    * the transform of q in float32: 7 stages, 6 sqrt(7 / 3) 2^-24 < 12 * 2^-24 of |q| |c|;
    * two fp16 parts: 2^-22 of each y_i, and 2^-20 of the largest |q_i| where the low part is
      subnormal (steps of 2^-24, sixteen times that for the channels which meet 16 (u - 8), of
      a row whose largest value lies in [1/2, 1));
    * n = d / 8 matrix steps (two parts of d / 16), each of 17 terms aligned to the largest with 24 bits or more
      and cut: 6 sqrt(17 n / 12) steps of 2^-23 of the partial sums if the cuts are independent,
      and n more if all cut the sum towards 0. Partial sums are as large as the constant term,
      the sum itself and four standard deviations of the products' sum, whichever way the product is taken;
    * eight float32 roundings of the score, and of its distance from the reference.
    The sum of n weights: chains of n / 32 additions (a row's keys go to 32 lanes and more), or of n
    where a row is done again key by key, and 40 of joins and exponentials.
    Outputs: weights bf16, 2^-8 each; matrix steps of 16 keys, as above, their errors independent
    from channel to channel of H o; the transform; half a step of bf16 at the end."""
    d = u_k.shape[-1]
    hk = u_k.shape[1]
    H = hadamard(d)
    n_tok, hq = Q.shape[:2]
    G = hq // hk
    scale = d ** -0.5 if scale is None else scale
    out, tol = np.full((n_tok, hq, d), np.nan), np.full((n_tok, hq, d), np.nan)
    lse, tol_lse = np.full((n_tok, hq), np.nan), np.full((n_tok, hq), np.nan)
    six = 6 / 3 ** 0.5
    steps = d / 8
    cuts = (6 * (17 * steps / 12) ** 0.5 + steps) * 2.0 ** -23
    for s in range(len(kv_len)):
        a, b, T = int(q_start[s]), int(q_start[s + 1]), int(kv_len[s])
        page, slot = token_slots(table[s], 0, T, P)
        for g in range(hk):
            c = u_k[page, g, slot].astype(np.float64) - 7.5
            t = t_k[page, g, slot].astype(np.float64)
            v = values(u_v[page, g, slot], t_v[page, g, slot])
            c2, z2, v2 = c ** 2, (c @ H) ** 2, v ** 2
            norm, size = np.sqrt(c2.sum(-1)), np.sqrt(v2.sum(-1))
            for h in range(g * G, g * G + G):
                for i in range(b - a):
                    p = T - (b - a) + i
                    m = sees(p, T, window, 0 if first is None else int(first[a + i]), 0 if prefix is None else int(prefix[s]))
                    r = a + i, h
                    if not m.any():
                        out[r], lse[r], tol[r], tol_lse[r] = 0.0, -np.inf, 0.0, 0.0
                        continue
                    q = Q[r].astype(np.float64)
                    y = H @ q
                    dot = c[m] @ y
                    x = scale * t[m] * dot
                    ways = np.sqrt(c2[m] @ y ** 2)
                    partial = np.abs(dot) + np.maximum(0.5 * abs(y.sum()) + 4 * (ways + 0.5 * np.sqrt((y ** 2).sum())),
                                                       4 * np.sqrt(z2[m] @ q ** 2))
                    e = scale * t[m] * (12 * 2.0 ** -24 * np.sqrt((q ** 2).sum()) * norm[m] + six * 2.0 ** -22 * ways
                                        + six * 2.0 ** -20 * np.abs(q).max() * norm[m] + cuts * partial)
                    e = e + 2.0 ** -21 * np.abs(x)
                    if cap:
                        x = cap * np.tanh(x / cap)
                        e = e + cap * 2.0 ** -21
                    if slopes is not None:
                        far = float(slopes[h]) * np.abs(p - np.arange(T)[m])
                        x, e = x - far, e + 2.0 ** -22 * far
                    top = x.max()
                    e = e + 2.0 ** -23 * np.abs(x) + 2.0 ** -23 * (top - x)
                    w = np.exp(x - top)
                    w, l = w / w.sum(), np.log(w.sum())
                    out[r], lse[r] = w @ v[m], top + l
                    n = x.size
                    chain = (n / 32 + six * n ** 0.5 + 40) * 2.0 ** -24
                    grown = np.exp(np.minimum(e, 50.0))
                    mean = np.log(w @ grown)
                    tol_lse[r] = mean + chain + 2.0 ** -20 + 2.0 ** -22 * abs(lse[r])
                    keys = n / 16 + 16
                    spread = np.sqrt(w ** 2 @ v2[m])
                    tol[r] = (2.0 ** -8 * (1 + 2.0 ** -7) * (np.abs(out[r]) + np.minimum(w @ np.abs(v[m]), six * spread))
                              + (w * (grown * np.exp(mean) - 1)) @ np.abs(v[m]) + (chain + 2.0 ** -21) * np.abs(out[r])
                              + 6 * (17 * keys / 12) ** 0.5 * 2.0 ** -23 * (w @ size[m]) / d ** 0.5
                              + keys * 2.0 ** -23 * (np.abs(out[r]) + 3 * spread)
                              + 12 * 2.0 ** -24 * np.sqrt((out[r] ** 2).sum()) + 1e-30)
    return out, lse, tol, tol_lse
