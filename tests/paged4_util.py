"""Helpers of the tests of paged caches in 4 bits: caches whose pages lie
scattered and whose unused slots hold NaN scales, and the check of attention."""

import numpy as np

from oracle import paged, paged4

from paged_util import Batch, bf16


class Batch4(Batch):
    """A Batch (queries, tables, lengths) whose pages are codes and scales."""

    def __init__(self, hk, hq, d, P, q, kv, seed=0, layers=1, layer=0, extra_rows=0, garbage=-7):
        super().__init__(hk, hq, d, P, q, kv, seed, layers, layer, extra_rows, garbage)
        r = np.random.default_rng(seed + 1000)
        shape = self.K.shape
        self.codes, self.scale = [], []
        for X in (self.K, self.V):
            known = np.isfinite(X).all(-1)
            u = r.integers(0, 16, shape, dtype=np.uint8)
            t = np.full(shape[:-1], np.nan, np.float32)
            u[known], t[known] = paged4.encode(X[known])
            self.codes.append(u)
            self.scale.append(t)

    def pages4(self, kp):
        import torch

        return kp.Pages4(*(torch.from_numpy(paged4.pack(u)).cuda() for u in self.codes),
                         *(torch.from_numpy(t).cuda() for t in self.scale))

    def dev4(self, kp):
        """(pages, layer, Q, table, kv_len, q_start) on the GPU."""
        import torch

        i = lambda x: torch.from_numpy(x).cuda()
        return (self.pages4(kp), self.layer, torch.from_numpy(self.Q).cuda().to(torch.bfloat16), i(self.table),
                i(self.kv_len), i(self.q_start))

    def ref4(self, **score):
        (uk, uv), (tk, tv) = self.codes, self.scale
        z = self.layer
        with np.errstate(invalid="ignore"):
            return paged4.attend(uk[z], tk[z], uv[z], tv[z], self.Q, self.table, self.kv_len, self.q_start, self.P, **score)


def check4(out, lse, ref):
    """out (bf16 values) and lse within the reference's bounds; rows of no sequence are passed over."""
    o, z, tol, tolz = ref
    mine = ~np.isnan(z)
    o, z, tol, tolz = o[mine], z[mine], tol[mine], tolz[mine]
    out, lse = out[mine].astype(np.float64), lse[mine].astype(np.float64)
    assert np.isfinite(out).all()
    empty = np.isneginf(z)
    assert (np.isneginf(lse) == empty).all() and (out[empty] == 0).all()
    worst = np.max(np.abs(out - o)[~empty] / tol[~empty]) if (~empty).any() else 0.0
    assert worst <= 1.0, f"output {worst:.3g} times its bound"
    d = np.abs(lse[~empty] - z[~empty]) / tolz[~empty]
    assert (d <= 1).all(), f"lse {np.max(d):.3g} times its bound"
    return worst


def rotation(positions, dim, base=10000.0):
    """cos, sin float32 [positions, dim / 2] (numpy, from angles in 64 bits)."""
    angle = np.arange(positions)[:, None] * base ** (-np.arange(0, dim, 2) / dim)
    return np.cos(angle).astype(np.float32), np.sin(angle).astype(np.float32)


def new_rows(b, seed, heads):
    """bf16 rows [tokens, heads, d] with channels of different sizes."""
    r = np.random.default_rng(seed)
    return bf16(r.standard_normal((b.tokens, heads, b.d), dtype=np.float32) * np.exp(r.standard_normal((heads, b.d))))


def token_positions(b):
    """Position of every row of the batch (-1: a row of nobody)."""
    at = np.full(b.tokens, -1)
    for s, n in enumerate(b.q):
        at[b.q_start[s]: b.q_start[s + 1]] = b.kv[s] - n + np.arange(n)
    return at


def place(pages, layer, rows, b):
    """Rows [tokens, heads, ...] into pages [layers, pages, heads, P, ...] of b's tables."""
    for s, n in enumerate(b.q):
        page, slot = paged.token_slots(b.table[s], b.kv[s] - n, n, b.P)
        for i in range(n):
            pages[layer, page[i], :, slot[i]] = rows[b.q_start[s] + i]
