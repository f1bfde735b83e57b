"""Paged private caches, restated plainly in float64 (tests only): which page
and slot a token has, which keys a row sees, and attention over them with the
score modifiers. Loops over sequences and heads; shares no code with the
library.

``attend`` also returns what a bound on a bf16 kernel's error needs: per row
and channel the weighted mean of |v|, and per row the largest error that
float32 products and sums may leave in a score.
"""

from __future__ import annotations

import numpy as np


class Pager:
    """The pager's rules, with a list of pages per sequence: lowest free page
    first, shared pages counted, a partly filled shared page replaced before it
    is written to."""

    def __init__(self, pages: int, page_tokens: int):
        self.P, self.pages = page_tokens, pages
        self.len: dict = {}
        self.table: dict = {}

    def owners(self, page: int) -> int:
        return sum(t.count(page) for t in self.table.values())

    def free(self) -> list:
        used = {p for t in self.table.values() for p in t}
        return [p for p in range(self.pages) if p not in used]

    def _number(self) -> int:
        n = 0
        while n in self.len:
            n += 1
        return n

    def new(self) -> int:
        s = self._number()
        self.len[s], self.table[s] = 0, []
        return s

    def fork(self, seq: int) -> int:
        s = self._number()
        self.len[s], self.table[s] = self.len[seq], list(self.table[seq])
        return s

    def extend(self, seq: int, n: int):
        """The (shared, own) pair to copy, None for none, or "oom"."""
        if n == 0:
            return None
        t = self.table[seq]
        want = -(-(self.len[seq] + n) // self.P)
        own = self.len[seq] % self.P != 0 and self.owners(t[-1]) > 1
        free = self.free()
        if want - len(t) + own > len(free):
            return "oom"
        pair = None
        if own:
            pair = (t[-1], free.pop(0))
            t[-1] = pair[1]
        while len(t) < want:
            t.append(free.pop(0))
        self.len[seq] += n
        return pair

    def truncate(self, seq: int, length: int):
        del self.table[seq][-(-length // self.P):]
        self.len[seq] = length

    def end(self, seq: int):
        del self.table[seq], self.len[seq]

    def compact(self):
        """(src, dst) pairs: highest owned page into the lowest free one."""
        pairs = []
        while True:
            used = {p for t in self.table.values() for p in t}
            free = self.free()
            if not used or not free or free[0] > max(used):
                return pairs
            a, b = max(used), free[0]
            pairs.append((a, b))
            for t in self.table.values():
                t[:] = [b if p == a else p for p in t]


def token_slots(table_row, first: int, count: int, P: int):
    """(page, slot) of tokens first ... first + count - 1."""
    j = np.arange(first, first + count)
    return np.asarray(table_row)[j // P], j % P


def append(K_pages, layer, X, table, kv_len, q_start):
    """Write X [tokens, kv_heads, d] into K_pages (in place)."""
    P = K_pages.shape[3]
    for s in range(len(kv_len)):
        a, b = int(q_start[s]), int(q_start[s + 1])
        page, slot = token_slots(table[s], int(kv_len[s]) - (b - a), b - a, P)
        for i in range(b - a):
            K_pages[layer, page[i], :, slot[i]] = X[a + i]


def sees(p: int, T: int, window=0, first=0, prefix=0):
    """Boolean [T]: the keys that a row at position p sees."""
    j = np.arange(T)
    near = j <= p
    if window:
        near &= j > p - window
    return (near | (j < prefix)) & (j >= first)


def attend(K_pages, V_pages, layer, Q, table, kv_len, q_start, cap=0.0, slopes=None, window=0, first=None, prefix=None,
           scale=None):
    """Float64 (out [tokens, q_heads, d], lse [tokens, q_heads], mean |v| like
    out, score error like lse); rows of no sequence are NaN."""
    P, d = K_pages.shape[3:]
    hk = K_pages.shape[2]
    n_tok, hq = Q.shape[:2]
    G = hq // hk
    scale = d ** -0.5 if scale is None else scale
    out = np.full((n_tok, hq, d), np.nan)
    mag = np.full((n_tok, hq, d), np.nan)
    lse = np.full((n_tok, hq), np.nan)
    err = np.full((n_tok, hq), np.nan)
    for s in range(len(kv_len)):
        a, b, T = int(q_start[s]), int(q_start[s + 1]), int(kv_len[s])
        page, slot = token_slots(table[s], 0, T, P)
        for h in range(hq):
            k = K_pages[layer, page, h // G, slot].astype(np.float64)
            v = V_pages[layer, page, h // G, slot].astype(np.float64)
            for i in range(b - a):
                p = T - (b - a) + i
                m = sees(p, T, window, 0 if first is None else int(first[a + i]), 0 if prefix is None else int(prefix[s]))
                q = Q[a + i, h].astype(np.float64)
                x = scale * (k[m] @ q)
                # a float32 dot product of d terms, its scaling, and the cap's tanh
                e = (d + 2) * 2.0 ** -24 * scale * (np.abs(k[m]) @ np.abs(q)) + 2.0 ** -23 * np.abs(x)
                if cap:
                    x = cap * np.tanh(x / cap)
                    e = e + cap * 2.0 ** -21
                if slopes is not None:
                    far = float(slopes[h]) * np.abs(p - np.arange(T)[m])
                    x, e = x - far, e + 2.0 ** -22 * far
                if not m.any():
                    out[a + i, h], lse[a + i, h], mag[a + i, h], err[a + i, h] = 0.0, -np.inf, 0.0, 0.0
                    continue
                top = x.max()
                w = np.exp(x - top)
                out[a + i, h] = (w @ v[m]) / w.sum()
                mag[a + i, h] = (w @ np.abs(v[m])) / w.sum()
                lse[a + i, h] = top + np.log(w.sum())
                err[a + i, h] = e.max() + 2.0 ** -23 * np.abs(x).max()
    return out, lse, mag, err
