"""Plain statements of the paged-cache operators for the tests: bookkeeping in
Python integers and numpy rows, attention in 64 bits."""
from __future__ import annotations

import math

import numpy as np


class RefPool:
    """One sequence is the list of its rows; pages, counts and tables are kept as the operators define them."""

    def __init__(self, n_pages, page_size, n_seqs, max_pages):
        self.ps, self.max_pages = page_size, max_pages
        self.refs = np.zeros(n_pages, np.int32)
        self.lens = np.zeros(n_seqs, np.int32)
        self.table = np.zeros((n_seqs, max_pages), np.int32)

    def held(self, s):
        return -(-int(self.lens[s]) // self.ps)

    def _take(self):
        i = int(np.flatnonzero(self.refs == 0)[0])
        self.refs[i] = 1
        return i

    def append(self, seqs, counts):
        """Places (page, row) of the new rows, in order; None when the call must be refused."""
        need = sum(-(-(int(self.lens[s]) + c) // self.ps) - self.held(s) for s, c in zip(seqs, counts))
        if need > int((self.refs == 0).sum()) or any(int(self.lens[s]) + c > self.ps * self.max_pages for s, c in zip(seqs, counts)):
            return None
        places = []
        for s, c in zip(seqs, counts):
            for _ in range(c):
                n = int(self.lens[s])
                if n % self.ps == 0:
                    self.table[s, n // self.ps] = self._take()
                places.append((int(self.table[s, n // self.ps]), n % self.ps))
                self.lens[s] = n + 1
        return places

    def fork(self, src, dst, rows=None):
        """Copies (from page, to page, rows); None when refused."""
        rows = [int(self.lens[s]) for s in src] if rows is None else rows
        if sum(1 for m in rows if m % self.ps) > int((self.refs == 0).sum()):
            return None
        copies = []
        for s, d, m in zip(src, dst, rows):
            for j in range(m // self.ps):
                self.table[d, j] = self.table[s, j]
                self.refs[self.table[s, j]] += 1
        for s, d, m in zip(src, dst, rows):
            j, t = m // self.ps, m % self.ps
            if t:
                self.table[d, j] = self._take()
                copies.append((int(self.table[s, j]), int(self.table[d, j]), t))
            self.lens[d] = m
        return copies

    def free(self, seqs, compact=False):
        """Moves (from page, to page)."""
        for s in dict.fromkeys(int(x) for x in seqs):
            for j in range(self.held(s)):
                self.refs[self.table[s, j]] -= 1
            self.lens[s] = 0
        if not compact:
            return []
        live = int((self.refs > 0).sum())
        holes = [i for i in range(live) if self.refs[i] == 0]
        moved = [i for i in range(live, len(self.refs)) if self.refs[i] > 0]
        to = dict(zip(moved, holes))
        for a, b in to.items():
            self.refs[b], self.refs[a] = self.refs[a], 0
        for s in range(len(self.lens)):
            for j in range(self.held(s)):
                self.table[s, j] = to.get(int(self.table[s, j]), int(self.table[s, j]))
        return list(to.items())


def attention(q, k_rows, v_rows, scale):
    """q [heads][hs], k_rows / v_rows [n][kv][hs], 64 bits.  Returns (out, lse, sum of w |v|, max of scale sum |q k|)."""
    H, KV = q.shape[0], k_rows.shape[1] if k_rows.ndim == 3 else 1
    out = np.zeros(q.shape)
    lse = np.full(H, -np.inf)
    mag = np.zeros(q.shape)
    spread = 0.0
    if len(k_rows):
        for h in range(H):
            g = h * KV // H
            x = scale * (k_rows[:, g] @ q[h])
            spread = max(spread, abs(scale) * float((np.abs(k_rows[:, g]) @ np.abs(q[h])).max()))
            m = x.max()
            w = np.exp(x - m)
            lse[h] = m + math.log(w.sum())
            w /= w.sum()
            out[h] = w @ v_rows[:, g]
            mag[h] = w @ np.abs(v_rows[:, g])
    return out, lse, mag, spread
