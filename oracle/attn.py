"""Float64 CPU oracle for the windowed attention, its backward pass, the paged decode step and the paged cache's books.

TEST INFRASTRUCTURE ONLY, like ``oracle.scan``: the product never imports it.

Token t of a sequence sees token j when j <= t and (j > t - window or j < n_sink); window 0 (decode) sees all j <= t.
The gradients are the formula's, row by row; the books are walked entry by entry in plain Python.
"""

from __future__ import annotations

import numpy as np

__all__ = ["visible", "window_attn", "window_attn_backward", "paged_attn_step", "Books"]


def visible(t, window, n_sink):
    """The tokens that token t sees, in order."""
    return [j for j in range(t + 1) if window <= 0 or j > t - window or j < n_sink]


def _row(q, k, v, vis, scale):
    s = scale * (k[vis] @ q)
    top = s.max()
    e = np.exp(s - top)
    return e / e.sum(), top + np.log(e.sum())


def window_attn(q, k, v, window, n_sink=0, lens=None, scale=None):
    """q [B,H,L,dk], k [B,Hkv,L,dk], v [B,Hkv,L,dv] -> (o [B,H,L,dv], lse [B,H,L]); rows behind lens[b] are 0."""
    q, k, v = (np.asarray(x, dtype=np.float64) for x in (q, k, v))
    B, H, L, dk = q.shape
    Hkv = k.shape[1]
    scale = dk ** -0.5 if scale is None else scale
    o, lse = np.zeros((B, H, L, v.shape[-1])), np.zeros((B, H, L))
    for b in range(B):
        n = L if lens is None else min(max(int(lens[b]), 0), L)
        for h in range(H):
            g = h // (H // Hkv)
            for t in range(n):
                vis = visible(t, window, n_sink)
                p, lse[b, h, t] = _row(q[b, h, t], k[b, g], v[b, g], vis, scale)
                o[b, h, t] = p @ v[b, g][vis]
    return o, lse


def window_attn_backward(q, k, v, dO, window, n_sink=0, lens=None, scale=None):
    """Gradients of sum(o * dO): {"dq", "dk", "dv"}."""
    q, k, v, dO = (np.asarray(x, dtype=np.float64) for x in (q, k, v, dO))
    B, H, L, d = q.shape
    Hkv = k.shape[1]
    scale = d ** -0.5 if scale is None else scale
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    for b in range(B):
        n = L if lens is None else min(max(int(lens[b]), 0), L)
        for h in range(H):
            g = h // (H // Hkv)
            for t in range(n):
                vis = visible(t, window, n_sink)
                p, _ = _row(q[b, h, t], k[b, g], v[b, g], vis, scale)
                dp = v[b, g][vis] @ dO[b, h, t]
                ds = p * (dp - p @ dp)
                dq[b, h, t] = scale * (ds @ k[b, g][vis])
                dk[b, g][vis] += scale * ds[:, None] * q[b, h, t]
                dv[b, g][vis] += p[:, None] * dO[b, h, t]
    return {"dq": dq, "dk": dk, "dv": dv}


def paged_attn_step(q, k_pages, v_pages, table, lens, rows=None, window=0, n_sink=0, scale=None):
    """q [n,H,dk] against row rows[i] (or i) of the paged cache -> (o [n,H,dv], lse [n,H])."""
    q, k_pages, v_pages = (np.asarray(x, dtype=np.float64) for x in (q, k_pages, v_pages))
    n, H, dk = q.shape
    _, Hkv, page, dv = v_pages.shape
    scale = dk ** -0.5 if scale is None else scale
    o, lse = np.zeros((n, H, dv)), np.full((n, H), -np.inf)
    for i in range(n):
        r = i if rows is None else int(rows[i])
        if lens[r] == 0:
            continue
        vis = np.array(visible(int(lens[r]) - 1, window, n_sink))
        at = np.asarray(table)[r][vis // page], vis % page
        for h in range(H):
            g = h // (H // Hkv)
            k, v = k_pages[at[0], g, at[1]], v_pages[at[0], g, at[1]]
            p, lse[i, h] = _row(q[i, h], k, v, np.arange(len(vis)), scale)
            o[i, h] = p @ v
    return o, lse


class Books:
    """The paged cache's books: lists of Python ints, changed one entry at a time.  Calls that cannot be carried out
    return the name of their status and change nothing."""

    def __init__(self, num_pages, page_size, rows, max_pages):
        self.page, self.most = page_size, max_pages
        self.table = [[-1] * max_pages for _ in range(rows)]
        self.lens, self.refs = [0] * rows, [0] * num_pages

    def _free(self):
        return [p for p, n in enumerate(self.refs) if n == 0]

    def _held(self, n):
        return -(-n // self.page)

    def reserve(self, rows, counts):
        if any(not 0 <= r < len(self.lens) for r in rows) or len(set(rows)) < len(rows) or min(counts, default=0) < 0:
            return "invalid"
        if any(self.lens[r] + c > self.most * self.page for r, c in zip(rows, counts)):
            return "capacity"
        free = self._free()
        need = [self._held(self.lens[r] + c) - self._held(self.lens[r]) for r, c in zip(rows, counts)]
        if sum(need) > len(free):
            return "capacity"
        for r, c, k in zip(rows, counts, need):
            for e in range(self._held(self.lens[r]), self._held(self.lens[r]) + k):
                self.table[r][e] = free.pop(0)
                self.refs[self.table[r][e]] = 1
            self.lens[r] += c
        return "ok"

    def fork(self, src, dst):
        none = [(-1, -1)] * len(src)
        if any(not 0 <= r < len(self.lens) for r in [*src, *dst]):
            return "invalid", none
        if any(self.lens[r] for r in dst) or len(set(dst)) < len(dst) or set(src) & set(dst):
            return "invalid", none
        free = self._free()
        if sum(self.lens[r] % self.page != 0 for r in src) > len(free):
            return "capacity", none
        moves = []
        for a, b in zip(src, dst):
            full = self.lens[a] // self.page
            self.lens[b] = self.lens[a]
            self.table[b][:full] = self.table[a][:full]
            for p in self.table[a][:full]:
                self.refs[p] += 1
            moves.append((-1, -1))
            if self.lens[a] % self.page:
                self.table[b][full] = free.pop(0)
                self.refs[self.table[b][full]] = 1
                moves[-1] = (self.table[a][full], self.table[b][full])
        return "ok", moves

    def free(self, rows):
        if any(not 0 <= r < len(self.lens) for r in rows):
            return "invalid"
        for r in rows:
            for e in range(self._held(self.lens[r])):
                self.refs[self.table[r][e]] -= 1
                self.table[r][e] = -1
            self.lens[r] = 0
        return "ok"

    def compact(self):
        used = sum(n > 0 for n in self.refs)
        holes = [p for p in self._free() if p < used]
        movers = [p for p, n in enumerate(self.refs) if n > 0 and p >= used]
        to = dict(zip(movers, holes))
        for a, b in to.items():
            self.refs[b], self.refs[a] = self.refs[a], 0
        self.table = [[to.get(p, p) for p in row] for row in self.table]
        moves = list(to.items())
        return moves + [(-1, -1)] * (len(self.refs) // 2 - len(moves))
