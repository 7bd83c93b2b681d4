"""Decoder-serving operators from their definitions: causal attention with grouped heads over packed prompts, and
a paged key-value cache kept with plain Python lists (fp64 arithmetic, exact page bookkeeping)."""
from __future__ import annotations

import numpy as np


class CacheError(Exception):
    """A call that the cache refuses; `code` is the device error word's value."""

    def __init__(self, code):
        super().__init__(code)
        self.code = code


LENGTH, ROWS, SLOT, PAGE, FULL = 1, 3, 5, 6, 7


def attend(q, K, V, scale):
    """One query: softmax_j(scale q . K[j]) V, zeros without keys."""
    if len(K) == 0:
        return np.zeros(V.shape[-1])
    s = scale * (np.asarray(K, np.float64) @ np.asarray(q, np.float64))
    w = np.exp(s - s.max())
    return (w / w.sum()) @ np.asarray(V, np.float64)


def causal_attention(q, k, v, cu, nh, nkv, d, scale=None):
    """Packed rows q [T, nh d], k and v [T, nkv d]: row i attends to rows cu[b] .. i of its sequence."""
    scale = d ** -0.5 if scale is None else scale
    out = np.zeros((q.shape[0], nh * d))
    for b in range(len(cu) - 1):
        a, e = cu[b], cu[b + 1]
        hide = np.triu(np.ones((e - a, e - a), bool), 1)
        for h in range(nh):
            c = slice(h * d, (h + 1) * d)
            kc = slice(h // (nh // nkv) * d, (h // (nh // nkv) + 1) * d)
            s = scale * (q[a:e, c].astype(np.float64) @ k[a:e, kc].astype(np.float64).T)
            s[hide] = -np.inf
            if e > a:
                w = np.exp(s - s.max(1, keepdims=True))
                out[a:e, c] = (w / w.sum(1, keepdims=True)) @ v[a:e, kc].astype(np.float64)
    return out


class PagedCache:
    """The cache's state as lists, the pool as an array of 16-bit words (moved, never computed with)."""

    def __init__(self, layers, pages, page_size, kv_heads, head_dim, slots, max_pages):
        self.pool = np.zeros((layers, pages, 2, kv_heads, page_size, head_dim), np.uint16)
        self.ps, self.max_pages = page_size, max_pages
        self.rows = [[] for _ in range(slots)]     # page numbers
        self.lens = [0] * slots
        self.refs = [0] * pages

    def table(self):
        t = np.full((len(self.rows), self.max_pages), -1, np.int32)
        for s, row in enumerate(self.rows):
            t[s, :len(row)] = row
        return t

    def _slots(self, slots):
        if any(not 0 <= s < len(self.rows) for s in slots) or len(set(slots)) < len(slots):
            raise CacheError(SLOT)

    def _take(self, n):
        free = [p for p, r in enumerate(self.refs) if r == 0]
        if n > len(free):
            raise CacheError(FULL)
        return free[:n]

    def reserve(self, slots, counts):
        self._slots(slots)
        for s, c in zip(slots, counts):
            if c < 0 or self.lens[s] + c > self.max_pages * self.ps:
                raise CacheError(LENGTH)
        need = [-(-(self.lens[s] + c) // self.ps) - len(self.rows[s]) for s, c in zip(slots, counts)]
        free = iter(self._take(sum(need)))
        for s, c, n in zip(slots, counts, need):
            for _ in range(n):
                p = next(free)
                self.rows[s].append(p)
                self.refs[p] = 1
            self.lens[s] += c

    def append(self, layer, k, v, slots, counts):
        """k, v: [sum counts, kv_heads, head_dim] 16-bit words."""
        self._slots(slots)
        t = 0
        for s, c in zip(slots, counts):
            for j in range(c):
                pos = self.lens[s] - c + j
                if pos < 0:
                    raise CacheError(LENGTH)
                p = self.rows[s][pos // self.ps]
                if self.refs[p] != 1:
                    raise CacheError(PAGE)
                self.pool[layer, p, 0, :, pos % self.ps] = k[t]
                self.pool[layer, p, 1, :, pos % self.ps] = v[t]
                t += 1

    def fork(self, src, dst):
        self._slots(dst)
        if any(not 0 <= s < len(self.rows) or s in dst for s in src) or any(self.lens[s] for s in dst):
            raise CacheError(SLOT)
        free = iter(self._take(sum(1 for s in src if self.lens[s] % self.ps)))
        for a, b in zip(src, dst):
            full, rest = divmod(self.lens[a], self.ps)
            self.rows[b] = self.rows[a][:full]
            for p in self.rows[b]:
                self.refs[p] += 1
            if rest:
                p = next(free)
                self.pool[:, p, :, :, :rest] = self.pool[:, self.rows[a][full], :, :, :rest]
                self.rows[b].append(p)
                self.refs[p] = 1
            self.lens[b] = self.lens[a]

    def free(self, slots):
        self._slots(slots)
        for s in slots:
            for p in self.rows[s]:
                self.refs[p] -= 1
            self.rows[s], self.lens[s] = [], 0

    def compact(self):
        """Returns (remap, live)."""
        used = [p for p, r in enumerate(self.refs) if r > 0]
        live = len(used)
        remap = {p: p for p in used if p < live}
        holes = [p for p in range(live) if self.refs[p] == 0]
        for a, b in zip([p for p in used if p >= live], holes):
            remap[a] = b
            self.pool[:, b] = self.pool[:, a]
            self.refs[b], self.refs[a] = self.refs[a], 0
        self.rows = [[remap[p] for p in row] for row in self.rows]
        return np.array([remap.get(p, -1) for p in range(len(self.refs))], np.int32), live

    def sequence(self, layer, slot):
        """K and V words of a slot's sequence: [len, kv_heads, head_dim] each."""
        n = self.lens[slot]
        if n == 0:
            e = np.zeros((0,) + self.pool.shape[3:4] + self.pool.shape[5:], np.uint16)
            return e, e
        x = self.pool[layer, self.rows[slot]]                      # [pages, 2, heads, ps, d]
        x = x.transpose(1, 0, 3, 2, 4).reshape(2, -1, x.shape[2], x.shape[4])
        return x[0, :n], x[1, :n]
