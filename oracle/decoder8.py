"""A paged key-value cache of 8-bit codes from its definition: values are code * 2^(b - 127), b a scale byte of each block
of tokens and head (fp64 arithmetic, tables and searches instead of bit tricks)."""
from __future__ import annotations

import numpy as np

from .decoder import LENGTH, PAGE, CacheError, PagedCache


def _e4m3_values():
    v = np.zeros(256)
    for c in range(256):
        sign, field, mant = (-1.0 if c & 128 else 1.0), (c >> 3) & 15, c & 7
        v[c] = sign * (mant * 2.0 ** -9 if field == 0 else (1 + mant / 8) * 2.0 ** (field - 7))
        if field == 15 and mant == 7:
            v[c] = np.nan
    return v


VALUES = {"int8": np.arange(256).astype(np.uint8).view(np.int8).astype(np.float64), "e4m3": _e4m3_values()}
TOP = {"int8": 127.0, "e4m3": 448.0}
PAST = {"int8": 127.5, "e4m3": 464.0}     # half a step past the top: what still rounds to no more than half a step off


def encode(x, kind):
    """The code (uint8) nearest to each x, the even one of two, saturated."""
    x = np.asarray(x, np.float64)
    codes = np.arange(256, dtype=np.uint8)
    keep = np.isfinite(VALUES[kind])
    if kind == "int8":
        keep &= codes != 128
    else:
        keep &= codes != 128          # -0 is given by the sign below
    v, c = VALUES[kind][keep], codes[keep]
    order = np.argsort(v)
    v, c = v[order], c[order]
    hi = np.clip(np.searchsorted(v, x), 1, len(v) - 1)
    lo = hi - 1
    dl, dh = x - v[lo], v[hi] - x
    even = c[lo] % 2 == 0             # neighbours differ by one in their codes, so one of the two is even
    code = np.where((dl < dh) | ((dl == dh) & even), c[lo], c[hi])
    if kind == "e4m3":
        code = np.where((code == 0) & np.signbit(x), np.uint8(128), code)
    return code.astype(np.uint8)


def scale(b):
    b = np.asarray(b, np.float64)
    return np.where(b == 255, np.nan, 2.0 ** (b - 127))


def scale_byte(most, kind):
    """The smallest byte at which `most` is no more than half a step past the largest code."""
    if not np.isfinite(most):
        return 255
    for b in range(255):
        if most <= PAST[kind] * 2.0 ** (b - 127):
            return b
    raise AssertionError(most)


class PagedCache8(PagedCache):
    def __init__(self, layers, pages, page_size, kv_heads, head_dim, slots, max_pages, kind, block):
        super().__init__(layers, pages, page_size, kv_heads, head_dim, slots, max_pages)
        self.pool = np.zeros(self.pool.shape, np.uint8)
        self.scales = np.zeros(self.pool.shape[:4] + (page_size // block,), np.uint8)
        self.kind, self.block = kind, block

    def append(self, layer, k, v, slots, counts):
        """k, v: [sum counts, kv_heads, head_dim] values."""
        self._slots(slots)
        t = 0
        for s, c in zip(slots, counts):
            if c > self.lens[s]:
                raise CacheError(LENGTH)
            begin = self.lens[s] - c
            at = begin
            while at < self.lens[s]:
                end = min(self.lens[s], at // self.block * self.block + self.block)
                page = self.rows[s][at // self.ps]
                if self.refs[page] != 1:
                    raise CacheError(PAGE)
                for kv, x in ((0, k), (1, v)):
                    for h in range(x.shape[1]):
                        self._block(layer, page, kv, h, at % self.ps, x[t:t + end - at, h].astype(np.float64))
                t += end - at
                at = end

    def _block(self, layer, page, kv, h, row, x):
        """Rows x from `row` of a page on, all in one block."""
        j, old = row // self.block, row % self.block
        codes, scales = self.pool[layer, page, kv, h], self.scales[layer, page, kv, h]
        b = scale_byte(np.abs(x).max() if np.isfinite(x).all() else np.inf, self.kind)
        if old:
            b = max(b, int(scales[j]))
            if b > scales[j] and b != 255:
                was = VALUES[self.kind][codes[row - old:row]]
                codes[row - old:row] = encode(was * 2.0 ** (int(scales[j]) - b), self.kind)
        codes[row:row + len(x)] = 0 if b == 255 else encode(x / 2.0 ** (b - 127), self.kind)
        scales[j] = b

    def fork(self, src, dst):
        ends = [(a, b, divmod(self.lens[a], self.ps)) for a, b in zip(src, dst)]
        super().fork(src, dst)
        for a, b, (full, rest) in ends:
            if rest:
                n = -(-rest // self.block)
                self.scales[:, self.rows[b][full], :, :, :n] = self.scales[:, self.rows[a][full], :, :, :n]

    def compact(self):
        remap, live = super().compact()
        for a, b in enumerate(remap):
            if b >= 0 and b != a:
                self.scales[:, b] = self.scales[:, a]
        return remap, live

    def values(self, layer, slot):
        """K and V of a slot's sequence: [len, kv_heads, head_dim] each, fp64."""
        n = self.lens[slot]
        pages = self.rows[slot]
        x = VALUES[self.kind][self.pool[layer, pages]] * np.repeat(scale(self.scales[layer, pages]), self.block, -1)[..., None]
        x = x.transpose(1, 0, 3, 2, 4).reshape((2, -1) + x.shape[2:3] + x.shape[4:])
        return x[0, :n], x[1, :n]


def read_back(x, top):
    """Values as a 16-bit type reads them, before its rounding: saturated at `top`, NaN kept."""
    return np.clip(x, -top, top)
