"""Plain float64 statements of the paged cache's operators (numpy, CPU).

Test infrastructure only, written from the formulas: attention over a row's
positions, the norm + rotation of a head, the cache entry of a vector, and a
page bookkeeper that does one thing after another.
"""
from __future__ import annotations

import math

import numpy as np

PAGE = 64


def e4m3_values():
    """The 256 e4m3 codes' values, from their bit fields."""
    out = np.empty(256)
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        x = math.nan if b & 127 == 127 else (m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
        out[b] = -x if b & 128 else x
    return out


def bf16_values(u16):
    """bf16 bit patterns as float64."""
    return (u16.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def page_values(pool, head_dim):
    """uint8 pool [pages, heads, bytes] as float64 [pages, heads, 64, head_dim]."""
    n, h, nb = pool.shape
    if nb == 2 * PAGE * head_dim:
        return bf16_values(np.ascontiguousarray(pool).view(np.uint16)).reshape(n, h, PAGE, head_dim)
    codes = pool[:, :, : PAGE * head_dim].reshape(n, h, PAGE, head_dim)
    scale = np.ascontiguousarray(pool[:, :, PAGE * head_dim:]).view(np.float32).astype(np.float64)
    return e4m3_values()[codes] * scale[..., None]


def row_positions(length, max_len, pos=None):
    """The positions that a row reads, as a list."""
    if not 0 <= length <= max_len:
        length = 0
    if pos is None:
        return list(range(length))
    return [int(p) for p in pos if 0 <= p < length]


def attention(q, k, v, scale):
    """q [Hq, D], k and v [n, Hkv, D] -> out [Hq, D], lse [Hq], and two
    magnitudes for error bounds: sum p |v| / sum p [Hq, D] and the largest
    scale * sum |q| |k| [Hq]."""
    hq, d = q.shape
    out, mag = np.zeros((hq, d)), np.zeros((hq, d))
    lse, size = np.full(hq, -np.inf), np.zeros(hq)
    if len(k) == 0:
        return out, lse, mag, size
    group = hq // k.shape[1]
    for h in range(hq):
        kh, vh = k[:, h // group], v[:, h // group]
        x = scale * (kh @ q[h])
        size[h] = abs(scale) * (np.abs(kh) @ np.abs(q[h])).max()
        top = x.max()
        p = np.exp(x - top)
        lse[h] = top + math.log(p.sum())
        out[h] = p @ vh / p.sum()
        mag[h] = p @ np.abs(vh) / p.sum()
    return out, lse, mag, size


def norm_rope(x, w, eps, cos, sin, neox):
    """One head's vector x [D]: norm (w None: none), rotation by cos / sin [rot / 2]."""
    y = np.array(x, dtype=np.float64)
    if w is not None:
        y = y / math.sqrt(float(np.mean(y * y)) + eps) * w
    half = len(cos)
    for i in range(half):
        a, b = (i, half + i) if neox else (2 * i, 2 * i + 1)
        ya, yb = y[a], y[b]
        y[a], y[b] = ya * cos[i] - yb * sin[i], yb * cos[i] + ya * sin[i]
    return y


class Pages:
    """Page tables, reference counts and the pages' contents, one step at a time."""

    def __init__(self, table, ref, data):
        self.table, self.ref, self.data = table.copy(), ref.copy(), data.copy()

    def take(self):
        """The lowest free page, now with one reference; -1 if there is none."""
        for p in range(len(self.ref)):
            if self.ref[p] == 0:
                self.ref[p] = 1
                return p
        return -1

    def alloc(self, old, new):
        for r in range(len(old)):
            for j in range(-(-old[r] // PAGE), -(-new[r] // PAGE)):
                self.table[r, j] = self.take()

    def fork(self, parent, child, length):
        src, dst = [], []
        for s, c, n in zip(parent, child, length):
            self.table[c] = -1
            for j in range(n // PAGE):
                self.table[c, j] = self.table[s, j]
                self.ref[self.table[s, j]] += 1
        for s, c, n in zip(parent, child, length):
            if n % PAGE == 0:
                src.append(-1), dst.append(-1)
                continue
            new = self.take()
            src.append(self.table[s, n // PAGE] if new >= 0 else -1)
            dst.append(new)
            self.table[c, n // PAGE] = new
        return src, dst

    def free(self, req):
        for r in req:
            for p in self.table[r]:
                if p >= 0:
                    self.ref[p] -= 1
            self.table[r] = -1

    def compact(self):
        n = int((self.ref > 0).sum())
        holes = [p for p in range(n) if self.ref[p] == 0]
        movers = [p for p in range(n, len(self.ref)) if self.ref[p] > 0]
        remap = np.where(self.ref > 0, np.arange(len(self.ref)), -1)
        for s, d in zip(movers, holes):
            remap[s] = d
            self.ref[d], self.ref[s] = self.ref[s], 0
        for e in np.ndindex(self.table.shape):
            if self.table[e] >= 0:
                self.table[e] = remap[self.table[e]]
        return movers, holes, remap

    def copy(self, src, dst):
        for s, d in zip(src, dst):
            if d >= 0:
                self.data[:, d] = self.data[:, s]
