"""Float64 CPU oracle of the 8-bit rolling cache and of rotary positions.

TEST INFRASTRUCTURE ONLY, as the rest of this package: it shares no code with the
CUDA library and neither imports the other.

``RollingCacheQ8`` takes one token at a time.  Slots are divided into blocks of
64 (the last block of a ring may be shorter); the rows of the block being filled
are kept as they are, and its last row rounds them all, keys and values of each
head with one power-of-two scale.  A query reads, for each position in its
window, the row as it is held at that time.
"""
from __future__ import annotations

import math
from typing import Sequence

import numpy as np

from . import _f64, attend

BLOCK = 64


def round_block(x, fmt: str):
    """(numbers [rows, d], scale) of one block's rows x, from the definition: the smallest power of
    two >= 2^-100 with max |x| / scale <= 448 or 127, x / scale rounded to nearest, ties to even."""
    amax = float(np.abs(x).max()) if x.size else 0.0
    top = 448.0 if fmt == "e4m3" else 127.0
    if amax == 0.0:
        return np.zeros_like(x), 1.0
    e = -100
    while amax > math.ldexp(top, e):
        e += 1
    y = x / math.ldexp(1.0, e)
    if fmt == "int8":
        return np.rint(y), math.ldexp(1.0, e)
    # e4m3: 3 bits after the leading one, smallest exponent -6, steps of 2^-9 below it
    exp = np.maximum(np.frexp(y)[1] - 1, -6)
    step = np.ldexp(1.0, exp - 3)
    return np.rint(y / step) * step, math.ldexp(1.0, e)


class RollingCacheQ8:
    """The ring of every sequence and kv head: 8-bit numbers, scales, tails and positions."""

    def __init__(self, batch: int, n_kv_heads: int, window: int, head_dim: int, fmt: str):
        self.B, self.H, self.W, self.d, self.fmt = batch, n_kv_heads, window, head_dim, fmt
        self.blocks = -(-window // BLOCK)
        shape = (batch, n_kv_heads, window, head_dim)
        self.k8, self.v8 = np.zeros(shape), np.zeros(shape)
        self.k_scale, self.v_scale = (np.zeros((batch, n_kv_heads, self.blocks)) for _ in range(2))
        self.k_tail, self.v_tail = (np.zeros((batch, n_kv_heads, BLOCK, head_dim)) for _ in range(2))
        self.held = np.full((batch, window), -1, dtype=np.int64)   # position rounded into each slot
        self.tail_pos = np.full((batch, BLOCK), -1, dtype=np.int64)
        self.next = np.zeros(batch, dtype=np.int64)                # tokens taken in so far

    def write(self, b: int, p: int, k, v) -> None:
        """Take in the [Hkv, d] rows of position p of sequence b."""
        self.next[b] = p + 1
        slot = p % self.W
        j, row = slot // BLOCK, slot % BLOCK
        size = min(BLOCK, self.W - j * BLOCK)
        kt, vt = self.k_tail[b].copy(), self.v_tail[b].copy()
        kt[:, row], vt[:, row] = k, v
        if row + 1 < size:
            self.k_tail[b], self.v_tail[b] = kt, vt
            self.tail_pos[b, row] = p
            return
        at = slice(j * BLOCK, j * BLOCK + size)
        for h in range(self.H):
            self.k8[b, h, at], self.k_scale[b, h, j] = round_block(kt[h, :size], self.fmt)
            self.v8[b, h, at], self.v_scale[b, h, j] = round_block(vt[h, :size], self.fmt)
        self.held[b, at] = np.arange(p - size + 1, p + 1)

    def rows(self, b: int, p: int):
        """Keys and values [n, Hkv, d] and positions [n] that sequence b holds before position p."""
        ks, vs, at = [], [], []
        open_from = p - (p % self.W) % BLOCK
        for i in range(max(0, p - self.W), p):
            slot = i % self.W
            if i >= open_from:
                row = slot % BLOCK
                assert self.tail_pos[b, row] == i
                ks.append(self.k_tail[b, :, row])
                vs.append(self.v_tail[b, :, row])
            elif self.held[b, slot] == i:
                j = slot // BLOCK
                ks.append(self.k8[b, :, slot] * self.k_scale[b, :, j, None])
                vs.append(self.v8[b, :, slot] * self.v_scale[b, :, j, None])
            else:
                assert i <= p - self.W  # only what has left the window may have been overwritten
                continue
            at.append(i)
        d = self.d
        return (np.array(ks).reshape(-1, self.H, d), np.array(vs).reshape(-1, self.H, d),
                np.array(at, dtype=np.int64))


def append(cache: RollingCacheQ8, k, v, start_pos: Sequence[int], n_tokens: Sequence[int]) -> None:
    k, v = _f64(k), _f64(v)
    for b in range(cache.B):
        for t in range(int(n_tokens[b])):
            cache.write(b, int(start_pos[b]) + t, k[b, t], v[b, t])


def prefill_chunk(cache: RollingCacheQ8, q, k, v, start_pos, n_tokens, scale: float):
    """(out, spread) [B, T, Hq, d]: attention over what is held and the chunk's own rows, and the same
    weights over |v| (what rounding the weights can move); rows past n_tokens are zero."""
    q, k, v = _f64(q), _f64(k), _f64(v)
    out, spread = np.zeros(q.shape), np.zeros(q.shape)
    for b in range(cache.B):
        n, s = int(n_tokens[b]), int(start_pos[b])
        if n == 0:
            continue
        ck, cv, cp = cache.rows(b, s)
        at = s + np.arange(n, dtype=np.int64)
        kk, vv, pp = np.concatenate([ck, k[b, :n]]), np.concatenate([cv, v[b, :n]]), np.concatenate([cp, at])
        out[b, :n] = attend(q[b, :n], at, kk, vv, pp, cache.W, scale)
        spread[b, :n] = attend(q[b, :n], at, kk, np.abs(vv), pp, cache.W, scale)
    return out, spread


def decode(cache: RollingCacheQ8, q, k_new, v_new, pos, scale: float):
    """(out, spread) [B, Hq, d] of one decode step, which takes the new rows in."""
    q, k_new, v_new = _f64(q), _f64(k_new), _f64(v_new)
    out, spread = prefill_chunk(cache, q[:, None], k_new[:, None], v_new[:, None], pos, [1] * cache.B, scale)
    append(cache, k_new[:, None], v_new[:, None], pos, [1] * cache.B)
    return out[:, 0], spread[:, 0]


def rope(x, positions, inv_freq, interleaved: bool, factor: float, transpose: bool = False):
    """x [T, H, d] with row t at positions[t]: pairs of the first 2 len(inv_freq) elements turned."""
    x = _f64(x)
    y = x.copy()
    f = np.asarray(inv_freq, dtype=np.float32).astype(np.longdouble)
    ang = np.asarray(positions, dtype=np.longdouble)[:, None] * f
    cos, sin = (np.asarray(w(ang), dtype=np.float64)[:, None] for w in (np.cos, np.sin))
    if transpose:
        sin = -sin
    r = 2 * len(f)
    ia, ib = (np.arange(0, r, 2), np.arange(1, r, 2)) if interleaved else (np.arange(r // 2), np.arange(r // 2, r))
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = factor * (a * cos - b * sin), factor * (b * cos + a * sin)
    return y
