"""The 4-bit key/value cache in 64 bits (numpy): what the library's kernels are
tested against.  TEST INFRASTRUCTURE ONLY, as the rest of this package.

Written from the definitions: a group of 32 dimensions of one token's head
holds codes q in [0, 15], an integral zero and a scale of seven significant
bits, and stands for scale * (q - zero).
"""
from __future__ import annotations

import numpy as np

GROUP = 32
TILE = 16
CLAMP = 57344.0


def encode(x):
    """x [..., D] (any float type) -> (codes uint8 [..., D], scale fp64 and
    zero int [..., D / 32]); a group with a NaN has scale NaN."""
    x = np.asarray(x).astype(np.float64)
    g = x.reshape(*x.shape[:-1], x.shape[-1] // GROUP, GROUP)
    nan = np.isnan(g).any(-1)
    g = np.clip(np.where(nan[..., None], 0.0, g), -CLAMP, CLAMP)
    lo, hi = np.minimum(g.min(-1), 0.0), np.maximum(g.max(-1), 0.0)
    d = (hi - lo) / 15.0
    with np.errstate(divide="ignore"):
        power = np.frexp(d)[1] - 1                       # d in [2^power, 2^(power + 1))
    unit = np.ldexp(1.0, np.maximum(np.where(d > 0, power - 6, -20), -20))
    scale = np.maximum(np.ceil(d / unit) * unit, 2.0 ** -20)
    zero = np.rint(-lo / scale)
    codes = np.clip(np.rint(g / scale[..., None]) + zero[..., None], 0, 15)
    codes = np.where(nan[..., None], 0, codes).astype(np.uint8)
    return codes.reshape(x.shape), np.where(nan, np.nan, scale), np.where(nan, 0, zero).astype(np.int64)


def values(codes, scale, zero):
    """scale * (code - zero), fp64."""
    g = codes.reshape(*codes.shape[:-1], codes.shape[-1] // GROUP, GROUP).astype(np.float64)
    return (scale[..., None] * (g - zero[..., None])).reshape(codes.shape)


def held(x):
    """What x stands for once it is in the cache."""
    return values(*encode(x))


def tile_bytes(dim):
    return TILE * (dim + dim // 8)


def store(cache, kv_heads, dim, page_tokens, k, v, slots):
    """Write rows k, v [tokens, kv_heads, D] into cache (uint8 [bytes]) byte by
    byte as the layout says; slots outside the cache are passed over."""
    size, tiles = tile_bytes(dim), page_tokens // TILE
    pages = cache.size // (size * tiles * kv_heads)
    for which, x in enumerate((k, v)):
        codes, scale, zero = encode(x)
        word = (scale.astype(np.float16).view(np.uint16) & 0xFFF0) | zero.astype(np.uint16)
        for t, slot in enumerate(slots):
            if slot < 0 or slot >= pages * page_tokens:
                continue
            page, off = divmod(int(slot), page_tokens)
            for h in range(kv_heads):
                base = ((page * kv_heads + h) * tiles + off // TILE) * size
                at = base + which * TILE * dim // 2 + off % TILE * (dim // 2)
                cache[at:at + dim // 2] = codes[t, h, 0::2] | (codes[t, h, 1::2] << 4)
                at = base + TILE * dim + which * TILE * dim // 16 + 2 * (off % TILE)
                for g in range(dim // GROUP):
                    cache[at + 2 * TILE * g:at + 2 * TILE * g + 2] = np.array([word[t, h, g]], "<u2").view(np.uint8)


def load(cache, kv_heads, dim, page_tokens, slots):
    """fp64 (k, v) [tokens, kv_heads, D] at slots inside the cache."""
    slots = np.asarray(slots, np.int64)
    size, tiles = tile_bytes(dim), page_tokens // TILE
    page, off = slots // page_tokens, slots % page_tokens
    base = ((page[:, None] * kv_heads + np.arange(kv_heads)) * tiles + off[:, None] // TILE) * size
    row = (off % TILE)[:, None, None]
    found = []
    for which in (0, 1):
        b = cache[base[..., None] + which * TILE * dim // 2 + row * (dim // 2) + np.arange(dim // 2)]
        codes = np.stack((b & 15, b >> 4), -1).reshape(*b.shape[:-1], dim)
        at = base[..., None] + TILE * dim + which * TILE * dim // 16 + 2 * TILE * np.arange(dim // GROUP) + 2 * row
        word = cache[at].astype(np.uint16) | (cache[at + 1].astype(np.uint16) << 8)
        scale = (word & 0xFFF0).view(np.float16).astype(np.float64)
        found.append(values(codes, scale, (word & 15).astype(np.int64)))
    return found


def attend(q, k, v, scale, positions=None, window=0):
    """One sequence: q [n, q_heads, D] over k, v [T, kv_heads, D], fp64.
    positions [n]: a query sees tokens up to its own (None: all), the last
    ``window`` of them if that is not 0.  Returns (out, lse, spread): spread
    is sum_j p_j |v_j|, the scale of out's rounding errors."""
    n, heads, dim = q.shape
    share, T = heads // k.shape[1], k.shape[0]
    seen = np.ones((n, T), bool)
    if positions is not None:
        t = np.arange(T)
        seen = t <= positions[:, None]
        if window:
            seen &= t > positions[:, None] - window
    out, spread = np.zeros((n, heads, dim)), np.zeros((n, heads, dim))
    lse = np.full((n, heads), -np.inf)
    for h in range(heads):
        y = scale * (q[:, h].astype(np.float64) @ k[:, h // share].T)
        for i in range(n):
            at = np.flatnonzero(seen[i])
            if at.size == 0:
                continue
            top = y[i, at].max()
            e = np.exp(y[i, at] - top)
            lse[i, h] = top + np.log(e.sum())
            out[i, h] = e / e.sum() @ v[at, h // share]
            spread[i, h] = e / e.sum() @ np.abs(v[at, h // share])
    return out, lse, spread
