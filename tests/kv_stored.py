"""Caches of the key-value cache's tests whose codes, scales and biases are given, not quantised from values."""
from __future__ import annotations

import numpy as np

from kv_cases import cache
from oracle import kv as ref


def pairs(c: ref.Cache) -> np.ndarray:
    """A view of a cache's (scale, bias) pairs: fp16 [pages, heads, tiles of a page, 16, K or V, groups, 2]."""
    tiles = c.data.reshape(c.pages, c.heads, c.page_size // 16, -1)
    return tiles[..., 32 * c.row:].view(np.float16).reshape(*tiles.shape[:3], 16, 2, c.ng, 2)


def places(c: ref.Cache, b: int, n: int):
    """Indexes of positions 0 .. n - 1 of sequence b in pairs(c).swapaxes(0, 1)[head] (pages, tiles, rows)."""
    pos = np.arange(n)
    return c.table[b, pos // c.page_size], pos % c.page_size // 16, pos % 16


def stored(lens, *, fill, heads=1, page_size=16, D, G, bits, seed, width=None) -> ref.Cache:
    """Random codes; fill(rng, shape) gives the scales and the biases of every page, arrays of shape [.., K or V, groups]."""
    c = cache(lens, heads=heads, page_size=page_size, D=D, G=G, bits=bits, seed=seed, width=width)
    at = pairs(c)
    assert np.shares_memory(at, c.data)
    at[..., 0], at[..., 1] = fill(np.random.default_rng(seed + 1), at.shape[:-1])
    return c
