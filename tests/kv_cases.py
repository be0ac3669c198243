"""Inputs of the key-value cache's tests: seeded caches in host memory, and their copies on the GPU."""
from __future__ import annotations

import numpy as np
import torch

from oracle import kv as ref


def bf16_bits(x: np.ndarray) -> np.ndarray:
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).bfloat16().view(torch.int16).numpy().view(np.uint16)


def to_gpu(bits: np.ndarray) -> torch.Tensor:
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).view(torch.bfloat16).cuda()


def bits_of(t: torch.Tensor) -> np.ndarray:
    return t.contiguous().cpu().view(torch.int16).numpy().view(np.uint16)


def cache(lens, *, heads, page_size, D, G, bits, seed, spare=2, width=None) -> ref.Cache:
    """A cache of random bytes with a page of its own for each position of the sequences, in random order."""
    rng = np.random.Generator(np.random.PCG64(seed))
    width = width or max(1, -(-max(max(lens), 1) // page_size))
    pages = len(lens) * width + spare
    data = rng.integers(0, 256, (pages, heads, page_size, ref.token_bytes(D, G, bits)), dtype=np.uint8)
    table = rng.permutation(pages)[: len(lens) * width].reshape(len(lens), width).astype(np.int32)
    return ref.Cache(data, table, np.array(lens, np.int32), D, G, bits)


def rows(n: int, heads: int, D: int, seed: int) -> np.ndarray:
    """bf16 patterns [n, heads, D]: rows with channels off zero, a row of one value, a row of zeros, a row with an outlier."""
    rng = np.random.Generator(np.random.PCG64(seed))
    x = rng.standard_normal((n, heads, D)) + rng.standard_normal((heads, D)) ** 3 / 4
    for i in range(n):
        if i % 7 == 3:
            x[i, i % heads] = -1.375
        elif i % 7 == 4:
            x[i, i % heads] = 0.0
        elif i % 7 == 5:
            x[i, i % heads, i % D] = 90.0
    return bf16_bits(x)


def filled(lens, *, heads, page_size, D, G, bits, seed, width=None) -> ref.Cache:
    """A cache whose sequences hold quantised rows; random bytes (NaN scales among them) behind their ends."""
    c = cache(lens, heads=heads, page_size=page_size, D=D, G=G, bits=bits, seed=seed, width=width)
    total = int(sum(lens))
    offsets = np.concatenate(([0], np.cumsum(lens)))
    ref.append(c, rows(total, heads, D, seed + 1), rows(total, heads, D, seed + 2), offsets)
    return c


def on_gpu(c: ref.Cache):
    """(cache, table, lens) on the GPU."""
    return torch.from_numpy(c.data).cuda(), torch.from_numpy(c.table).cuda(), torch.from_numpy(c.lens).cuda()


def queries(batch, tokens, q_heads, D, seed) -> np.ndarray:
    rng = np.random.Generator(np.random.PCG64(seed))
    return bf16_bits(rng.standard_normal((batch, tokens, q_heads, D)) * 1.5)
