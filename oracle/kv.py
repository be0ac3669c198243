"""CPU oracle of the paged, quantised key-value cache (test infrastructure).

The cache's bytes follow the layout that include/aq.h states; a cached row is quantised and dequantised by the C
oracle's weight quantizer, so a row of K or V means exactly what a weight row means.  Everything else is NumPy, one
row at a time, and attention is summed in 64 bits.
"""
from __future__ import annotations

import numpy as np

import oracle


def token_bytes(D: int, G: int, bits: int) -> int:
    return 2 * (D * bits // 8) + 8 * (D // G)


class Cache:
    """Bytes uint8 [pages, heads, page_size, token_bytes] with the sequences' table [batch, width] and lens [batch]."""

    def __init__(self, data, table, lens, D, G, bits):
        self.data, self.table, self.lens = data, table, lens
        self.D, self.G, self.bits = D, G, bits
        self.pages, self.heads = data.shape[:2]
        self.page_size = data.shape[2]
        self.row = D * bits // 8
        self.ng = D // G

    def locate(self, seq: int, pos: int):
        """(page, byte offset of the tile in the page, row in the tile), or None where the position is absent."""
        i = pos // self.page_size
        if pos < 0 or i >= self.table.shape[1] or not 0 <= self.table[seq, i] < self.pages:
            return None
        in_page = pos % self.page_size
        return int(self.table[seq, i]), in_page // 16 * 16 * token_bytes(self.D, self.G, self.bits), in_page % 16

    def spans(self, tile: int, row: int, which: int):
        """Byte ranges of a row's codes and of its (scale, bias) pairs; which: 0 for K, 1 for V."""
        codes = tile + (16 * which + row) * self.row
        pairs = tile + 32 * self.row + (2 * row + which) * 4 * self.ng
        return slice(codes, codes + self.row), slice(pairs, pairs + 4 * self.ng)

    def stored(self, seq: int, pos: int, head: int, which: int):
        """(packed uint32 [1, words], scales [1, ng], biases [1, ng]) of a cached row, or None."""
        at = self.locate(seq, pos)
        if at is None:
            return None
        codes, pairs = self.spans(at[1], at[2], which)
        page = self.data[at[0], head].reshape(-1)
        sb = page[pairs].copy().view(np.uint16).reshape(1, self.ng, 2)
        return page[codes].copy().view(np.uint32)[None], np.ascontiguousarray(sb[..., 0]), np.ascontiguousarray(sb[..., 1])


def rows_of(lens, rows, offsets):
    """For each row: (sequence, position), or None where no sequence has it."""
    if offsets is None:
        n = rows // len(lens)
        offsets = [n * b for b in range(len(lens) + 1)]
    found = [None] * rows
    for b, length in enumerate(lens):
        for r in range(max(0, int(offsets[b])), min(rows, int(offsets[b + 1]))):
            found[r] = (b, int(length) - int(offsets[b + 1]) + r)
    return found


def f32(bf16_bits: np.ndarray) -> np.ndarray:
    return (bf16_bits.astype(np.uint32) << 16).view(np.float32)


def append(c: Cache, k_bits, v_bits, offsets=None) -> None:
    """k_bits, v_bits: bf16 patterns uint16 [rows, heads, D]."""
    for r, at in enumerate(rows_of(c.lens, len(k_bits), offsets)):
        place = c.locate(*at) if at else None
        if place is None:
            continue
        for which, x in enumerate((k_bits, v_bits)):
            packed, scales, biases = oracle.quantize(f32(x[r]), c.G, c.bits)
            for h in range(c.heads):
                codes, pairs = c.spans(place[1], place[2], which)
                page = c.data[place[0], h].reshape(-1)  # (a view: the cache is contiguous)
                page[codes] = packed[h].view(np.uint8)
                page[pairs] = np.stack((scales[h], biases[h]), -1).reshape(-1).view(np.uint8)


def read(c: Cache, rows: int, offsets=None, out=None):
    """-> (k, v) bf16 patterns [rows, heads, D]; rows of no sequence as in `out` (zeros without one)."""
    k, v = out if out is not None else (np.zeros((rows, c.heads, c.D), np.uint16) for _ in range(2))
    for r, at in enumerate(rows_of(c.lens, rows, offsets)):
        if at is None:
            continue
        for which, x in enumerate((k, v)):
            for h in range(c.heads):
                s = c.stored(*at, h, which)
                x[r, h] = 0 if s is None else oracle.dequantize_bf16(*s, c.D, c.G, c.bits)[0]
    return k, v


def _fields(c: Cache, seq: int, pos: int, head: int, which: int):
    """(codes [D], scales [D], biases [D]) in 64 bits."""
    packed, s, b = c.stored(seq, pos, head, which)
    q = ((packed[0][:, None] >> np.arange(0, 32, c.bits, dtype=np.uint32)) & (2**c.bits - 1)).reshape(-1)
    wide = lambda x: np.repeat(x[0].view(np.float16).astype(np.float64), c.G)  # noqa: E731
    return q.astype(np.float64), wide(s), wide(b)


def attention(c: Cache, q_bits, scale: float, window: int = 0):
    """q_bits: bf16 patterns [batch, tokens, q_heads, D] -> a dict of 64-bit arrays:

    out [.., D] and lse [..], the attention; and for bounds of rounding errors
    spread [.., D] = sum_t w_t |scale_t| code_td, size [.., D] = sum_t w_t |v_td| (w: the softmax weights),
    terms [..] = max_t |scale| sum_d |q_d| (|scale_t| code_td + |bias_t|), the size of what a score is summed from, and
    least [..] = n max |scale_t| max code over V of the n positions that any of the sequence's tokens sees."""
    q = f32(q_bits).astype(np.float64)
    B, n, hq, D = q.shape
    out, spread, size = np.zeros(q.shape), np.zeros(q.shape), np.zeros(q.shape)
    lse, terms, least = np.full(q.shape[:3], -np.inf), np.zeros(q.shape[:3]), np.zeros(q.shape[:3])
    rep = hq // c.heads
    for b in range(B):
        length = int(c.lens[b])
        first = max(0, length - n + 1 - window) if window else 0
        known = [p for p in range(first, length) if c.locate(b, p) is not None]
        for h in range(c.heads):
            if not known:
                continue
            k, v = ([np.stack(x) for x in zip(*(_fields(c, b, p, h, which) for p in known))] for which in (0, 1))
            kx, vx = k[0] * k[1] + k[2], v[0] * v[1] + v[2]
            least[b, :, h * rep:(h + 1) * rep] = len(known) * max(np.abs(v[1]).max(), 2.0**-15) * (2**c.bits - 1)
            pos = np.array(known)
            for j in range(n):
                p = length - n + j
                see = (pos <= p) & (pos > p - window if window else True)
                if not see.any():
                    continue
                for i in range(h * rep, (h + 1) * rep):
                    x = scale * (kx[see] @ q[b, j, i])
                    m = x.max()
                    w = np.exp(x - m)
                    lse[b, j, i] = m + np.log(w.sum())
                    w /= w.sum()
                    out[b, j, i] = w @ vx[see]
                    spread[b, j, i] = w @ (v[0] * np.abs(v[1]))[see]
                    size[b, j, i] = w @ np.abs(vx[see])
                    terms[b, j, i] = abs(scale) * ((k[0] * np.abs(k[1]) + np.abs(k[2]))[see] @ np.abs(q[b, j, i])).max()
    return dict(out=out, lse=lse, spread=spread, size=size, terms=terms, least=least)


def attention_bounds(r: dict, D: int):
    """What aq_kv_attention may be off by: (out, lse), from its arithmetic as include/aq.h states it.

    A score is a sum of D products (and of the groups' biases) in fp32, each step off by at most one unit 2^-23 of the
    sum's size; with the factor, the maximum's subtraction and exp2 that makes an absolute error of at most
    e = (D + 16) 2^-23 terms + 2^-21, so a weight is off by a factor of 1 +- 2e (its own and the sum's).  A weight's product
    with a V scale rounds to fp16 (2^-11), the sums over tokens are in fp32 (2^-23 for each of the at most 2^11 joined
    partial sums and accumulations that follow one another: 2^-12), and the result rounds to bf16 (2^-8).

    Where the rounded product is subnormal its error is absolute instead, half a unit, 2^-25.  It stands for
    2^(x - M + 13 - e) s, M at most the row's maximum and 2^e at most twice the largest magnitude s of a V scale (or 2^-14), and the
    result is divided by the sum of 2^(x - M + 13 - e), which is at least 2^(13 - e).  So a token's code adds an error of at most
    2^-25 2^(e - 13) code = 2^-38 2^e code <= 2^-37 max(s, 2^-15) code, and n tokens at most 2^-37 least."""
    e = ((D + 16) * 2.0**-23 * r["terms"] + 2.0**-21)[..., None]
    off = (2.0**-11 + 2.0**-12) * r["spread"] + (2 * e + 2.0**-12) * r["size"] + 2.0**-37 * r["least"][..., None]
    with np.errstate(invalid="ignore"):
        lse = e[..., 0] + 2.0**-21 * (np.where(np.isfinite(r["lse"]), np.abs(r["lse"]), 0.0) + 1.0)
    return 2.0**-8 * np.abs(r["out"]) + (1 + 2.0**-8) * off + 2.0**-133, lse
