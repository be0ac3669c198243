"""The key-value cache's oracle against closed forms and an independent statement; the library's host-side checks.

No GPU: every library call here is refused by argument validation, or has nothing to do."""
import ctypes

import numpy as np
import pytest

import oracle
import weight_only_group_b200 as aq
from kv_cases import bf16_bits, cache, filled, queries, rows
from oracle import kv as ref

FORMS = [(64, 32, 4), (64, 64, 8), (128, 64, 4), (128, 128, 8), (256, 32, 8), (256, 128, 4)]


@pytest.mark.parametrize("D,G,bits", FORMS)
def test_token_bytes(D, G, bits):
    # codes of K and V, and a 2-byte scale and a 2-byte bias for each group of each
    assert ref.token_bytes(D, G, bits) == (2 * D * bits + 2 * (D // G) * 32) // 8 == aq.aq_kv_token_bytes(D, G, bits)


def test_token_bytes_of_the_common_form_is_the_weights_ratio():
    # 4 bits, G = 64: 4.5 bits a value, as for weights
    assert aq.aq_kv_token_bytes(128, 64, 4) * 8 == 4.5 * 256


@pytest.mark.parametrize("D,G,bits", [(128, 64, 3), (128, 64, 2), (96, 32, 4), (64, 128, 4), (128, 16, 4), (0, 64, 4), (-128, 64, 4)])
def test_unsupported_forms(D, G, bits):
    assert aq.aq_kv_token_bytes(D, G, bits) == 0


@pytest.mark.parametrize("D,G,bits", FORMS)
def test_append_then_read_is_quantize_then_dequantize(D, G, bits):
    lens = [5, 0, 37]
    c = cache(lens, heads=3, page_size=16, D=D, G=G, bits=bits, seed=1)
    before = c.data.copy()
    k, v = rows(42, 3, D, 2), rows(42, 3, D, 3)
    offsets = [0, 5, 5, 42]
    ref.append(c, k, v, offsets)
    for x, y in zip((k, v), ref.read(c, 42, offsets)):
        w = ref.f32(x).reshape(-1, D)
        assert np.array_equal(y.reshape(-1, D), oracle.dequantize_bf16(*oracle.quantize(w, G, bits), D, G, bits))
    # 42 tokens of 3 heads at most were changed, and no byte of another page
    used = {int(c.table[b, p]) for b, n in enumerate(lens) for p in range(-(-n // 16))}
    other = [p for p in range(c.pages) if p not in used]
    assert np.array_equal(before[other], c.data[other])
    changed = (before != c.data).sum()
    assert 0 < changed <= 42 * 3 * ref.token_bytes(D, G, bits)


def test_layout_by_hand():
    """Token 17 of a sequence, in row 1 of the second tile of its page: the bytes, worked out from the layout."""
    D, G, bits = 64, 64, 4
    c = ref.Cache(np.zeros((2, 1, 32, ref.token_bytes(D, G, bits)), np.uint8), np.array([[1]], np.int32),
                  np.array([18], np.int32), D, G, bits)
    x = np.zeros((1, 1, D))
    x[0, 0, :16] = np.arange(16)  # min 0, max 15: scale 1, bias 0, and the codes are the values
    k = bf16_bits(x)
    ref.append(c, k, bf16_bits(x + 2), offsets=[0, 1])  # V: scale 1, bias 2
    page, tile = c.data[1, 0].reshape(-1), 16 * ref.token_bytes(D, G, bits)
    assert tile == 16 * (32 + 32 + 8)
    low = [0x10, 0x32, 0x54, 0x76, 0x98, 0xBA, 0xDC, 0xFE] + [0] * 24
    assert page[tile + 32:tile + 64].tolist() == low                  # K, row 1
    assert page[tile + 16 * 32 + 32:tile + 16 * 32 + 64].tolist() == low  # V, row 1
    pairs = page[tile + 1024 + 8:tile + 1024 + 16].copy().view(np.float16)
    assert pairs.tolist() == [1.0, 0.0, 1.0, 2.0]
    assert np.count_nonzero(c.data) == np.count_nonzero(page[tile:tile + 16 * 72])


def test_rows_of_short_and_absent_sequences():
    # 4 rows each: of a sequence of 2 the first two rows have no position; row 12 belongs to no sequence
    assert ref.rows_of([2, 0, 9], 12, None)[:5] == [(0, -2), (0, -1), (0, 0), (0, 1), (1, -4)]
    assert ref.rows_of([2, 0, 9], 13, [0, 2, 2, 11])[10:] == [(2, 8), None, None]


@pytest.mark.parametrize("window", (0, 5, 100))
def test_attention_against_a_direct_softmax(window):
    D, G, bits, n = 64, 32, 4, 3
    lens = [40, 2, 0]
    c = filled(lens, heads=2, page_size=16, D=D, G=G, bits=bits, seed=5)
    q = queries(3, n, 4, D, 6)
    r = ref.attention(c, q, 0.125, window)
    for b, length in enumerate(lens):
        if length:
            k, v = (ref.f32(x).astype(np.float64) for x in ref.read(c, length, [0] * (b + 1) + [length] * (3 - b)))
        for j in range(n):
            at = length - n + j
            lo = max(0, at - window + 1) if window else 0
            for i in range(4):
                if at < 0:
                    assert not r["out"][b, j, i].any() and r["lse"][b, j, i] == -np.inf
                    continue
                x = 0.125 * k[lo:at + 1, i // 2] @ ref.f32(q[b, j, i]).astype(np.float64)
                w = np.exp(x)
                # (what is read back is rounded to bf16: half a unit, 2^-9, of each term)
                assert np.allclose(r["out"][b, j, i], w @ v[lo:at + 1, i // 2] / w.sum(), rtol=0.1, atol=0.05)
                assert abs(r["lse"][b, j, i] - np.log(w.sum())) < 0.1


def test_attention_of_equal_scores_is_the_mean():
    c = filled([23], heads=1, page_size=16, D=64, G=64, bits=8, seed=9)
    r = ref.attention(c, np.zeros((1, 1, 2, 64), np.uint16), 1.0)
    v = np.stack([f[0] * f[1] + f[2] for f in (ref._fields(c, 0, p, 0, 1) for p in range(23))])
    assert np.allclose(r["out"][0, 0, 1], v.mean(0), rtol=1e-12)
    assert np.allclose(r["lse"], np.log(23))


# ------------------------------------------------------------------------------ the library's own checks

A, U = 0x10000, 0x10004  # addresses that nothing reads: every call below is refused, or has nothing to do


def _desc(**kw):
    d = dict(data=A, pages=4, heads=2, page_size=16, D=128, G=64, bits=4, table=A, lens=A, batch=2, width=2) | kw
    return aq._KVCache(*d.values())


def _append(c, k=A, v=A, rows=2, offsets=None, s=(256, 128, 256, 128)):
    return aq.lib().aq_kv_append(c, k, s[0], s[1], v, s[2], s[3], rows, offsets, None)


def _read(c, k=A, v=A, rows=2, offsets=None):
    return aq.lib().aq_kv_read(c, rows, offsets, k, v, None)


def _attend(c, q=A, tokens=1, q_heads=8, s=(1024, 1024, 128), scale=0.1, window=0, out=A, lse=None, ws=A, wb=1 << 40):
    return aq.lib().aq_kv_attention(c, q, tokens, q_heads, *s, scale, window, out, lse, ws, wb, None)


@pytest.mark.parametrize("call", (_append, _read, _attend))
def test_cache_validation(call):
    bad, unsupported, alignment = aq.AQ_ERR_INVALID_ARG, aq.AQ_ERR_UNSUPPORTED, aq.AQ_ERR_ALIGNMENT
    for kw in (dict(bits=2), dict(bits=3), dict(D=96), dict(D=512), dict(G=16), dict(D=64, G=128), dict(page_size=8),
               dict(page_size=48), dict(page_size=2048), dict(page_size=0), dict(page_size=-16)):
        assert call(_desc(**kw)) == unsupported, kw
    for kw in (dict(pages=0), dict(pages=1 << 31), dict(heads=0), dict(heads=1 << 16), dict(data=None), dict(batch=-1),
               dict(table=None), dict(lens=None), dict(width=0), dict(width=1 << 27)):
        assert call(_desc(**kw)) == bad, kw
    for kw in (dict(data=U), dict(table=A + 2), dict(lens=A + 1)):
        assert call(_desc(**kw)) == alignment, kw
    assert call(None) == bad
    # no sequences: nothing to do, whatever the table
    assert call(_desc(batch=0, table=None, lens=None, width=0)) == aq.AQ_OK


def test_append_and_read_validation():
    c = _desc()
    for call in (_append, _read):
        assert call(c, k=None) == aq.AQ_ERR_INVALID_ARG
        assert call(c, v=None) == aq.AQ_ERR_INVALID_ARG
        assert call(c, rows=-1) == aq.AQ_ERR_INVALID_ARG
        assert call(c, rows=3) == aq.AQ_ERR_INVALID_ARG  # two sequences, no offsets
        assert call(c, rows=1 << 40, offsets=A) == aq.AQ_ERR_INVALID_ARG
        assert call(c, k=U) == aq.AQ_ERR_ALIGNMENT
        assert call(c, v=U) == aq.AQ_ERR_ALIGNMENT
        assert call(c, offsets=A + 2) == aq.AQ_ERR_ALIGNMENT
        assert call(c, rows=0) == aq.AQ_OK
    for i in range(4):
        s = [256, 128, 256, 128]
        s[i] += 4
        assert _append(c, s=s) == aq.AQ_ERR_ALIGNMENT


def test_attention_validation():
    c = _desc()
    bad = aq.AQ_ERR_INVALID_ARG
    for kw in (dict(q=None), dict(out=None), dict(tokens=0), dict(tokens=-1), dict(q_heads=0), dict(q_heads=7),
               dict(window=-1), dict(scale=float("inf")), dict(scale=float("nan"))):
        assert _attend(c, **kw) == bad, kw
    for kw in (dict(q=U), dict(out=U), dict(lse=A + 2), dict(ws=U), dict(s=(1028, 1024, 128)), dict(s=(1024, 1028, 128)),
               dict(s=(1024, 1024, 132))):
        assert _attend(c, **kw) == aq.AQ_ERR_ALIGNMENT, kw
    # more units of work than are counted in 32 bits
    assert _attend(_desc(batch=1 << 24, width=1 << 20)) == aq.AQ_ERR_UNSUPPORTED
    need = aq.lib().aq_kv_attention_workspace_bytes(c, 1, 8, 0)
    if need:
        assert _attend(c, wb=need - 1) == bad
        assert _attend(c, ws=None) == bad
    assert aq.lib().aq_kv_attention_workspace_bytes(_desc(bits=3), 1, 8, 0) == 0
    assert aq.lib().aq_kv_attention_workspace_bytes(c, 1, 7, 0) == 0


def test_descriptor_matches_the_header():
    # pointer, 2 x int64, 4 x int32, 2 pointers, 2 x int64
    assert ctypes.sizeof(aq._KVCache) == 8 + 16 + 16 + 16 + 16
