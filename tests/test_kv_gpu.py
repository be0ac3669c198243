"""The quantised key-value cache on the GPU against the 64-bit oracle: bytes and read-back values bit for bit, attention
within the bounds that follow from its arithmetic (oracle/kv.py, attention_bounds)."""
import itertools

import numpy as np
import pytest
import torch

from kv_cases import bf16_bits, bits_of, cache, filled, on_gpu, queries, rows, to_gpu
from oracle import kv as ref

pytestmark = pytest.mark.gpu

aq = pytest.importorskip("weight_only_group_b200")


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    aq.lib()


@pytest.fixture(autouse=True)
def _no_fault():
    yield
    assert aq.aq_device_fault() == 0


def _gpu(offsets):
    return None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device="cuda")


FORMS = [(D, G, bits) for D, G, bits in itertools.product((64, 128, 256), (32, 64, 128), (4, 8)) if G <= D]


# ------------------------------------------------------------------------------ write and read

@pytest.mark.parametrize("D,G,bits", FORMS)
@pytest.mark.parametrize("lens,offsets,page,heads", [
    ([1], None, 16, 1),
    ([40, 3, 17], None, 16, 3),                       # one token each
    ([40, 0, 17], None, 32, 2),                       # a padded batch: the second slot is empty
    ([33, 0, 64, 5], [0, 33, 33, 43, 48], 16, 2),     # whole, empty, a tail across tiles, whole
    ([100], [0, 100], 64, 5),
])
def test_append_and_read(D, G, bits, lens, offsets, page, heads):
    c = cache(lens, heads=heads, page_size=page, D=D, G=G, bits=bits, seed=11)
    n = offsets[-1] if offsets else len(lens)
    k, v = rows(n, heads, D, 12), rows(n, heads, D, 13)
    data, table, ln = on_gpu(c)
    aq.aq_kv_append(data, to_gpu(k), to_gpu(v), table, ln, G, bits, offsets=_gpu(offsets))
    ref.append(c, k, v, offsets)
    assert np.array_equal(data.cpu().numpy(), c.data)  # untouched bytes too
    got = aq.aq_kv_read(data, table, ln, n, D, G, bits, offsets=_gpu(offsets))
    for x, y in zip(got, ref.read(c, n, offsets)):
        assert np.array_equal(bits_of(x), y)


def test_append_from_a_fused_projection():
    """k and v as a layer's projection gives them: slices of one buffer, rows and heads apart."""
    D, G, bits, H, Hq = 128, 64, 4, 4, 12
    c = cache([9, 30], heads=H, page_size=16, D=D, G=G, bits=bits, seed=3)
    qkv = torch.randn(7, (Hq + 2 * H) * D, device="cuda").bfloat16()
    k = qkv[:, Hq * D:(Hq + H) * D].view(7, H, D)
    v = qkv[:, (Hq + H) * D:].view(7, H, D)
    data, table, ln = on_gpu(c)
    offsets = [0, 2, 7]
    aq.aq_kv_append(data, k, v, table, ln, G, bits, offsets=_gpu(offsets))
    ref.append(c, bits_of(k), bits_of(v), offsets)
    assert np.array_equal(data.cpu().numpy(), c.data)
    # heads before rows
    kt, vt = (x.transpose(0, 1).contiguous().transpose(0, 1) for x in (k, v))
    again = on_gpu(c)[0]
    again.random_(0, 256)
    first = again.clone()
    aq.aq_kv_append(again, kt, vt, table, ln, G, bits, offsets=_gpu(offsets))
    aq.aq_kv_append(first, k, v, table, ln, G, bits, offsets=_gpu(offsets))
    assert torch.equal(again, first)


@pytest.mark.parametrize("bits", (4, 8))
def test_rows_that_begin_on_16_bytes(bits):
    """k, v and the outputs of a read on 16 bytes but not on 32, and rows an odd number of 16 bytes apart."""
    D, G, H, n = 128, 32, 3, 11
    c = cache([20], heads=H, page_size=16, D=D, G=G, bits=bits, seed=6)
    data, table, ln = on_gpu(c)
    flat = torch.randn(2 * n * (H * D + 8) + 8, device="cuda").bfloat16()[8:]
    k, v = flat.view(2, n, H * D + 8)[:, :, :H * D].unflatten(2, (H, D))
    assert k.data_ptr() % 32 == 16
    aq.aq_kv_append(data, k, v, table, ln, G, bits, offsets=_gpu([0, n]))
    ref.append(c, bits_of(k), bits_of(v), [0, n])
    assert np.array_equal(data.cpu().numpy(), c.data)
    room = torch.zeros(2, n * H * D + 8, dtype=torch.bfloat16, device="cuda")
    out = tuple(x[8:].view(n, H, D) for x in room)
    aq.aq_kv_read(data, table, ln, n, D, G, bits, offsets=_gpu([0, n]), out=out)
    for x, y in zip(out, ref.read(c, n, [0, n])):
        assert np.array_equal(bits_of(x), y)
    assert not room[:, :8].any()


def test_rows_of_no_sequence_stay():
    """Offsets that begin behind row 0 and end before the last: the rows around them are nobody's."""
    D, G, bits = 64, 64, 8
    c = filled([10, 4], heads=2, page_size=16, D=D, G=G, bits=bits, seed=4)
    data, table, ln = on_gpu(c)
    out = tuple(torch.full((20, 2, D), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    offsets = [3, 13, 17]
    aq.aq_kv_read(data, table, ln, 20, D, G, bits, offsets=_gpu(offsets), out=out)
    seven = np.full((20, 2, D), int(bf16_bits(np.array([7.0]))[0]), np.uint16)
    for x, y in zip(out, ref.read(c, 20, offsets, (seven.copy(), seven.copy()))):
        assert np.array_equal(bits_of(x), y)
        assert (bits_of(x)[[0, 1, 2, 17, 18, 19]] == seven[0]).all()
    k, v = rows(20, 2, D, 5), rows(20, 2, D, 6)
    aq.aq_kv_append(data, to_gpu(k), to_gpu(v), table, ln, G, bits, offsets=_gpu(offsets))
    ref.append(c, k, v, offsets)
    assert np.array_equal(data.cpu().numpy(), c.data)


def test_more_rows_than_positions():
    """A sequence given more rows than its length: the first of them have no position."""
    D, G, bits = 128, 32, 4
    c = filled([3, 20], heads=1, page_size=16, D=D, G=G, bits=bits, seed=8)
    data, table, ln = on_gpu(c)
    k, v = rows(12, 1, D, 9), rows(12, 1, D, 10)
    aq.aq_kv_append(data, to_gpu(k), to_gpu(v), table, ln, G, bits)  # 6 rows each
    ref.append(c, k, v)
    assert np.array_equal(data.cpu().numpy(), c.data)
    got = aq.aq_kv_read(data, table, ln, 12, D, G, bits)
    for x, y in zip(got, ref.read(c, 12)):
        assert np.array_equal(bits_of(x), y)
        assert not bits_of(x)[:3].any()


def test_extreme_rows():
    """Ties of the rounding, subnormal scales, fp16's largest values, one value against zeros, signed zeros."""
    D, G = 64, 32
    x = np.zeros((8, 1, D))
    x[0] = np.arange(D) % 32 / 2
    x[1] = np.where(np.arange(D) % 2, 1e-7, -1e-7)
    x[2] = np.where(np.arange(D) % 3, 65280.0, -65280.0) / 2
    x[3, 0, 5] = 3.0
    x[4] = np.where(np.arange(D) % 2, 0.0, -0.0)
    x[5] = -np.arange(D) * 2.0**-20
    x[6] = 1e-30
    x[7] = np.linspace(-7.5, 7.5, D)
    for bits in (4, 8):
        c = cache([8], heads=1, page_size=16, D=D, G=G, bits=bits, seed=2)
        data, table, ln = on_gpu(c)
        k = bf16_bits(x)
        aq.aq_kv_append(data, to_gpu(k), to_gpu(k[::-1]), table, ln, G, bits, offsets=_gpu([0, 8]))
        ref.append(c, k, k[::-1], [0, 8])
        assert np.array_equal(data.cpu().numpy(), c.data)


@pytest.mark.parametrize("bits", (4, 8))
def test_quotients_at_and_beside_ties(bits):
    """Inputs of few bits on every scale: quotients that lie on the middle between two codes, or an ulp of it away."""
    D, G, n = 256, 32, 600
    rng = np.random.default_rng(bits)
    step = 2.0 ** rng.integers(-9, 4, (n, 1, D // G, 1))
    x = rng.integers(-255, 256, (n, 1, D // G, G)) * step
    x[::3] += rng.integers(-128, 129, (len(x[::3]), 1, D // G, 1)) * 2.0 ** rng.integers(-12, 3, (len(x[::3]), 1, D // G, 1))
    k = bf16_bits(x.reshape(n, 1, D))
    c = cache([n], heads=1, page_size=128, D=D, G=G, bits=bits, seed=3)
    data, table, ln = on_gpu(c)
    aq.aq_kv_append(data, to_gpu(k), to_gpu(k[::-1]), table, ln, G, bits, offsets=_gpu([0, n]))
    ref.append(c, k, k[::-1], [0, n])
    assert np.array_equal(data.cpu().numpy(), c.data)


# ------------------------------------------------------------------------------ attention

def _check(c, q, got, lse=None, scale=None, window=0):
    D = q.shape[-1]
    scale = D**-0.5 if scale is None else scale
    r = ref.attention(c, q, scale, window)
    far, far_lse = ref.attention_bounds(r, D)
    x = got.float().cpu().numpy().astype(np.float64).reshape(q.shape)
    assert np.isfinite(x).all()
    off = np.abs(x - r["out"]) / far
    assert off.max() <= 1, f"{off.max():.2f} times the bound at {np.unravel_index(off.argmax(), off.shape)}"
    if lse is not None:
        y = lse.cpu().numpy().astype(np.float64).reshape(r["lse"].shape)
        none = np.isneginf(r["lse"])
        assert np.array_equal(np.isneginf(y), none)
        assert (np.abs(y[~none] - r["lse"][~none]) <= far_lse[~none]).all()
    return r


def _attend(c, q, gpu=None, **kw):
    data, table, ln = gpu or on_gpu(c)
    lse = torch.full(q.shape[:3], 5.0, device="cuda")
    out = aq.aq_kv_attention(to_gpu(q), data, table, ln, c.G, c.bits, lse=lse, **kw)
    _check(c, q, out, lse, kw.get("scale"), kw.get("window", 0))
    return out, lse


@pytest.mark.parametrize("D,G,bits", FORMS)
@pytest.mark.parametrize("lens,page,heads,q_heads,tokens", [
    ([1], 16, 1, 1, 1),
    ([0, 47, 16, 17], 16, 2, 8, 1),
    ([33, 300, 31, 32, 15], 32, 1, 7, 1),
    ([70, 2], 64, 3, 3, 4),
    ([190], 128, 1, 16, 2),
])
def test_attention(D, G, bits, lens, page, heads, q_heads, tokens):
    c = filled(lens, heads=heads, page_size=page, D=D, G=G, bits=bits, seed=sum(lens) + D)
    _attend(c, queries(len(lens), tokens, q_heads, D, 21))


@pytest.mark.parametrize("tokens,q_heads,heads", [(1, 8, 1), (1, 9, 1), (1, 16, 1), (1, 17, 1), (3, 12, 2), (6, 8, 1), (5, 64, 2)])
def test_attention_head_groups(tokens, q_heads, heads):
    """Rows of a KV head below, at and above the widths of the matrix instructions' tiles."""
    c = filled([61, 4, 130], heads=heads, page_size=16, D=128, G=64, bits=4, seed=31)
    _attend(c, queries(3, tokens, q_heads, 128, 32))


@pytest.mark.parametrize("length", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 255, 256, 257, 513])
@pytest.mark.parametrize("bits", (4, 8))
def test_attention_lengths(length, bits):
    c = filled([length], heads=1, page_size=16, D=64, G=32, bits=bits, seed=length)
    _attend(c, queries(1, 2, 4, 64, length + 1))


@pytest.mark.parametrize("window", (1, 2, 15, 16, 17, 33, 100, 1 << 40))
@pytest.mark.parametrize("tokens", (1, 3))
def test_attention_window(window, tokens):
    c = filled([150, 1, 90, 16, 0], heads=2, page_size=32, D=128, G=64, bits=4, seed=41)
    _attend(c, queries(5, tokens, 8, 128, 42), window=window)


def test_attention_window_far_from_the_start():
    """Pages before the window are not needed: their entries may hold anything, and set no fault."""
    c = filled([1000, 700], heads=1, page_size=16, D=64, G=64, bits=8, seed=43)
    c.table[:, :30] = 1 << 30
    _attend(c, queries(2, 2, 2, 64, 44), window=200)


@pytest.mark.parametrize("bits", (4, 8))
@pytest.mark.parametrize("bad", (0x7C00, 0xFC00, 0x7E01))
def test_attention_beside_tokens_that_are_not_finite(bits, bad):
    """A drafted token whose scales and biases are infinite or NaN, and one in front of the window: rows that do not see
    them are as they would be without."""
    D, G, n, window = 64, 32, 4, 25
    c = filled([60, 35], heads=1, page_size=16, D=D, G=G, bits=bits, seed=45)
    q = queries(2, n, 6, D, 46)
    good = on_gpu(c)
    r = ref.attention(c, q, 0.125, window)
    for b, length in enumerate(c.lens.tolist()):
        # the last token is seen by the last row alone; the one at length - n + 1 - window + 1 by rows 0 and 1 alone
        for pos in (length - 1, length - n + 2 - window):
            page, tile, row = c.locate(b, pos)
            flat = c.data[page, 0].reshape(-1)
            for which in (0, 1):
                flat[c.spans(tile, row, which)[1]] = np.full(2 * c.ng, bad, np.uint16).view(np.uint8)
    data, table, ln = on_gpu(c)
    for gpu, rows_ok in (((data, table, ln), [2]), (good, [0, 1, 2, 3])):
        x = aq.aq_kv_attention(to_gpu(q), *gpu, G, bits, scale=0.125, window=window).float().cpu().numpy().astype(np.float64)
        far, _ = ref.attention_bounds(r, D)
        assert (np.abs(x - r["out"]) <= far)[:, rows_ok].all()


@pytest.mark.parametrize("scale", (0.0, -0.125, 3.0, 1e-6))
def test_attention_scales(scale):
    c = filled([77, 30], heads=2, page_size=16, D=64, G=32, bits=8, seed=51)
    _attend(c, queries(2, 1, 6, 64, 52), scale=scale)


@pytest.mark.parametrize("tokens,q_heads", [(1, 3), (2, 6)])
@pytest.mark.parametrize("bad", (float("nan"), float("inf"), -float("inf")))
def test_attention_beside_a_query_that_is_not_finite(tokens, q_heads, bad):
    c = filled([50, 9], heads=1, page_size=16, D=64, G=32, bits=4, seed=53)
    gpu, q = on_gpu(c), to_gpu(queries(2, tokens, q_heads, 64, 54))
    want = aq.aq_kv_attention(q, *gpu, 32, 4)
    q[0, 0, 1, 7] = bad
    got = aq.aq_kv_attention(q, *gpu, 32, 4)
    assert not torch.isfinite(got[0, 0, 1]).all()
    want[0, 0, 1] = got[0, 0, 1] = 0
    assert torch.equal(got, want)


def test_attention_of_queries_of_extreme_sizes():
    """Queries of 2^-120 to 2^90 against keys that bring the scores back to where a softmax is neither flat nor sharp."""
    D, G, bits = 64, 32, 8
    rng = np.random.default_rng(8)
    q, sizes = rng.standard_normal((1, 1, 6, D)), 2.0 ** np.array([-120, -60, -14, 0, 12, 14])
    c = cache([70], heads=6, page_size=16, D=D, G=G, bits=bits, seed=55)
    k = rng.standard_normal((70, 6, D)) / np.clip(sizes, 2.0**-13, None)[None, :, None]
    ref.append(c, bf16_bits(k), rows(70, 6, D, 56), [0, 70])
    _attend(c, bf16_bits(q * sizes[None, None, :, None]))


def test_attention_of_many_tokens():
    """As many new tokens as a short prompt has: a triangle of masks."""
    c = filled([130, 90, 7], heads=1, page_size=32, D=64, G=64, bits=4, seed=57)
    _attend(c, queries(3, 90, 2, 64, 58))
    _attend(c, queries(3, 90, 2, 64, 59), window=20)


def test_attention_sharp_and_flat():
    """Scores far apart, the largest of them first, last and in between; q of very different sizes, and zero."""
    lens = [400, 400, 400, 400]
    D, G, bits = 128, 64, 4
    c = cache(lens, heads=1, page_size=16, D=D, G=G, bits=bits, seed=61)
    k, v = np.zeros((1600, 1, D)), np.random.default_rng(0).standard_normal((1600, 1, D))
    k[:, 0] = np.random.default_rng(1).standard_normal((1600, D))
    for i, at in enumerate((0, 399, 200, 17)):
        k[400 * i + at] *= 9
    kb = bf16_bits(k)
    ref.append(c, kb, bf16_bits(v), [0, 400, 800, 1200, 1600])
    q = np.zeros((4, 1, 4, D))
    for i, at in enumerate((0, 399, 200, 17)):
        d = ref.f32(kb[400 * i + at, 0])
        for j, size in enumerate((1.0, 1e-3, 30.0, 0.0)):
            q[i, 0, j] = d * size
    q[2, 0, 1, ::2] *= 1e-6
    _attend(c, bf16_bits(q))


def test_attention_scales_of_v_far_apart():
    """Tokens whose values differ by a factor of 2^20, the large ones late, early, and of no weight."""
    D, G, bits = 64, 32, 8
    rng = np.random.default_rng(3)
    k, v = rng.standard_normal((600, 1, D)), rng.standard_normal((600, 1, D))
    v[150] *= 2.0**14
    v[200:] *= 2.0**-6
    v[599] *= 2.0**8
    k[320] = -8.0
    v[320] *= 2.0**12
    c = cache([200, 400], heads=1, page_size=16, D=D, G=G, bits=bits, seed=5)
    ref.append(c, bf16_bits(k), bf16_bits(v), [0, 200, 600])
    _attend(c, np.concatenate((queries(2, 1, 3, D, 7), bf16_bits(np.full((2, 1, 1, D), 1.0))), 2))


def test_attention_constant_values():
    """Groups of one value have scale 0: all of them lies in the bias."""
    D, G, bits = 64, 64, 4
    c = cache([90], heads=1, page_size=16, D=D, G=G, bits=bits, seed=71)
    k = np.random.default_rng(2).standard_normal((90, 1, D))
    ref.append(c, bf16_bits(k), bf16_bits(np.full((90, 1, D), -2.5)), [0, 90])
    out, _ = _attend(c, queries(1, 1, 2, D, 72))
    assert (out == -2.5).all()


def test_attention_long():
    """A length that is split over the whole GPU, and short ones beside it."""
    lens = [20011, 3, 700]
    D, G, bits = 64, 64, 4
    rng = np.random.Generator(np.random.PCG64(81))
    c = cache(lens, heads=1, page_size=64, D=D, G=G, bits=bits, seed=81)
    # codes stay random bytes; scales and biases of a plausible size
    tiles = c.data.reshape(c.pages, 1, 4, 16 * ref.token_bytes(D, G, bits))
    meta = np.stack((rng.uniform(0.05, 0.4, (c.pages, 1, 4, 32)), rng.uniform(-3, 0, (c.pages, 1, 4, 32))), -1)
    tiles[..., 1024:] = meta.astype(np.float16).reshape(c.pages, 1, 4, 64).view(np.uint8)
    _attend(c, queries(3, 2, 3, D, 82))


def test_attention_many_sequences():
    lens = [int(n) for n in np.random.default_rng(4).integers(0, 70, 700)]
    c = filled(lens, heads=1, page_size=16, D=64, G=64, bits=4, seed=91)
    _attend(c, queries(700, 1, 2, 64, 92))


def test_attention_strided_queries():
    D, H, Hq, B, n = 128, 2, 6, 3, 2
    c = filled([50, 20, 90], heads=H, page_size=16, D=D, G=64, bits=8, seed=15)
    data, table, ln = on_gpu(c)
    qkv = torch.randn(B * n, (Hq + 2 * H) * D, device="cuda").bfloat16()
    q = qkv[:, :Hq * D].view(B, n, Hq, D)
    got = aq.aq_kv_attention(q, data, table, ln, 64, 8)
    assert got.shape == q.shape and got.is_contiguous()
    assert torch.equal(got, aq.aq_kv_attention(q.contiguous(), data, table, ln, 64, 8))
    turned = q.permute(2, 1, 0, 3).contiguous().permute(2, 1, 0, 3)
    assert torch.equal(got, aq.aq_kv_attention(turned, data, table, ln, 64, 8))
    _check(c, bits_of(q), got)
    # one token a sequence: three dimensions
    one = q[:, 1]
    flat = aq.aq_kv_attention(one, data, table, ln, 64, 8)
    assert flat.shape == (B, Hq, D)
    _check(c, bits_of(one)[:, None], flat)


def test_attention_repeats_bit_for_bit():
    c = filled([900, 5, 333], heads=2, page_size=16, D=128, G=64, bits=4, seed=17)
    gpu = on_gpu(c)
    q = queries(3, 1, 16, 128, 18)
    first, lse = _attend(c, q, gpu)
    for _ in range(5):
        again = torch.empty_like(lse)
        assert torch.equal(first, aq.aq_kv_attention(to_gpu(q), *gpu, 64, 4, lse=again)) and torch.equal(lse, again)


def test_shared_pages():
    """Two sequences that share a prefix's pages, and one page that stands twice in a sequence."""
    c = filled([64, 64, 48], heads=1, page_size=16, D=64, G=32, bits=4, seed=19)
    c.table[1, :3] = c.table[0, :3]
    c.table[2, 2] = c.table[2, 0]
    _attend(c, queries(3, 1, 4, 64, 20))
    got = aq.aq_kv_read(*on_gpu(c), 176, 64, 32, 4, offsets=_gpu([0, 64, 128, 176]))
    for x, y in zip(got, ref.read(c, 176, [0, 64, 128, 176])):
        assert np.array_equal(bits_of(x), y)


# ------------------------------------------------------------------------------ together, as a decoder uses them

def test_decode_loop():
    """Prompts are written, then tokens come one or a few at a time: written, then attended to, in two layers."""
    D, G, bits, H, Hq, page = 128, 64, 4, 2, 8, 16
    width, B = 6, 3
    rng = np.random.default_rng(5)
    layers = []
    for layer in range(2):
        c = cache([0] * B, heads=H, page_size=page, D=D, G=G, bits=bits, seed=100 + layer, width=width, spare=1)
        layers.append((c, on_gpu(c)[:2]))
    lens = np.zeros(B, np.int64)
    steps = [[14, 1, 30]] + [[1, 1, 1]] * 4 + [[3, 3, 3]] + [[1, 0, 1]] * 2
    for i, new in enumerate(steps):
        lens += new
        offsets = [0, *np.cumsum(new).tolist()]
        ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
        for layer, (c, (data, table)) in enumerate(layers):
            c.lens = lens.astype(np.int32)
            k, v = rows(offsets[-1], H, D, 7 * i + layer), rows(offsets[-1], H, D, 7 * i + layer + 50)
            even = len(set(new)) == 1
            aq.aq_kv_append(data, to_gpu(k), to_gpu(v), table, ln, G, bits, offsets=None if even else _gpu(offsets))
            ref.append(c, k, v, offsets)
            n = new[0] if even else 1
            q = bf16_bits(rng.standard_normal((B, n, Hq, D)))
            _attend(c, q, (data, table, ln))
            assert np.array_equal(data.cpu().numpy(), c.data)
    total = [0, *np.cumsum(lens).tolist()]
    for c, (data, table) in layers:
        got = aq.aq_kv_read(data, table, ln, total[-1], D, G, bits, offsets=_gpu(total))
        for x, y in zip(got, ref.read(c, total[-1], total)):
            assert np.array_equal(bits_of(x), y)


def test_captured_and_replayed():
    """A captured step is replayed on new tokens, lengths and pages; an eager call runs between two replays."""
    D, G, bits, H, Hq, B = 128, 64, 4, 2, 8, 4
    c = filled([100, 37, 0, 250], heads=H, page_size=16, D=D, G=G, bits=bits, seed=23, width=20)
    data, table, ln = on_gpu(c)
    k, v, q = (torch.zeros(B, x, D, dtype=torch.bfloat16, device="cuda") for x in (H, H, Hq))

    def step():
        aq.aq_kv_append(data, k, v, table, ln, G, bits)
        return aq.aq_kv_attention(q, data, table, ln, G, bits)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        scratch = data.clone()
        step()
        data.copy_(scratch)
    torch.cuda.current_stream().wait_stream(side)
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    outs = []
    for g in graphs:  # two graphs of the same step
        with torch.cuda.graph(g):
            outs.append(step())
    for i in range(4):
        c.lens = c.lens + np.array([1, 1, 1, 1], np.int32)
        if i == 1:
            c.lens[2] = 0  # a slot is given up
        ln.copy_(torch.from_numpy(c.lens))
        kb, vb, qb = rows(B, H, D, 30 + i), rows(B, H, D, 40 + i), queries(B, 1, Hq, D, 50 + i)
        k.copy_(to_gpu(kb)), v.copy_(to_gpu(vb)), q.copy_(to_gpu(qb[:, 0]))
        graphs[i % 2].replay()
        ref.append(c, kb, vb)
        eager = aq.aq_kv_attention(q, data, table, ln, G, bits)
        _check(c, qb, outs[i % 2])
        assert torch.equal(eager, outs[i % 2])
    assert np.array_equal(data.cpu().numpy(), c.data)


@pytest.mark.parametrize("captured", (False, True))
def test_steps_that_follow_one_another(captured):
    """Steps queued without a wait between them: each kernel reads what the one just before it wrote (lengths, tokens,
    queries, the cache).  The same bits as with a wait after every call."""
    D, G, bits, H, Hq, B, steps = 64, 32, 4, 4, 8, 3, 24
    c = filled([40, 300, 7], heads=H, page_size=16, D=D, G=G, bits=bits, seed=61, width=24)
    tokens = torch.randn(steps, 3, B, Hq, D, device="cuda").bfloat16()

    def run(wait):
        data, table, ln = on_gpu(c)
        q, k, v = (torch.empty(B, x, D, dtype=torch.bfloat16, device="cuda") for x in (Hq, H, H))
        last = torch.zeros(B, Hq, D, dtype=torch.bfloat16, device="cuda")
        outs = []

        def step(i):
            ln.add_(1)
            torch.add(tokens[i, 0], last, out=q)  # the step before goes into this one
            k.copy_(tokens[i, 1][:, :H])
            v.copy_(tokens[i, 2][:, :H])
            wait()
            aq.aq_kv_append(data, k, v, table, ln, G, bits)
            wait()
            aq.aq_kv_attention(q, data, table, ln, G, bits, out=last)
            wait()
            kr, vr = aq.aq_kv_read(data, table, ln, B, D, G, bits)
            wait()
            outs.append((last.clone(), kr, vr))

        if not captured or wait is not nothing:
            for i in range(steps):
                step(i)
        else:
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                for i in range(steps):
                    step(i)
            graph.replay()
        torch.cuda.synchronize()
        return data, outs

    def nothing():
        pass

    (d0, o0), (d1, o1) = run(torch.cuda.synchronize), run(nothing)
    assert torch.equal(d0, d1)
    for x, y in zip(o0, o1):
        assert all(torch.equal(a, b) for a, b in zip(x, y))


def test_broadcast_inputs_and_drafts_taken_back():
    """One head's values for all heads and one query for all rows (strides of 0); tokens that a draft wrote are written anew."""
    D, G, bits, H, Hq = 64, 32, 8, 3, 6
    c = filled([40, 17], heads=H, page_size=16, D=D, G=G, bits=bits, seed=61, width=4)
    data, table, ln = on_gpu(c)
    for new, back, seed in ((3, 2, 62), (2, 0, 63)):
        c.lens = c.lens + np.int32(new)
        ln.copy_(torch.from_numpy(c.lens))
        k, v = rows(2 * new, 1, D, seed), rows(2 * new, 1, D, seed + 10)
        aq.aq_kv_append(data, to_gpu(k).expand(-1, H, -1), to_gpu(v).expand(-1, H, -1), table, ln, G, bits)
        ref.append(c, np.repeat(k, H, 1), np.repeat(v, H, 1))
        assert np.array_equal(data.cpu().numpy(), c.data)
        q = queries(1, 1, 1, D, seed + 20)
        got = aq.aq_kv_attention(to_gpu(q).expand(2, new, Hq, D), data, table, ln, G, bits)
        _check(c, np.broadcast_to(q, (2, new, Hq, D)), got)
        c.lens = c.lens - np.int32(back)
    assert aq.aq_device_fault() == 0


def test_two_streams_at_once():
    """Calls on two streams, each with a workspace of its own, many of them in flight."""
    D, G, bits = 128, 64, 4
    cases = [filled([800, 60], heads=2, page_size=16, D=D, G=G, bits=bits, seed=s) for s in (1, 2)]
    qs = [queries(2, 1, 8, D, s) for s in (3, 4)]
    gpus = [on_gpu(c) for c in cases]
    qg = [to_gpu(q) for q in qs]
    want = [aq.aq_kv_attention(q, *g, G, bits) for q, g in zip(qg, gpus)]
    for c, q, w in zip(cases, qs, want):
        _check(c, q, w)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(aq.aq_kv_attention(qg[i], *gpus[i], G, bits))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(x, want[i]) for x in got[i])


def test_workspace_given():
    c = filled([500, 90], heads=2, page_size=16, D=64, G=64, bits=8, seed=27)
    gpu = on_gpu(c)
    q = to_gpu(queries(2, 1, 8, 64, 28))
    need = aq.aq_kv_attention_workspace_bytes(*gpu, 1, 8, 64, 64, 8)
    want = aq.aq_kv_attention(q, *gpu, 64, 8)
    guard = torch.full((need + 512,), 171, dtype=torch.uint8, device="cuda")
    got = aq.aq_kv_attention(q, *gpu, 64, 8, workspace=guard[256:256 + need])
    assert torch.equal(got, want)
    assert (guard[:256] == 171).all() and (guard[256 + need:] == 171).all()
    if need > 16:
        with pytest.raises(aq.AqError):
            aq.aq_kv_attention(q, *gpu, 64, 8, workspace=guard[256:256 + need - 16])


def test_a_cache_behind_32_bits():
    """A cache of over 4 GB whose last pages are used: byte offsets pass 2^32."""
    D, G, bits, H, page = 128, 32, 8, 8, 1024
    small = filled([1500], heads=H, page_size=page, D=D, G=G, bits=bits, seed=29)
    page_bytes = small.data[0].size
    pages = (1 << 32) // page_bytes + 8
    big = torch.empty((pages, *small.data.shape[1:]), dtype=torch.uint8, device="cuda")
    moved = small.table + (pages - small.pages)
    big[pages - small.pages:] = torch.from_numpy(small.data).cuda()
    assert int(moved.min()) * page_bytes > 1 << 32
    table, ln = torch.from_numpy(moved).cuda(), torch.from_numpy(small.lens).cuda()
    _attend(small, queries(1, 1, 8, D, 30), (big, table, ln))
    k, v = rows(5, H, D, 31), rows(5, H, D, 32)
    aq.aq_kv_append(big, to_gpu(k), to_gpu(v), table, ln, G, bits, offsets=_gpu([0, 5]))
    ref.append(small, k, v, [0, 5])
    assert np.array_equal(big[pages - small.pages:].cpu().numpy(), small.data)
    got = aq.aq_kv_read(big, table, ln, 9, D, G, bits, offsets=_gpu([0, 9]))
    for x, y in zip(got, ref.read(small, 9, [0, 9])):
        assert np.array_equal(bits_of(x), y)


# ------------------------------------------------------------------------------ absent pages, refusals

def test_absent_pages():
    """Entries outside the cache, and lengths behind the table's end: left out, read as zeros, and reported."""
    D, G, bits = 64, 32, 4
    c = filled([100, 60, 112, 16], heads=2, page_size=16, D=D, G=G, bits=bits, seed=33)
    c.table[0, 2], c.table[1, 0], c.table[3, 0] = -1, c.pages, 2**31 - 1
    assert c.table.shape[1] == 7
    c.lens[2] = 112 + 20
    gpu = on_gpu(c)
    _attend(c, queries(4, 1, 4, D, 34), gpu)
    assert aq.aq_device_fault() == aq.AQ_FAULT_BAD_INDEX
    _attend(c, queries(4, 2, 4, D, 35), gpu, window=40)
    assert aq.aq_device_fault() == aq.AQ_FAULT_BAD_INDEX
    n = [100, 60, int(c.lens[2]), 16]
    offsets = [0, *np.cumsum(n).tolist()]
    got = aq.aq_kv_read(*gpu, offsets[-1], D, G, bits, offsets=_gpu(offsets))
    for x, y in zip(got, ref.read(c, offsets[-1], offsets)):
        assert np.array_equal(bits_of(x), y)
    assert aq.aq_device_fault() == aq.AQ_FAULT_BAD_INDEX
    k, v = rows(offsets[-1], 2, D, 36), rows(offsets[-1], 2, D, 37)
    aq.aq_kv_append(gpu[0], to_gpu(k), to_gpu(v), *gpu[1:], G, bits, offsets=_gpu(offsets))
    ref.append(c, k, v, offsets)
    assert np.array_equal(gpu[0].cpu().numpy(), c.data)
    assert aq.aq_device_fault() == aq.AQ_FAULT_BAD_INDEX


def test_negative_lengths_are_empty():
    c = filled([20, 20], heads=1, page_size=16, D=64, G=64, bits=4, seed=38)
    c.lens[1] = -(2**31)
    _attend(c, queries(2, 2, 4, 64, 39), window=3)
    _attend(c, queries(2, 2, 4, 64, 39))
    assert not any(x[10:].any() for x in aq.aq_kv_read(*on_gpu(c), 20, 64, 64, 4))


def test_nothing_to_do():
    data = aq.aq_kv_cache(2, 1, 16, 64, 64, 4)
    assert data.shape == (2, 1, 16, 72) and not data.any()
    none = torch.empty((0, 1, 64), dtype=torch.bfloat16, device="cuda")
    table, ln = torch.zeros((1, 1), dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    aq.aq_kv_append(data, none, none, table, ln, 64, 4)
    assert aq.aq_kv_read(data, table, ln, 0, 64, 64, 4)[0].shape == (0, 1, 64)
    q = torch.empty((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    assert aq.aq_kv_attention(q, data, table[:0], ln[:0], 64, 4).shape == (0, 2, 64)


def test_refusals():
    D, G, bits, H = 128, 64, 4, 2
    data = aq.aq_kv_cache(4, H, 16, D, G, bits)
    table = torch.zeros((2, 2), dtype=torch.int32, device="cuda")
    ln = torch.ones(2, dtype=torch.int32, device="cuda")
    k = torch.zeros((2, H, D), dtype=torch.bfloat16, device="cuda")
    q = torch.zeros((2, 8, D), dtype=torch.bfloat16, device="cuda")
    ok = dict(cache=data, k=k, v=k, table=table, lens=ln, G=G, bits=bits)
    aq.aq_kv_append(**ok)
    for kw in (dict(cache=data.cpu()), dict(cache=data[:, :, ::2]), dict(cache=data[0]), dict(k=k.float()), dict(k=k[:, :1]), dict(v=k[:1]),
               dict(k=k.cpu()), dict(table=table.long()), dict(table=table[:1]), dict(table=table.cpu()), dict(lens=ln.float()),
               dict(lens=ln[:1]), dict(bits=3), dict(G=128), dict(k=k.transpose(1, 2)), dict(offsets=ln),
               dict(offsets=torch.zeros(3, dtype=torch.int64, device="cuda")), dict(k=k.repeat(2, 1, 1)[:3], v=k.repeat(2, 1, 1)[:3])):
        with pytest.raises((TypeError, ValueError, aq.AqError)):
            aq.aq_kv_append(**(ok | kw))
    with pytest.raises(aq.AqError):  # rows that do not begin on 16 bytes
        aq.aq_kv_append(**(ok | dict(k=torch.zeros(2 * H * D + 8, dtype=torch.bfloat16, device="cuda")[4:4 + 2 * H * D].view(2, H, D))))
    with pytest.raises(aq.AqError):
        aq.aq_kv_cache(4, H, 16, D, G, 2)
    ok = dict(q=q, cache=data, table=table, lens=ln, G=G, bits=bits)
    aq.aq_kv_attention(**ok)
    for kw in (dict(q=q[:1]), dict(q=q[:, :5]), dict(q=q.float()), dict(q=q[0]), dict(q=q[..., :64]), dict(window=-1),
               dict(scale=float("nan")), dict(out=q[:1]), dict(out=q.float()), dict(lse=torch.zeros(2, device="cuda")),
               dict(lse=torch.zeros((2, 8), dtype=torch.float64, device="cuda")), dict(lens=ln.cpu()), dict(G=32)):
        with pytest.raises((TypeError, ValueError, aq.AqError)):
            aq.aq_kv_attention(**(ok | kw))
    for kw in (dict(rows=3), dict(rows=-2), dict(out=(k, k[:1])), dict(out=(k, k.float())), dict(out=(k,)), dict(offsets=ln)):
        with pytest.raises((TypeError, ValueError, RuntimeError, aq.AqError)):
            aq.aq_kv_read(**(dict(cache=data, table=table, lens=ln, rows=2, D=D, G=G, bits=bits) | kw))
