"""Attention over the key-value cache at the edges of what the cache and the queries may hold: scales of either sign, scores
of any size, queries of very different sizes.  Against the 64-bit oracle, within the bounds of its arithmetic."""
import itertools

import numpy as np
import pytest
import torch

from kv_cases import bf16_bits, queries
from kv_stored import pairs, places, stored
from oracle import kv as ref
from test_kv_gpu import _attend

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


FORMS = [(D, G, bits) for D, G, bits in itertools.product((64, 128, 256), (32, 64, 128), (4, 8)) if G <= D]


@pytest.mark.parametrize("D,G,bits", FORMS)
@pytest.mark.parametrize("signs", ("mixed", "negative", "large and negative"))
def test_scales_below_zero(D, G, bits, signs):
    """Scales of either sign, which the format allows though the library's own quantiser writes none below 0."""
    def fill(rng, shape):
        s = rng.uniform(0.05, 0.4, shape) * 2.0 ** (4 - bits)
        if signs == "mixed":
            s *= rng.choice((-1.0, 1.0), shape)
        elif signs == "negative":
            s = -s
        else:  # a few large ones below 0 among small ones above
            s = np.where(rng.random(shape) < 0.1, -20.0 * s, 2.0**-10 * s)
        return s, rng.uniform(-3, 3, shape)

    c = stored([150, 33], fill=fill, heads=2, D=D, G=G, bits=bits, seed=D + G)
    _attend(c, queries(2, 1, 8, D, 5))
    _attend(c, queries(2, 3, 8, D, 6), window=40)


@pytest.mark.parametrize("q_heads", (4, 8, 16))
def test_scores_far_from_zero(q_heads):
    """Scores of tens of thousands that differ by little, beside V scales just below a power of two.  A warp's second chunk
    holds a score that is a factor of about 8 above its first chunk's, where a weight is the largest it may be; at such a
    size an fp32 has steps of 2^-8 to 2^-7 to tell."""
    D, G, bits, B, n = 128, 32, 4, 64, 1024

    def fill(rng, shape):
        s, b = np.zeros(shape), np.zeros(shape)
        s[..., 1, :] = 1.0 - 2.0**-11
        b[..., 0, 0] = -30000.0
        return s, b

    c = stored([n] * B, fill=fill, page_size=64, D=D, G=G, bits=bits, seed=9)
    at, rng = pairs(c).swapaxes(0, 1)[0], np.random.default_rng(10)
    for b in range(B):
        where = places(c, b, n)
        k = at[where][:, 0, :, 1].copy()  # biases of K: the first group is a score's bulk, the others what it differs by
        for first in range(0, n, 64):
            k[first + 5, 0] = k[first + 40, 0] = 32 * rng.integers(1024, 2047)
            k[first + 40, 1] = 2.0 + 0.0078125 * rng.integers(6, 14)
            k[first + 40, 2] = 0.00390625 * rng.integers(0, 3)
        at[where[0], where[1], where[2], 0, :, 1] = k
    # a row's score is the sum of its token's biases: q = 1 in all of a group's 32 places, and the factor 1 / 32
    q = bf16_bits(np.ones((B, 1, q_heads, D)))
    _attend(c, q, scale=1 / 32)


@pytest.mark.parametrize("bits", (4, 8))
@pytest.mark.parametrize("v_scale", (1.0 - 2.0**-11, 2.0**-14, 2.0**-20, 65504.0))
@pytest.mark.parametrize("size", (2.0**12, 2.0**20, -(2.0**22), 2.0**30, -(2.0**50)))
def test_scores_so_far_apart_that_one_token_counts(size, v_scale, bits):
    """Each row's softmax is one token's, so the row is that token's v.  What is off is the rounding to bf16 and that of the
    weighted scale to fp16: 2^-8 of the value and 2^-11 of scale * code."""
    D, G, n = 64, 32, 300

    def fill(rng, shape):
        s, b = np.zeros(shape), np.zeros(shape)
        s[..., 1, :] = v_scale
        b[..., 1, :] = -v_scale
        b[..., 0, 0] = 100.0 + 0.5 * rng.permutation(int(np.prod(shape[:-2]))).reshape(shape[:-2])
        return s, b

    c = stored([n, 77], fill=fill, D=D, G=G, bits=bits, seed=11)
    q = bf16_bits(np.full((2, 1, 6, D), size))
    out, _ = _attend(c, q)
    r = ref.attention(c, q, D**-0.5)
    far = 2.0**-8 * np.abs(r["out"]) + (1 + 2.0**-8) * (2.0**-11 + 2.0**-20) * r["spread"]
    assert (np.abs(out.float().cpu().numpy() - r["out"].reshape(out.shape)) <= far.reshape(out.shape)).all()


@pytest.mark.parametrize("lens,width", [([1], None), ([300, 40, 0], None), ([700, 3, 40], 512)])
@pytest.mark.parametrize("size", (2.0**80, 2.0**95))
def test_scores_far_below_zero(size, lens, width):
    """Every score of a row is below -2^80: the row still is the softmax of what it sees.  k = 100 to 250, q = -size."""
    D, G, bits = 64, 32, 4

    def fill(rng, shape):
        s, b = np.zeros(shape), np.zeros(shape)
        s[..., 1, :] = 0.25
        return s, b

    c = stored(lens, fill=fill, D=D, G=G, bits=bits, seed=13, width=width)
    at, rng = pairs(c).swapaxes(0, 1)[0], np.random.default_rng(14)
    for b, n in enumerate(lens):
        page, tile, row = places(c, b, n)
        at[page, tile, row, 0, 0, 1] = 100.0 + 0.125 * rng.permutation(1200)[:n]
    q = bf16_bits(np.full((len(lens), 2, 4, D), -size))
    out, lse = _attend(c, q)
    r = ref.attention(c, q, D**-0.5)
    far = 2.0**-8 * np.abs(r["out"]) + (1 + 2.0**-8) * (2.0**-11 + 2.0**-20) * r["spread"]
    assert (np.abs(out.float().cpu().numpy() - r["out"]) <= far).all()
    assert torch.isneginf(lse).cpu().numpy().sum() == np.isneginf(r["lse"]).sum()


def test_a_factor_near_the_largest_number():
    """Queries of 2^-128 under a factor near fp32's largest: scores of a usual size."""
    c = stored([60, 9], fill=lambda rng, shape: (rng.uniform(0.01, 0.1, shape), rng.uniform(-2, 0, shape)), D=64, G=32, bits=4, seed=15)
    q = np.random.default_rng(16).standard_normal((2, 1, 4, 64)) * 2.0**-128
    _attend(c, bf16_bits(q), scale=3e38)


@pytest.mark.parametrize("bits", (4, 8))
def test_queries_with_elements_of_very_different_sizes(bits):
    """Elements down to 2^-28 of their row's largest count in full: the largest meets keys of 0, and the factor makes the
    rest a score of some size."""
    D, G, B = 64, 32, 3

    def fill(rng, shape):
        s, b = np.zeros(shape), np.zeros(shape)
        s[..., 0, 1] = rng.uniform(10, 60, shape[:-2]) * 2.0 ** (8 - bits)
        s[..., 1, :] = 0.1
        return s, b

    c = stored([50, 7, 90], fill=fill, D=D, G=G, bits=bits, seed=17)
    rng = np.random.default_rng(18)
    q = np.zeros((B, 1, 4, D))
    q[..., 3] = 1.0
    q[..., 32:] = rng.choice((-1, 1), (B, 1, 4, 32)) * 2.0**-28 * (1 + rng.integers(64, 128, (B, 1, 4, 32)) / 128)
    _attend(c, bf16_bits(q), scale=2.0**14)


def test_queries_below_the_normal_numbers():
    """Rows of the smallest bf16 there are, and a factor that makes scores of them."""
    D, G, bits = 64, 32, 8
    c = stored([60, 9], fill=lambda rng, shape: (rng.uniform(0.01, 0.1, shape), rng.uniform(-9, 0, shape)), D=D, G=G, bits=bits, seed=19)
    rng = np.random.default_rng(20)
    q = rng.integers(-255, 256, (2, 1, 4, D)) * 2.0 ** -np.array([133.0, 130.0, 120.0, 110.0])[:, None]
    _attend(c, bf16_bits(q), scale=2.0**110)
