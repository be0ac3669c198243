"""Attention over the key-value cache at the edges of what the cache and the queries may hold: scales of either sign, scores
of any size, queries of very different sizes.  Against the 64-bit oracle, within the bounds of its arithmetic."""
import itertools

import numpy as np
import pytest
import torch

from kv_cases import queries
from kv_stored import stored
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
