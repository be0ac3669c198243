"""Attention over the key-value cache gives up a wait that does not end, says so, and leaves the context usable."""
import pytest
import torch

from kv_cases import filled, on_gpu, queries, to_gpu
from test_kv_gpu import _check

pytestmark = pytest.mark.gpu

aq = pytest.importorskip("weight_only_group_b200")


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    aq.lib()


@pytest.mark.parametrize("bits", (4, 8))
@pytest.mark.parametrize("width", (None, 1024))  # a CTA for each unit; units cut across CTAs, and a join
def test_a_wait_that_runs_out(bits, width):
    """A launch that also waits on a barrier that nothing completes, its copies in flight, with its waits limited to 20,000
    SM cycles: it sets the bit of its own, waits for its copies and returns.  The next call is right, and leaves no fault."""
    D, G = 64, 32
    c = filled([300, 0, 41], heads=2, page_size=16, D=D, G=G, bits=bits, seed=1, width=width)
    q, gpu = queries(3, 2, 4, D, 2), on_gpu(c)
    assert aq.aq_device_fault() == 0
    aq.aq_set_wait_limit(20000)
    aq.aq_set_wait_stall(True)
    try:
        aq.aq_kv_attention(to_gpu(q), *gpu, G, bits)
        torch.cuda.synchronize()
    finally:
        aq.aq_set_wait_stall(False)
        aq.aq_set_wait_limit(0)
    assert aq.aq_device_fault() == 0x40 == aq.AQ_FAULT_WAIT_MASK & ~0x1F
    _check(c, q, aq.aq_kv_attention(to_gpu(q), *gpu, G, bits))
    assert aq.aq_device_fault() == 0
