"""Counts of the key-value cache near the end of 32 bits."""
import numpy as np
import pytest
import torch

from kv_cases import bits_of, cache, rows, to_gpu
from oracle import kv as ref

pytestmark = pytest.mark.gpu

aq = pytest.importorskip("weight_only_group_b200")


def test_as_many_sequences_as_there_may_be():
    """2^31 - 1 sequences, two of which have a row: steps of the search through the offsets pass 2^31 nowhere."""
    if not torch.cuda.is_available() or torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 26 GB of the GPU's memory")
    D, G, bits, batch, middle = 64, 32, 4, 2**31 - 1, 1234567890
    c = cache([3, 9], heads=2, page_size=16, D=D, G=G, bits=bits, seed=1)
    k, v = rows(2, 2, D, 2), rows(2, 2, D, 3)
    offsets, lens = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (batch + 1, batch))
    table = torch.full((batch, 1), -1, dtype=torch.int32, device="cuda")
    offsets[middle + 1:], offsets[batch] = 1, 2
    for b, at in enumerate((middle, batch - 1)):
        lens[at], table[at] = int(c.lens[b]), int(c.table[b, 0])
    data = torch.from_numpy(c.data).cuda()
    aq.aq_kv_append(data, to_gpu(k), to_gpu(v), table, lens, G, bits, offsets=offsets)
    ref.append(c, k, v)
    assert np.array_equal(data.cpu().numpy(), c.data)
    got = aq.aq_kv_read(data, table, lens, 2, D, G, bits, offsets=offsets)
    for x, y in zip(got, ref.read(c, 2)):
        assert np.array_equal(bits_of(x), y)
    assert aq.aq_device_fault() == 0
