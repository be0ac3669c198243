"""Forms of the key-value cache whose tokens have the same number of bytes are told apart."""
import itertools

import pytest
import torch

pytestmark = pytest.mark.gpu

aq = pytest.importorskip("weight_only_group_b200")

FORMS = [(D, G, bits) for D, G, bits in itertools.product((64, 128, 256), (32, 64, 128), (4, 8)) if G <= D]


@pytest.mark.parametrize("form", FORMS)
def test_a_cache_is_refused_for_another_form(form):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    same = [f for f in FORMS if f != form and aq.aq_kv_token_bytes(*f) == aq.aq_kv_token_bytes(*form)]
    assert all(f[0] != form[0] for f in same)
    cache = aq.aq_kv_cache(2, 1, 16, *form)
    table, lens = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in ((1, 1), (1,)))

    def calls(cache, D, G, bits):
        x = torch.zeros((1, 1, D), dtype=torch.bfloat16, device="cuda")
        yield lambda: aq.aq_kv_append(cache, x, x, table, lens, G, bits)
        yield lambda: aq.aq_kv_read(cache, table, lens, 1, D, G, bits)
        yield lambda: aq.aq_kv_attention(x, cache, table, lens, G, bits)
        yield lambda: aq.aq_kv_attention_workspace_bytes(cache, table, lens, 1, 1, D, G, bits)

    for call in calls(cache, *form):
        call()
    for other in same:
        for call in calls(cache, *other):
            with pytest.raises(ValueError, match="made for"):
                call()
        for call in calls(cache.view(2, 1, 16, -1), *other):  # a view does not know: bytes are all there is
            call()
    assert aq.aq_device_fault() == 0
