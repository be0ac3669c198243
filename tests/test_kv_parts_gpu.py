"""Attention over the key-value cache where the work is cut by its bytes: units (a sequence's KV head and query rows) that
several warps and several CTAs have a part of, which a second kernel joins.  Calls whose table has room for few tokens
take one CTA for each unit instead, so here tables are as wide as a server's longest context, or units are many.  Short
sequences are cut all the same: a warp's run is then one chunk."""
import itertools

import numpy as np
import pytest
import torch

import kv_cases
import test_kv_gpu as narrow
from kv_cases import on_gpu, queries, to_gpu
from kv_stored import stored
from oracle import kv as ref
from test_kv_gpu import _attend

pytestmark = pytest.mark.gpu

aq = pytest.importorskip("weight_only_group_b200")

ROOM = 8192  # tokens of a table's row


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


def _wide(make):
    def made(lens, *, page_size, width=None, **kw):
        return make(lens, page_size=page_size, width=max(width or 1, ROOM // page_size), **kw)

    return made


def filled(lens, **kw):
    return _wide(kv_cases.filled)(lens, **kw)


@pytest.fixture
def wide(monkeypatch):
    """The tests of narrow tables, with wide ones."""
    monkeypatch.setattr(narrow, "filled", _wide(kv_cases.filled))
    monkeypatch.setattr(narrow, "cache", _wide(kv_cases.cache))


FORMS = [(D, G, bits) for D, G, bits in itertools.product((64, 128, 256), (32, 64, 128), (4, 8)) if G <= D]


def test_a_wide_table_needs_room_for_parts():
    c, w = (make([40], heads=1, page_size=16, D=64, G=64, bits=4, seed=1) for make in (kv_cases.filled, filled))
    need = [aq.aq_kv_attention_workspace_bytes(*on_gpu(x), 1, 4, 64, 64, 4) for x in (c, w)]
    assert need[1] > need[0]


@pytest.mark.parametrize("D,G,bits", FORMS)
@pytest.mark.parametrize("heads,q_heads,tokens", [(2, 8, 1), (1, 7, 1), (1, 4, 3), (1, 5, 4)])  # 4, 7, 12 and 20 rows a KV head
def test_forms(D, G, bits, heads, q_heads, tokens):
    c = filled([300, 0, 77, 33], heads=heads, page_size=32, D=D, G=G, bits=bits, seed=D + G)
    _attend(c, queries(4, tokens, q_heads, D, 21))


def _synthetic(lens, D, G, bits, seed, heads=1, page_size=64, width=None):
    """Random codes under scales and biases of a usual size, quicker to make than quantised rows."""
    def fill(rng, shape):
        return rng.uniform(0.05, 0.4, shape) * 2.0 ** (4 - bits), rng.uniform(-3, 0, shape)

    return stored(lens, fill=fill, heads=heads, page_size=page_size, D=D, G=G, bits=bits, seed=seed, width=width)


@pytest.mark.parametrize("D,G,bits,rows", [(64, 64, 4, 4), (128, 64, 4, 4), (64, 32, 8, 8), (128, 128, 4, 16), (256, 64, 4, 8), (256, 128, 8, 3)])
def test_one_long_sequence_among_short_ones(D, G, bits, rows):
    """Of 60 units one has dozens of parts, the others one or two."""
    lens = [5 + i % 40 for i in range(60)]
    lens[23] = 7001
    c = _synthetic(lens, D, G, bits, 3)
    q = queries(60, 1, rows, D, 4)
    gpu = on_gpu(c)
    out, lse = _attend(c, q, gpu)
    for _ in range(3):
        again = torch.empty_like(lse)
        assert torch.equal(out, aq.aq_kv_attention(to_gpu(q), *gpu, G, bits, lse=again)) and torch.equal(lse, again)


@pytest.mark.parametrize("D,G,bits,rows", [(256, 64, 4, 4), (256, 32, 8, 8), (128, 64, 4, 16), (64, 32, 4, 4)])
@pytest.mark.parametrize("lens", ([2500], [9000, 1, 600]))
def test_few_units_of_many_parts(D, G, bits, rows, lens):
    c = _synthetic(lens, D, G, bits, 5, width=256)
    _attend(c, queries(len(lens), 2, rows // 2, D, 6))


@pytest.mark.parametrize("window", (300, 333, 1000))
@pytest.mark.parametrize("tokens,q_heads", [(1, 4), (3, 4)])
def test_windows(window, tokens, q_heads):
    """Windows of more tokens than a unit of one CTA has (8 bits, D = 256: 256), that begin inside a tile."""
    lens = [900, 310, 40, 0, 1500, 301]
    c = _synthetic(lens, 256, 32, 8, 7, page_size=16)
    first = max(0, (1500 - tokens + 1 - window) // 16 - 1)
    c.table[4, :first] = 1 << 30  # pages before the window: not needed
    _attend(c, queries(len(lens), tokens, q_heads, 256, 8), window=window)


def test_windows_of_many_sequences():
    """More units than the GPU holds CTAs."""
    lens = [int(n) for n in np.random.default_rng(9).integers(0, 200, 120)]
    c = _synthetic(lens, 64, 64, 4, 9, heads=4, page_size=16)
    _attend(c, queries(120, 2, 8, 64, 10), window=40)


@pytest.mark.parametrize("bits", (4, 8))
def test_absent_pages(bits):
    D, G = 128, 64
    lens = [100, 600, 112, 16, 512]
    c = _synthetic(lens, D, G, bits, 11, page_size=16, width=ROOM // 16)
    c.table[0, 2], c.table[1, 0], c.table[3, 0] = -1, c.pages, 2**31 - 1
    c.table[4, ::2] = -5
    c.lens[2] = 0
    _attend(c, queries(5, 2, 8, D, 12))
    assert aq.aq_device_fault() == aq.AQ_FAULT_BAD_INDEX


def test_lengths_behind_the_table():
    D, G, bits = 256, 32, 8
    c = _synthetic([512, 300], D, G, bits, 13, page_size=16, width=32)
    c.lens[0] = 512 + 37
    q = queries(2, 3, 4, D, 14)
    want, _ = _attend(c, q)
    assert aq.aq_device_fault() == aq.AQ_FAULT_BAD_INDEX
    c.lens[0] = 2**31 - 1  # every row of the sequence sees the whole table, as before
    assert torch.equal(want, aq.aq_kv_attention(to_gpu(q), *on_gpu(c), G, bits))
    assert aq.aq_device_fault() == aq.AQ_FAULT_BAD_INDEX


@pytest.mark.parametrize("bits", (4, 8))
@pytest.mark.parametrize("bad", (0x7C00, 0xFC00, 0x7E01))
def test_beside_tokens_that_are_not_finite(bits, bad):
    """Random bytes lie behind every sequence's end; the last drafted token is seen by the last row alone."""
    D, G, n = 64, 32, 4
    c = filled([700, 35, 64], heads=1, page_size=16, D=D, G=G, bits=bits, seed=17)
    q = queries(3, n, 6, D, 18)
    want, _ = _attend(c, q)
    for b, length in enumerate(c.lens.tolist()):
        page, tile, row = c.locate(b, length - 1)
        flat = c.data[page, 0].reshape(-1)
        for which in (0, 1):
            flat[c.spans(tile, row, which)[1]] = np.full(2 * c.ng, bad, np.uint16).view(np.uint8)
    got = aq.aq_kv_attention(to_gpu(q), *on_gpu(c), G, bits)
    r = ref.attention(filled([700, 35, 64], heads=1, page_size=16, D=D, G=G, bits=bits, seed=17), q, D**-0.5)
    far, _ = ref.attention_bounds(r, D)
    assert (np.abs(got.float().cpu().numpy() - r["out"]) <= far)[:, :-1].all()
    assert not torch.isfinite(got[:, -1]).all()


# ------------------------------------------------------------------------------ the tests of narrow tables, with wide ones

@pytest.mark.parametrize("tokens,q_heads,heads", [(1, 9, 1), (1, 16, 1), (1, 17, 1), (3, 12, 2), (6, 8, 1), (5, 64, 2)])
def test_head_groups(wide, tokens, q_heads, heads):
    narrow.test_attention_head_groups(tokens, q_heads, heads)


@pytest.mark.parametrize("length", [1, 16, 17, 31, 32, 33, 64, 65, 128, 256, 257, 513])
@pytest.mark.parametrize("bits", (4, 8))
def test_lengths(wide, length, bits):
    narrow.test_attention_lengths(length, bits)


@pytest.mark.parametrize("test", ("test_attention_of_many_tokens", "test_attention_sharp_and_flat", "test_attention_scales_of_v_far_apart",
                                  "test_attention_constant_values", "test_attention_strided_queries",
                                  "test_attention_repeats_bit_for_bit", "test_shared_pages", "test_decode_loop",
                                  "test_captured_and_replayed", "test_broadcast_inputs_and_drafts_taken_back",
                                  "test_two_streams_at_once", "test_workspace_given", "test_negative_lengths_are_empty",
                                  "test_attention_of_queries_of_extreme_sizes"))
def test_of_narrow_tables(wide, test):
    getattr(narrow, test)()


@pytest.mark.parametrize("captured", (False, True))
def test_steps_that_follow_one_another(wide, captured):
    narrow.test_steps_that_follow_one_another(captured)


@pytest.mark.parametrize("tokens,q_heads", [(1, 3), (2, 6)])
def test_beside_a_query_that_is_not_finite(wide, tokens, q_heads):
    narrow.test_attention_beside_a_query_that_is_not_finite(tokens, q_heads, float("nan"))
