"""The key-value cache's calls, which are launched as programmatic dependents, behind and beside every kind of work: fills,
copies, and other streams' calls, in a captured graph and without one."""
import pytest
import torch

from kv_cases import filled, on_gpu

pytestmark = pytest.mark.gpu

aq = pytest.importorskip("weight_only_group_b200")


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    aq.lib()


@pytest.mark.parametrize("width", (24, 1024))  # a CTA for each unit; units cut across CTAs, and a join
@pytest.mark.parametrize("captured", (False, True))
def test_calls_behind_fills_copies_and_other_streams(width, captured):
    """Two layers, one on a side stream that comes off the main one and goes back to it, over and over; the same bits as
    with a wait after every call."""
    D, G, bits, H, Hq, B, steps = 64, 32, 4, 2, 8, 3, 6
    layers = [filled([40, 300, 7], heads=H, page_size=16, D=D, G=G, bits=bits, seed=s, width=width) for s in (1, 2)]
    torch.manual_seed(0)
    tokens = torch.randn(steps, 2, 3, B, Hq, D, device="cuda").bfloat16()
    lengths = torch.tensor([[41 + i, 301 + i, 8 + i] for i in range(steps)], dtype=torch.int32, device="cuda")

    def run(wait):
        gpus = [on_gpu(c) for c in layers]
        ln = gpus[0][2]
        qs, ks, vs = ([torch.empty(B, n, D, dtype=torch.bfloat16, device="cuda") for _ in layers] for n in (Hq, H, H))
        lse = [torch.empty(B, Hq, device="cuda") for _ in layers]
        outs = [torch.empty(B, Hq, D, dtype=torch.bfloat16, device="cuda") for _ in layers]
        kept = []
        side = torch.cuda.Stream()

        def layer(i, n):
            data, table, _ = gpus[n]
            ks[n].copy_(tokens[i, n, 1, :, :H].clone())
            vs[n].copy_(tokens[i, n, 2, :, :H].clone())
            qs[n].copy_(tokens[i, n, 0])
            wait()
            aq.aq_kv_append(data, ks[n], vs[n], table, ln, G, bits)
            wait()
            lse[n].zero_()
            aq.aq_kv_attention(qs[n], data, table, ln, G, bits, lse=lse[n], out=outs[n])
            wait()

        def go():
            main = torch.cuda.current_stream()
            for i in range(steps):
                ln.copy_(lengths[i])  # a copy right in front of a call
                side.wait_stream(main)
                layer(i, 0)
                with torch.cuda.stream(side):
                    layer(i, 1)
                main.wait_stream(side)
                # behind two streams at once
                kept.append(aq.aq_kv_read(gpus[1][0], gpus[1][1], ln, B, D, G, bits))
                wait()
                kept.append((outs[0].clone(), outs[1].clone(), lse[0].clone(), lse[1].clone()))
                outs[0].zero_(), outs[1].zero_()

        if captured and wait is not torch.cuda.synchronize:
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                go()
            graph.replay()
        else:
            go()
        torch.cuda.synchronize()
        return [g[0] for g in gpus], kept

    want, got = run(torch.cuda.synchronize), run(lambda: None)
    assert all(torch.equal(a, b) for a, b in zip(want[0], got[0]))
    for x, y in zip(want[1], got[1]):
        assert all(torch.equal(a, b) for a, b in zip(x, y))
    assert aq.aq_device_fault() == 0
