"""Routing, sums of attention and eviction together, as a decoder layer uses them (examples/decoder_layer.py)."""
import importlib.util
import os

import pytest
import torch

import router_softmax_top_gb300 as moe
from tests import attention_ref as R

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LENS = [100, 37, 200]


def example():
    spec = importlib.util.spec_from_file_location("decoder_layer", os.path.join(ROOT, "examples", "decoder_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def routing():
    return dict(score="sigmoid", bias=torch.linspace(-0.1, 0.1, 8, device="cuda"), n_groups=4, top_groups=2, renormalise=True)


def start(budget, **kw):
    E = example()
    layer, hidden = E.build(kind=E.BoundedDecoderLayer, budget=budget, **kw)
    g = torch.Generator().manual_seed(0)
    cu = torch.tensor([0, 100, 137, 337], dtype=torch.int32, device="cuda")
    x = torch.randn(337, hidden, generator=g).cuda()
    return E, layer, cu, x, [torch.randn(3, hidden, generator=g).cuda() for _ in range(12)]


def test_the_example_runs():
    example().main()


def test_with_room_for_all_it_is_the_plain_layer():
    E, layer, cu, x, steps = start(512)
    plain, _ = E.build()
    assert torch.equal(layer.prompt(x, cu), plain.prompt(x, cu))
    for s in steps[:4]:
        kept = layer.bound()
        assert torch.equal(layer.decode(s), plain.decode(s))
    assert torch.equal(layer.pages, plain.pages) and torch.equal(layer.lens, plain.lens)
    assert [int((kept[i, 0] >= 0).sum()) for i in range(3)] == [103, 40, 203]
    assert int(layer.status) == 0


def test_weights_sum_to_the_queries_and_evictions_keep_the_heaviest():
    E, layer, cu, x, steps = start(64, routing=routing())
    layer.prompt(x, cu)
    for s in steps[:3]:
        layer.decode(s)

    def held(s):
        tok = torch.arange(int(layer.lens[s]), device="cuda")
        return layer.totals[layer.table[s][tok // 64].long(), :, tok % 64]
    for s, n in enumerate(LENS):
        # a row's weights sum to 1, and two query heads share a key head; lse of the prompt is of keys before they were quantised
        assert bool(((held(s).sum(0) / (2 * (n + 3)) - 1).abs() < 1e-3).all())
    before = [held(s) for s in range(3)]
    k0 = [R.sequence(layer.pages.cpu(), layer.table[s].cpu(), LENS[s] + 3, 64, 2, 64) for s in range(3)]
    kept = layer.bound()
    assert layer.lens.tolist() == [64, 40, 64] and layer.positions.tolist() == [103, 40, 203]
    for s in (0, 2):
        n = LENS[s] + 3
        k1 = R.sequence(layer.pages.cpu(), layer.table[s].cpu(), 64, 64, 2, 64)
        for h in range(2):
            mid = before[s][4:n - 16, h].sort(descending=True, stable=True).indices[:44] + 4
            want = torch.cat([torch.arange(4, device="cuda"), mid.sort().values, torch.arange(n - 16, n, device="cuda")])
            assert torch.equal(kept[s, h].long(), want)
            assert torch.equal(held(s)[:, h], before[s][want, h])
            for a, b in zip(k0[s], k1):
                assert torch.equal(a[want.cpu(), h], b[:, h])
    # and on: new tokens take the places after, at their own positions
    for s in steps[3:6]:
        out = layer.decode(s)
    assert layer.lens.tolist() == [67, 43, 67] and layer.positions.tolist() == [106, 43, 206]
    assert bool(out.isfinite().all()) and int(layer.status) == 0 and layer.experts.sync() == moe.MOE_OK


def test_captured_steps_are_the_eager_ones():
    E, a, cu, x, steps = start(80, routing=routing())
    _, b, _, _, _ = start(80, routing=routing())
    for layer in (a, b):
        layer.prompt(x, cu)
        layer.bound()
        layer.decode(steps[0])
    torch.cuda.synchronize()
    step = steps[1].clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = a.decode(step)
        a.bound()
    for s in steps[1:]:
        step.copy_(s)
        g.replay()
        want = b.decode(s)
        b.bound()
        assert torch.equal(out, want)
    assert torch.equal(a.pages, b.pages) and torch.equal(a.totals, b.totals)
    assert a.lens.tolist() == b.lens.tolist() == [80, 49, 80]
    assert int(a.status) == 0
