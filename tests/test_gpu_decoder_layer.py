"""The attention operators and the routed layer together (examples/decoder_layer.py): a
prompt in one piece, in two, and token by token give the same sequence outputs up to the
rounding of the 4-bit cache."""
import importlib.util
import os

import pytest
import torch

import router_softmax_top_gb300 as moe

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("decoder_layer", os.path.join(ROOT, "examples", "decoder_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_example_runs(example, capsys):
    example.main()
    assert "status ok" in capsys.readouterr().out


def test_prompt_chunks_and_decode_agree(example):
    torch.manual_seed(3)
    layer, hidden = example.build(seqs=2)
    x = torch.randn(2 * 70, hidden, device="cuda")
    cu = torch.tensor([0, 70, 140], dtype=torch.int32, device="cuda")
    a = layer._append(x, cu)
    whole = moe.prompt_attention(*a, cu)
    # the same tokens over the 4-bit cache, all at once and one after the other
    kc, vc = moe.kv_read(layer.pages, layer.table, torch.zeros_like(layer.lens), cu, 140, page_size=64, n_kv_heads=2,
                         head_dim=64)
    cached = moe.prompt_attention(a[0], kc, vc, cu)
    for n in (1, 31, 33, 64, 70):
        rows = [n - 1, 70 + n - 1]
        lens = torch.full((2,), n, dtype=torch.int32, device="cuda")
        one = moe.kv_attention(a[0][rows], layer.pages, layer.table, lens, page_size=64, n_kv_heads=2)
        # both are attention over the same values (read back as bf16: half a step of each, and of both results)
        lim = 4 * 2.0 ** -8 * float(vc.float().abs().max())
        assert float((one.float() - cached[rows].float()).abs().max()) <= lim
    # a 4-bit value is off by at most half a step of its block (an eighth of its largest): its share of the result is
    # bounded by that, the keys' by the change of the weights; together well under half of the values' size
    off = (whole.float() - cached.float()).norm() / whole.float().norm()
    assert float(off) < 0.5
    # through the layer: a second piece after a first one, against both in one
    l1, _ = example.build(seqs=2)
    l2, _ = example.build(seqs=2)
    first = torch.tensor([0, 40, 80], dtype=torch.int32, device="cuda")
    second = torch.tensor([0, 30, 60], dtype=torch.int32, device="cuda")
    xs = x.view(2, 70, -1)
    l1.prompt(xs[:, :40].reshape(80, -1), first)
    got = l1.chunk(xs[:, 40:].reshape(60, -1), second, 80)
    l2.prompt(x, cu)
    assert l1.lens.tolist() == l2.lens.tolist() == [70, 70]
    # the cache does not depend on how the tokens came, but for codes that the projections' rounding (matrix products of
    # another number of rows) puts on the other side of a border
    assert float((l1.pages != l2.pages).float().mean()) < 0.02
    assert got.shape == (60, hidden) and bool(torch.isfinite(got).all())
    nxt = torch.randn(2, hidden, device="cuda")
    d1, d2 = l1.decode(nxt), l2.decode(nxt)
    assert float((d1 - d2).norm() / d2.norm()) < 0.05
    assert moe.status_message(l1.status) == "" and moe.status_message(l2.status) == ""
