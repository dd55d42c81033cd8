"""A prompt over a cache that tokens were evicted from: appended at positions that are not places, read back, attended over
and its weights summed, by itself and as a layer does it (examples/decoder_layer.py)."""
import pytest
import torch

import router_softmax_top_gb300 as moe
from tests import attention_ref as R
from tests import weigh_ref as W
from tests.test_gpu_bounded_layer import routing, start
from tests.test_gpu_kv_cache import i32, make_table
from tests.test_gpu_prompt_weigh import cu_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,hq,hkv,window", [(64, 6, 2, 0), (128, 4, 4, 0), (256, 4, 1, 0), (64, 4, 2, 50)])
def test_weights_of_a_prompt_over_what_is_left(d, hq, hkv, window):
    before, new, budget, ps = [300, 90, 517, 129, 0], [40, 0, 130, 1, 33], 128, 64
    g = torch.Generator().manual_seed(d)
    most = [b + n for b, n in zip(before, new)]
    n_pages = sum(-(-n // ps) for n in most) + 2
    pages, table = moe.kv_pages(n_pages, hkv, d, ps), make_table(most, ps, n_pages, 1).cuda()
    cos, sin = moe.rope_table(1024, d)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = dict(page_size=ps, cos=cos, sin=sin, status=status)

    def tokens(n, heads):
        return torch.randn(n, heads, d, generator=g).cuda().bfloat16()
    moe.kv_append(pages, table, i32([0] * 5), i32(cu_of(before)), tokens(sum(before), hkv), tokens(sum(before), hkv), **args)
    totals = torch.rand(n_pages, hkv, ps, generator=g).cuda()
    lens, _ = moe.kv_evict(pages, table, i32(before), budget, totals=totals, page_size=ps, n_kv_heads=hkv, head_dim=d, first=4,
                           recent=16, status=status)
    held = [min(b, budget) for b in before]
    assert lens.tolist() == held
    q, _ = moe.kv_append(pages, table, lens, i32(cu_of(new)), tokens(sum(new), hkv), tokens(sum(new), hkv), q=tokens(sum(new), hq),
                         positions=i32(before), **args)
    keys = [h + n for h, n in zip(held, new)]
    cu, cu_k = i32(cu_of(new)), i32(cu_of(keys))
    k, v = moe.kv_read(pages, table, i32([0] * 5), cu_k, sum(keys), page_size=ps, n_kv_heads=hkv, head_dim=d, status=status)
    o, lse = moe.prompt_attention(q, k, v, cu, cu_k, window=window, return_lse=True, status=status)
    old = totals.cpu()
    moe.prompt_weigh(q, k, lse, cu, cu_k, totals=totals, page_table=table, window=window, status=status)
    assert int(status) == 0 and bool(o.isfinite().all())
    want, tol = old.double(), torch.zeros(old.shape, dtype=torch.float64)
    for s, (n, m) in enumerate(zip(new, keys)):
        if m == 0:
            continue
        qs, ks = q[cu[s]:cu[s + 1]].cpu().double(), k[cu_k[s]:cu_k[s + 1]].cpu().double()
        # what is read back is what the cache holds, in the places that the kept tokens have now
        exact, _ = R.sequence(pages.cpu(), table[s].cpu(), m, ps, hkv, d)
        assert torch.equal(ks, exact.bfloat16().double())
        add, off = W.received(qs, ks, lse[cu[s]:cu[s + 1]].cpu().double(), [m - n + i for i in range(n)], m, d ** -0.5, window)
        tok = torch.arange(m)
        page = table[s].cpu()[tok // ps].long()
        was = want[page, :, tok % ps]
        was[m - n:] = 0
        want[page, :, tok % ps] = was + add
        tol[page, :, tok % ps] = off + 2.0 ** -23 * was + 2.0 ** -24 * (32 + n * hq // hkv / 128 + 4) * add
    err = (totals.cpu().double() - want).abs()
    assert bool((err <= tol).all()), float((err / tol.clamp(min=1e-300))[err > 0].max())


def more(hidden):
    g = torch.Generator().manual_seed(7)
    return torch.randn(25, hidden, generator=g).cuda(), torch.tensor([0, 5, 5, 25], dtype=torch.int32, device="cuda")


def test_with_room_for_all_a_chunk_is_the_plain_layers():
    E, layer, cu, x, steps = start(512)
    plain, hidden = E.build()
    piece, cu2 = more(hidden)
    for a in (layer, plain):
        a.prompt(x, cu)
        a.decode(steps[0])
    layer.bound()
    assert torch.equal(layer.chunk(piece, cu2, 340), plain.chunk(piece, cu2, 340))
    assert torch.equal(layer.pages, plain.pages) and torch.equal(layer.lens, plain.lens)
    assert layer.positions.tolist() == layer.lens.tolist() == [106, 38, 221]
    assert torch.equal(layer.decode(steps[1]), plain.decode(steps[1])) and int(layer.status) == 0


def test_a_second_turn_over_a_bounded_cache():
    E, layer, cu, x, steps = start(64, routing=routing())
    layer.prompt(x, cu)
    layer.decode(steps[0])
    layer.bound()
    piece, cu2 = more(x.shape[1])

    def held(s):
        tok = torch.arange(int(layer.lens[s]), device="cuda")
        return layer.totals[layer.table[s][tok // 64].long(), :, tok % 64]
    before = [held(s).sum(0) for s in range(3)]
    out = layer.chunk(piece, cu2, int(layer.lens.sum()))
    assert layer.lens.tolist() == [69, 38, 84] and layer.positions.tolist() == [106, 38, 221]
    for s, n in enumerate((5, 0, 20)):
        # a row's weights sum to 1, and two query heads share a key head
        assert bool(((held(s).sum(0) - before[s] - 2 * n).abs() <= 1e-3 * (before[s] + 2 * n)).all())
    layer.bound()
    assert layer.lens.tolist() == [64, 38, 64]
    assert bool(out.isfinite().all() & layer.decode(steps[1]).isfinite().all())
    assert int(layer.status) == 0 and layer.experts.sync() == moe.MOE_OK
