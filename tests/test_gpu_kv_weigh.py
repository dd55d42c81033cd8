"""Weights that cached tokens receive, on the GPU, against a plain 64-bit statement (tests/weigh_ref.py, with what bounds
the error).  A total that was there before adds a rounding of the sum: 2^-24 of it."""
import pytest
import torch

import router_softmax_top_gb300 as moe
from tests import attention_ref as R
from tests import weigh_ref as W
from tests.test_gpu_kv_cache import filled, i32

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def case(lens, ps, hq, hkv, d, dtype, q_tokens=1, window=0, scale=None, seed=0, k_size=1.0, q_size=1.0):
    pages, table = filled(lens, ps, hkv, d, seed, k_size=k_size)
    g = torch.Generator().manual_seed(seed + 1)
    q = (torch.randn(len(lens) * q_tokens, hq, d, generator=g) * q_size).to(DT[dtype]).cuda()
    scale = d ** -0.5 if scale is None else scale
    host = pages.cpu()
    keys = [R.sequence(host, table[s], n, ps, hkv, d)[0] for s, n in enumerate(lens)]
    at = [[n - q_tokens + j for j in range(q_tokens)] for n in lens]
    rows = [q[s * q_tokens:(s + 1) * q_tokens].cpu().double() for s in range(len(lens))]
    lse = torch.cat([W.seen_lse(rows[s], keys[s], at[s], n, scale, window) for s, n in enumerate(lens)]).float()
    totals = torch.rand(pages.shape[0], hkv, ps, generator=g)
    return dict(pages=pages, table=table, q=q, lse=lse, totals=totals, lens=lens, ps=ps, hkv=hkv, scale=scale, window=window,
                q_tokens=q_tokens, keys=keys, rows=rows, at=at)


def run(c, totals=None, **kw):
    t = c["totals"].cuda() if totals is None else totals
    out = moe.kv_weigh(c["q"], c["pages"], c["table"].cuda(), i32(c["lens"]), c["lse"].cuda(), totals=t, page_size=c["ps"],
                       n_kv_heads=c["hkv"], q_tokens=c["q_tokens"], scale=c["scale"], window=c["window"], **kw)
    assert out is t
    return out


def check(c, restart=False, lse=None):
    got = run(c, restart=restart).cpu()
    want, tol = c["totals"].double(), torch.zeros_like(c["totals"], dtype=torch.float64)
    q_tokens = c["q_tokens"]
    for s, n in enumerate(c["lens"]):
        l = c["lse"][s * q_tokens:(s + 1) * q_tokens].double()
        add, off = W.received(c["rows"][s], c["keys"][s], l, c["at"][s], n, c["scale"], c["window"])
        tok = torch.arange(n)
        page = c["table"][s][tok // c["ps"]].long()
        old = want[page, :, tok % c["ps"]]
        old[0 if restart else max(0, n - q_tokens):] = 0
        want[page, :, tok % c["ps"]] = old + add
        tol[page, :, tok % c["ps"]] = off + 2.0 ** -23 * (old + add)
    err = (got.double() - want).abs()
    assert bool((err <= tol).all()), float((err / tol.clamp(min=1e-300))[err > 0].max())
    return got


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("hq,hkv,dtype,ps,lens,q_tokens,window", [
    (1, 1, "bf16", 32, [1], 1, 0),
    (16, 8, "bf16", 64, [333], 1, 0),
    (8, 2, "f16", 96, [31, 32, 33, 0, 64, 500, 1], 1, 0),
    (6, 2, "bf16", 32, [70, 5, 129], 3, 0),
    (16, 1, "f16", 64, [100, 40], 1, 0),
    (16, 2, "bf16", 128, [200, 3], 5, 0),
    (8, 8, "bf16", 32, [300, 33, 2], 2, 64),
    (24, 8, "f16", 256, [1000, 257], 1, 100),
    (4, 1, "bf16", 32, [90], 37, 0),
    (4, 4, "bf16", 64, [500, 20, 130], 40, 33),
    (12, 4, "bf16", 64, [65] * 40, 1, 1)])
def test_weights_received(d, hq, hkv, dtype, ps, lens, q_tokens, window):
    c = case(lens, ps, hq, hkv, d, dtype, q_tokens, window, seed=d + hq)
    check(c)
    check(c, restart=True)


def test_more_sequences_than_lanes_and_empty_ones():
    lens = [(7 * i) % 90 if i % 3 else 0 for i in range(150)]
    check(case(lens, 32, 4, 2, 64, "bf16", seed=3))


def test_large_and_small_queries():
    for size, k_size, scale in ((1e-30, 1.0, None), (300.0, 1.0, 1e-3), (2.0 ** 100, 1.0, 2.0 ** -104), (2.0 ** -90, 1.0, 2.0 ** 88),
                                (1.0, 1e-3, 30.0), (1.0, 1000.0, 1e-4)):
        check(case([77, 40], 32, 4, 2, 128, "bf16", scale=scale, k_size=k_size, q_size=size, seed=9))


def test_attentions_own_lse_gives_weights_that_sum_to_one():
    c = case([700, 33, 1, 64], 64, 16, 4, 128, "bf16", seed=5)
    _, lse = moe.kv_attention(c["q"], c["pages"], c["table"].cuda(), i32(c["lens"]), page_size=64, n_kv_heads=4, return_lse=True)
    got = moe.kv_weigh(c["q"], c["pages"], c["table"].cuda(), i32(c["lens"]), lse, totals=c["totals"].cuda(), page_size=64,
                       n_kv_heads=4, restart=True).cpu()
    for s, n in enumerate(c["lens"]):
        tok = torch.arange(n)
        mine = got[c["table"][s][tok // 64].long(), :, tok % 64]
        assert bool((mine.sum(0) - 4).abs().max() < 4e-3)   # four query heads share a key head; lse is off by 2^-17 Z


def test_the_same_call_gives_the_same_bits_and_steps_add_up():
    c = case([900, 450], 64, 8, 2, 128, "bf16", q_tokens=2, seed=6)
    a, b = run(c), run(c)
    assert torch.equal(a, b)
    again = run(c, totals=a.clone()).double() - a.double()
    first = b.double() - c["totals"].cuda().double()
    for s, n in enumerate(c["lens"]):  # of tokens that are not new
        tok = torch.arange(n - 2)
        page = c["table"][s][tok // 64].long().cuda()
        assert torch.allclose(again[page, :, tok.cuda() % 64], first[page, :, tok.cuda() % 64], atol=2.0 ** -22)


def test_what_is_not_seen_stays_as_it_is():
    c = case([200], 64, 4, 2, 64, "bf16", q_tokens=2, window=40, seed=7)
    c["totals"].fill_(float("nan"))
    got = run(c).cpu()
    tok = torch.arange(200)
    mine = got[c["table"][0][tok // 64].long(), :, tok % 64]
    assert bool(mine[:198].isnan().all()) and not bool(mine[198:].isnan().any())   # the new ones begin at 0
    # a key that is NaN and out of the window, one that is past the end
    c = case([200], 64, 4, 2, 64, "bf16", window=40, seed=7)
    clean = run(c)
    t = moe.kv_read(c["pages"], c["table"].cuda(), i32([100]), i32([0, 1]), 1, page_size=64, n_kv_heads=2, head_dim=64)[0]
    assert bool(t.isfinite().all())
    bad = torch.full((1, 2, 64), float("nan"), device="cuda")
    for at in (100, 200):
        pages = c["pages"].clone()
        moe.kv_append(pages, c["table"].cuda(), i32([at]), i32([0, 1]), bad, bad, page_size=64)
        assert torch.equal(run(dict(c, pages=pages)), clean)
    pages = c["pages"].clone()
    moe.kv_append(pages, c["table"].cuda(), i32([190]), i32([0, 1]), bad, bad, page_size=64)
    one = run(dict(c, pages=pages))
    page = int(c["table"][0][190 // 64])
    assert bool(one[page, :, 190 % 64].isnan().all())
    one[page, :, 190 % 64] = clean[page, :, 190 % 64]
    assert torch.equal(one, clean)


def test_bad_pages_and_lengths_touch_nothing():
    c = case([200, 100], 64, 4, 2, 64, "bf16", seed=8)
    clean = run(c)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for bad in (-1, c["pages"].shape[0], 1 << 30):
        t = c["table"].clone()
        t[0, 1] = bad
        status.zero_()
        got = run(dict(c, table=t), status=status)
        assert int(status) == moe.MOE_KV_BAD_PAGE
        keep = int(c["table"][0, 1])
        assert torch.equal(got[keep].cpu(), c["totals"][keep])
        got[keep] = clean[keep]
        assert torch.equal(got, clean)
    for bad in (-1, c["table"].shape[1] * 64 + 1, 0x7fffffff):
        status.zero_()
        got = run(dict(c, lens=[bad, 100]), status=status)
        assert int(status) == moe.MOE_KV_BAD_LENGTH
        for p in c["table"][0].tolist():
            assert torch.equal(got[p].cpu(), c["totals"][p])


def test_strides_streams_and_graphs():
    c = case([130, 77, 300], 32, 8, 4, 128, "bf16", seed=10)
    want = run(c)
    wide = torch.randn(3, 12, 256, device="cuda").bfloat16()
    wide[:, 2:10, 64:192] = c["q"]
    pool = torch.zeros(c["pages"].shape[0], 2 * c["pages"].shape[1], dtype=torch.uint8, device="cuda")
    pool[:, :c["pages"].shape[1]] = c["pages"]
    t = torch.full((3, 40), -1, dtype=torch.int32)
    t[:, :c["table"].shape[1]] = c["table"]
    assert torch.equal(run(dict(c, q=wide[:, 2:10, 64:192], pages=pool[:, :c["pages"].shape[1]], table=t)), want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = run(c, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, want)
    table, lens, lse, totals = c["table"].cuda(), i32(c["lens"]), c["lse"].cuda(), c["totals"].cuda()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.kv_weigh(c["q"], c["pages"], table, lens, lse, totals=totals, page_size=32, n_kv_heads=4, scale=c["scale"])
    for n in ([130, 77, 300], [100, 1, 0]):
        lens.copy_(i32(n))
        totals.copy_(c["totals"])
        g.replay()
        assert torch.equal(totals, run(dict(c, lens=n)))


def test_refusals():
    c = case([40], 32, 4, 2, 64, "bf16", seed=11)
    good = dict(q=c["q"], pages=c["pages"], page_table=c["table"].cuda(), seq_lens=i32([40]), lse=c["lse"].cuda(),
                totals=c["totals"].cuda(), page_size=32, n_kv_heads=2)
    moe.kv_weigh(**good)
    for bad in (dict(q=c["q"].float()), dict(q=c["q"].cpu()), dict(q=c["q"][0]), dict(lse=good["lse"].double()),
                dict(lse=good["lse"][:, :2]), dict(lse=good["lse"].cpu()), dict(totals=good["totals"].half()),
                dict(totals=good["totals"][:, :1]), dict(totals=good["totals"].cpu()), dict(totals=good["totals"][:-1]),
                dict(page_size=48), dict(n_kv_heads=3), dict(q_tokens=2), dict(scale=0.0), dict(scale=-1.0),
                dict(scale=float("nan")), dict(window=-1), dict(seq_lens=i32([40, 1])), dict(seq_lens=torch.tensor([40])),
                dict(status=torch.zeros(1, device="cuda"))):
        with pytest.raises(moe.MoeError):
            moe.kv_weigh(**dict(good, **bad))
    empty = moe.kv_weigh(c["q"][:0], c["pages"], torch.zeros(0, 2, dtype=torch.int32, device="cuda"), i32([]), good["lse"][:0],
                         totals=good["totals"], page_size=32, n_kv_heads=2)
    assert empty is good["totals"]
