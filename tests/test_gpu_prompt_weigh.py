"""Weights that the keys of whole prompts receive, on the GPU, against a plain 64-bit statement (tests/weigh_ref.py, with
what bounds the error).  Sums of n rows: a tile's 128 in four, then tiles one by one, 2^-24 (32 + n / 128) of the sum."""
import pytest
import torch

import router_softmax_top_gb300 as moe
from tests import weigh_ref as W
from tests.test_gpu_kv_cache import i32, make_table

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def cu_of(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


def case(lens, hq, hkv, d, dtype, ps=32, prefix=0, window=0, scale=None, seed=0, q_size=1.0):
    g = torch.Generator().manual_seed(seed)
    keys = [n + prefix if not isinstance(prefix, list) else n + prefix[i] for i, n in enumerate(lens)]
    q = (torch.randn(sum(lens), hq, d, generator=g) * q_size).to(DT[dtype])
    k = torch.randn(sum(keys), hkv, d, generator=g).to(DT[dtype])
    n_pages = sum(-(-n // ps) for n in keys) + 2
    c = dict(q=q.cuda(), k=k.cuda(), cu=cu_of(lens), cu_k=cu_of(keys), table=make_table(keys, ps, n_pages, seed), ps=ps, window=window,
             scale=d ** -0.5 if scale is None else scale, totals=torch.rand(n_pages, hkv, ps, generator=g), lens=lens, keys=keys)
    lse = [W.seen_lse(*_part(c, s), c["scale"], window) for s in range(len(lens))]
    c["lse"] = torch.cat(lse).float() if lse else torch.zeros(0, hq)
    return c


def _part(c, s):
    n, m = c["lens"][s], c["keys"][s]
    q, k = c["q"][c["cu"][s]:c["cu"][s + 1]].cpu().double(), c["k"][c["cu_k"][s]:c["cu_k"][s + 1]].cpu().double()
    return q, k, [m - n + i for i in range(n)], m


def run(c, totals=None, **kw):
    t = c["totals"].cuda() if totals is None else totals
    same = c["cu"] == c["cu_k"]
    out = moe.prompt_weigh(c["q"], c["k"], c["lse"].cuda(), i32(c["cu"]), None if same else i32(c["cu_k"]), totals=t,
                           page_table=c["table"].cuda(), scale=c["scale"], window=c["window"], **kw)
    assert out is t
    return out


def check(c, restart=False):
    got = run(c, restart=restart).cpu()
    want, tol = c["totals"].double(), torch.zeros_like(c["totals"], dtype=torch.float64)
    for s, (n, m) in enumerate(zip(c["lens"], c["keys"])):
        q, k, at, _ = _part(c, s)
        add, off = W.received(q, k, c["lse"][c["cu"][s]:c["cu"][s + 1]].double(), at, m, c["scale"], c["window"])
        tok = torch.arange(m)
        page = c["table"][s][tok // c["ps"]].long()
        old = want[page, :, tok % c["ps"]]
        old[0 if restart else max(0, m - n):] = 0
        want[page, :, tok % c["ps"]] = old + add
        rows = n * c["q"].shape[1] // c["k"].shape[1]
        tol[page, :, tok % c["ps"]] = off + 2.0 ** -23 * old + 2.0 ** -24 * (32 + rows / 128 + 4) * add
    err = (got.double() - want).abs()
    assert bool((err <= tol).all()), float((err / tol.clamp(min=1e-300))[err > 0].max())
    return got


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("hq,hkv,dtype,lens,prefix,window", [
    (1, 1, "bf16", [1], 0, 0),
    (16, 8, "bf16", [37], 0, 0),
    (6, 2, "f16", [130, 1, 0, 257], 0, 0),
    (4, 4, "bf16", [300], 0, 64),
    (5, 1, "bf16", [200, 33], 100, 0),
    (14, 2, "f16", [40, 129], [500, 3], 0),
    (8, 8, "bf16", [128, 127, 129], 0, 1),
    (64, 1, "bf16", [50], 70, 33),
    (3, 1, "f16", [5], 700, 0),
    (2, 2, "bf16", [260], 300, 200)])
def test_weights_received(d, hq, hkv, dtype, lens, prefix, window):
    c = case(lens, hq, hkv, d, dtype, prefix=prefix, window=window, seed=d + hq)
    check(c)
    check(c, restart=True)


def test_many_sequences_and_large_pages():
    check(case([(11 * i) % 70 for i in range(75)], 4, 2, 64, "bf16", ps=256, seed=1))


def test_a_longer_prompt():
    check(case([1500], 4, 2, 128, "bf16", seed=2))


def test_more_queries_than_keys():
    # the first rows stand before the first key and see nothing
    c = case([100], 4, 2, 64, "bf16", seed=3)
    c["keys"], c["cu_k"] = [60], [0, 60]
    c["lse"] = W.seen_lse(*_part(c, 0), c["scale"], 0).float()
    assert bool(c["lse"][:40].isinf().all())
    check(c)


def test_large_and_small_queries():
    for size, scale in ((1e-30, None), (300.0, 1e-3), (2.0 ** 100, 2.0 ** -103), (2.0 ** -100, 2.0 ** 98)):
        check(case([90], 2, 1, 64, "bf16", scale=scale, q_size=size, seed=4))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("hq", [2, 3])
def test_lse_of_any_size_over_whole_tiles(dtype, hq):
    # rows that all see all keys of a tile, with scores and scales from small to near the types' limits
    for size, scale in ((1.0, None), (0.01, 3.0), (300.0, 1e-4), (3000.0, 1e-10), (1e-3, 1e4)):
        check(case([450], hq, 1, 64, dtype, prefix=40, scale=scale, q_size=size, seed=14))
    if dtype == "bf16":
        for size, scale in ((2.0 ** 100, 2.0 ** -104), (2.0 ** -100, 2.0 ** 97), (2.0 ** 110, 2.0 ** -126)):
            check(case([450], hq, 1, 64, dtype, scale=scale, q_size=size, seed=15))
    c = case([450], hq, 1, 64, dtype, seed=16)
    c["lse"][400:405] += 40.0          # rows that count for little, for nothing and for much
    c["lse"][410] = float("inf")
    c["lse"][420] -= 30.0
    check(c)


def test_attentions_own_lse_gives_weights_that_sum_to_one():
    c = case([700, 33, 1], 16, 4, 128, "bf16", seed=5)
    _, lse = moe.prompt_attention(c["q"], c["k"], c["k"], i32(c["cu"]), return_lse=True)
    got = moe.prompt_weigh(c["q"], c["k"], lse, i32(c["cu"]), totals=c["totals"].cuda(), page_table=c["table"].cuda()).cpu()
    for s, n in enumerate(c["lens"]):
        tok = torch.arange(n)
        mine = got[c["table"][s][tok // 32].long(), :, tok % 32].double()
        assert bool(((mine.sum(0) / (4 * n) - 1).abs() < 1e-4).all())   # lse is off by 2^-17 Z, Z below 13


def test_what_is_not_seen_does_not_reach_a_key():
    c = case([200, 150], 4, 2, 64, "bf16", prefix=90, window=70, seed=6)
    clean = run(c)
    for row in (0, 149, 199, 200):
        q = c["q"].clone()
        q[row] = float("nan")
        got = run(dict(c, q=q))
        s = int(row >= 200)
        p = row - (200 if s else 0) + 90
        tok = torch.arange(max(0, p - 69), p + 1)
        page = c["table"][s][tok // 32].long().cuda()
        assert bool(got[page, :, tok.cuda() % 32].isnan().all())
        got[page, :, tok.cuda() % 32] = clean[page, :, tok.cuda() % 32]
        assert torch.equal(got, clean)
    k = c["k"].clone()
    k[100], k[290 + 10] = float("inf"), float("nan")
    got = run(dict(c, k=k))
    for s, i in ((0, 100), (1, 10)):
        page = int(c["table"][s][i // 32])
        got[page, :, i % 32] = clean[page, :, i % 32]
    assert torch.equal(got, clean)
    # of a group that leaves rows of a tile empty, an infinite key is weighed by the rows that there are
    c = case([300], 3, 1, 64, "f16", seed=7)
    k, q = c["k"].clone(), c["q"].abs() + 0.1
    clean = run(dict(c, q=q))
    k[20] = -float("inf")
    got = run(dict(c, q=q, k=k))
    page = int(c["table"][0][0])
    assert bool((got[page, :, 20] == 0).all())
    got[page, :, 20] = clean[page, :, 20]
    assert torch.equal(got, clean)


def test_the_same_call_gives_the_same_bits_and_chunks_add_up():
    c = case([600], 8, 2, 128, "bf16", seed=8)
    whole = run(c)
    assert torch.equal(whole, run(c))
    t = c["totals"].cuda()
    for a, b in ((0, 250), (250, 251), (251, 600)):
        part = dict(c, q=c["q"][a:b], k=c["k"][:b], lse=c["lse"][a:b], cu=[0, b - a], cu_k=[0, b])
        run(part, totals=t)
    tok = torch.arange(600)
    page = c["table"][0][tok // 32].long().cuda()
    a, b = whole[page, :, tok.cuda() % 32], t[page, :, tok.cuda() % 32]
    assert bool(((a - b).abs() <= 2.0 ** -18 * b).all())


def test_offsets_and_pages_that_make_no_sense():
    c = case([100, 80, 60], 4, 2, 64, "bf16", seed=9)
    clean = run(c)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    totals = c["totals"].cuda()
    own = [sorted(set(c["table"][s].tolist()) - {-1}) for s in range(3)]

    def expect(cu_q, cu_k, counts, bit):
        status.zero_()
        got = moe.prompt_weigh(c["q"], c["k"], c["lse"].cuda(), i32(cu_q), i32(cu_k), totals=totals.clone(),
                               page_table=c["table"].cuda(), status=status)
        assert int(status) == bit
        for s in range(3):
            assert torch.equal(got[own[s]], clean[own[s]] if s in counts else totals[own[s]]), (s, cu_q, cu_k)
    cu = c["cu"]
    expect(cu, cu, (0, 1, 2), 0)
    expect([0, 100, 180, 241], cu, (0, 1), moe.MOE_KV_BAD_LENGTH)
    expect(cu, [0, 100, 180, 241], (0, 1), moe.MOE_KV_BAD_LENGTH)
    expect(cu, [-1, 100, 180, 240], (1, 2), moe.MOE_KV_BAD_LENGTH)
    expect(cu, [0, 1000, 180, 240], (), moe.MOE_KV_BAD_LENGTH)
    t = c["table"].clone()
    t[1, 1] = 1 << 20
    status.zero_()
    got = run(dict(c, table=t), status=status)
    assert int(status) == moe.MOE_KV_BAD_PAGE
    keep = int(c["table"][1, 1])
    assert torch.equal(got[keep].cpu(), c["totals"][keep])
    got[keep] = clean[keep]
    assert torch.equal(got, clean)
    status.zero_()                           # a row of the table that is too short
    got = run(dict(c, table=c["table"][:, :3]), status=status)
    assert int(status) == moe.MOE_KV_BAD_LENGTH
    assert torch.equal(got[own[2]], clean[own[2]]) and torch.equal(got[own[0]].cpu(), c["totals"][own[0]])


def test_no_queries_and_no_keys():
    c = case([0, 0], 4, 2, 64, "bf16", prefix=50, seed=10)
    assert torch.equal(run(c).cpu(), c["totals"])
    got = run(c, restart=True).cpu()
    for s in range(2):
        tok = torch.arange(50)
        assert not bool(got[c["table"][s][tok // 32].long(), :, tok % 32].any())
    empty = moe.prompt_weigh(c["q"], c["k"][:0], c["lse"].cuda(), i32([0, 0, 0]), totals=c["totals"].cuda(), page_table=c["table"].cuda())
    assert torch.equal(empty.cpu(), c["totals"])


def test_strides_streams_and_graphs():
    c = case([130, 77], 6, 2, 64, "bf16", seed=11)
    want = run(c)
    fused = torch.randn(207, 10, 64, device="cuda").bfloat16()
    fused[:, :6], fused[:, 6:8] = c["q"], c["k"]
    assert torch.equal(run(dict(c, q=fused[:, :6], k=fused[:, 6:8])), want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = run(c, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, want)
    cu, lse, table, totals = i32(c["cu"]), c["lse"].cuda(), c["table"].cuda(), c["totals"].cuda()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.prompt_weigh(c["q"], c["k"], lse, cu, totals=totals, page_table=table, scale=c["scale"])
    for _ in range(2):
        totals.copy_(c["totals"])
        g.replay()
        assert torch.equal(totals, want)


def test_refusals():
    c = case([40], 4, 2, 64, "bf16", seed=12)
    good = dict(q=c["q"], k=c["k"], lse=c["lse"].cuda(), cu_q=i32([0, 40]), totals=c["totals"].cuda(), page_table=c["table"].cuda())
    moe.prompt_weigh(**good)
    for bad in (dict(q=c["q"].float()), dict(k=c["k"].half()), dict(q=c["q"].cpu()), dict(lse=good["lse"][:, :1]), dict(lse=good["lse"].double()),
                dict(cu_q=i32([0, 40, 40])), dict(cu_q=torch.tensor([0, 40])), dict(cu_k=i32([0])), dict(totals=good["totals"][0]),
                dict(totals=good["totals"][:, :1]), dict(totals=good["totals"].cpu()), dict(page_table=good["page_table"].long()),
                dict(page_table=c["table"]), dict(scale=0.0), dict(window=-1), dict(k=torch.cat([c["k"]] * 3, 1)[:, :3])):
        with pytest.raises(moe.MoeError):
            moe.prompt_weigh(**dict(good, **bad))
