"""Eviction on the GPU against a plain statement: bytes, totals and choices are equal."""
import pytest
import torch

import router_softmax_top_gb300 as moe
from tests.test_gpu_kv_cache import i32, make_table

pytestmark = pytest.mark.gpu


def pool(lens, ps, hkv, d, seed, spread="wide", width=None):
    n_pages = sum(-(-n // ps) for n in lens) + 2
    g = torch.Generator().manual_seed(seed)
    pages = torch.randint(0, 256, (n_pages, moe.kv_page_bytes(hkv, d, ps)), generator=g, dtype=torch.uint8)
    x = torch.randn(n_pages, hkv, ps, generator=g)
    totals = {"wide": torch.exp(x * 2), "ties": (x * 2).round().abs(), "zero": torch.zeros_like(x), "near": 1 + x.abs() * 2.0 ** -22,
              "signed": x, "tiny": x * 1e-42}[spread]
    return pages, make_table(lens, ps, n_pages, seed, width), totals


def rows(pages, table_row, n, ps, hkv, d):
    """The bytes of a sequence's slots: [n, hkv, bytes of a token]."""
    t = pages[table_row[:-(-n // ps)].long()].unflatten(1, (hkv, ps // 32, 36 * d))
    out = []
    for v in (0, 1):
        part = t[..., 18 * d * v:18 * d * (v + 1)]
        out.append(part[..., :16 * d].unflatten(-1, (d // 32, 32, 16)).transpose(-2, -3).flatten(-2))
        out.append(part[..., 16 * d:].unflatten(-1, (32, d // 16)))
    return torch.cat(out, -1).permute(0, 2, 3, 1, 4).flatten(0, 2)[:n]


def same(a, b):
    """Equal, NaN being equal to NaN."""
    return torch.equal(a.isnan(), b.isnan()) and torch.equal(a.nan_to_num(0.0, 7.0, 9.0), b.nan_to_num(0.0, 7.0, 9.0))


def order(v):
    """Keys that order as the kernel's: NaN above all."""
    return [(1, 0.0) if x != x else (0, x) for x in v]


def expect(pages, table, totals, lens, budget, first, recent, ps, hkv, d):
    """kept per (sequence, head), and the state after."""
    kept = torch.full((len(lens), hkv, budget), -1, dtype=torch.int32)
    after = []
    for s, n in enumerate(lens):
        tok = torch.arange(n)
        held = rows(pages, table[s], n, ps, hkv, d) if n else None
        t = totals[table[s][tok // ps].long(), :, tok % ps].clone() if n else torch.zeros(0, hkv)
        for h in range(hkv):
            if n <= budget:
                mine = list(range(n))
            else:
                key = order(t[:, h].tolist())
                mid = sorted(range(first, n - recent), key=lambda i: (-key[i][0], -key[i][1] if key[i][0] == 0 else 0, i))
                mine = sorted(list(range(first)) + mid[:budget - first - recent] + list(range(n - recent, n)))
            kept[s, h, :len(mine)] = torch.tensor(mine, dtype=torch.int32)
            if n > budget:
                held_h, t_h = held[:, h].clone(), t[:, h].clone()
                held[:len(mine), h], t[:len(mine), h] = held_h[mine], t_h[mine]
                t[len(mine):, h] = 0
        after.append((held, t))
    return kept, after


def check(lens, ps, hkv, d, budget, first=0, recent=0, spread="wide", seed=0, width=None, state=None, **kw):
    pages, table, totals = pool(lens, ps, hkv, d, seed, spread, width) if state is None else state
    p, t = pages.cuda(), totals.cuda()
    new, kept = moe.kv_evict(p, table.cuda(), i32(lens), budget, totals=t, page_size=ps, n_kv_heads=hkv, head_dim=d, first=first,
                             recent=recent, **kw)
    want, after = expect(pages, table, totals, lens, budget, first, recent, ps, hkv, d)
    assert new.tolist() == [min(n, budget) for n in lens]
    assert torch.equal(kept.cpu(), want)
    p, t = p.cpu(), t.cpu()
    used = torch.zeros(pages.shape[0], dtype=torch.bool)
    for s, n in enumerate(lens):
        if n == 0:
            continue
        tok = torch.arange(n)
        used[table[s][:-(-n // ps)].long()] = True
        assert torch.equal(rows(p, table[s], n, ps, hkv, d), after[s][0]), s
        assert same(t[table[s][tok // ps].long(), :, tok % ps], after[s][1]), s
        # slots past the sequence's end
        rest = torch.arange(n, -(-n // ps) * ps)
        assert same(t[table[s][rest // ps].long(), :, rest % ps], totals[table[s][rest // ps].long(), :, rest % ps])
    assert torch.equal(p[~used], pages[~used]) and same(t[~used], totals[~used])
    return p, t, new, kept


@pytest.mark.parametrize("d,hkv,ps", [(64, 2, 32), (128, 1, 96), (256, 3, 64)])
@pytest.mark.parametrize("lens,budget,first,recent", [
    ([1], 1, 0, 0), ([2], 1, 0, 0), ([2], 1, 1, 0), ([2], 1, 0, 1), ([40], 0, 0, 0), ([33, 32, 31, 0, 64], 32, 4, 8),
    ([300, 10, 257], 256, 0, 0), ([700, 513, 512, 40], 300, 4, 64), ([1500], 1499, 1, 1), ([1100, 900], 100, 100, 0),
    ([1100, 900], 100, 0, 100), ([1000], 999, 0, 0), ([2000], 50, 25, 25)])
def test_eviction(d, hkv, ps, lens, budget, first, recent):
    check(lens, ps, hkv, d, budget, first, recent, seed=budget)


@pytest.mark.parametrize("spread", ["ties", "zero", "near", "signed", "tiny"])
def test_ties_and_spreads(spread):
    check([900, 300, 2100], 64, 2, 64, 250, 3, 20, spread, seed=4)


def test_totals_that_are_not_numbers():
    lens, ps = [600, 100], 32
    pages, table, totals = pool(lens, ps, 2, 64, 5)
    flat = totals.view(-1)
    g = torch.Generator().manual_seed(1)
    for v in (float("nan"), float("inf"), -float("inf"), -0.0, 0.0):
        flat[torch.randint(0, flat.numel(), (200,), generator=g)] = v
    flat[torch.randint(0, flat.numel(), (50,), generator=g)] = torch.tensor([0xFFC00000 - (1 << 32)], dtype=torch.int32).view(torch.float32)
    check(lens, ps, 2, 64, 90, state=(pages, table, totals))


def test_long_sequences_and_many_groups():
    # a pair over several CTAs; every slot's token comes from far behind, or from the next one
    for budget, first in ((20000, 0), (39999, 0), (39999, 20000), (300, 0)):
        check([40000], 256, 1, 64, budget, first, 0, seed=budget + first)
    # the first token goes, everything else moves by one
    pages, table, totals = pool([30000], 64, 2, 64, 6)
    totals[table[0, 0], :, 0] = -1.0
    p, t, _, kept = check([30000], 64, 2, 64, 29999, state=(pages, table, totals))
    assert torch.equal(kept[0, 0].cpu(), torch.arange(1, 30000, dtype=torch.int32))


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("last", [0, 70])
def test_groups_with_any_share_kept(d, last):
    # of the i-th 128 tokens 4 i stay, then as many again of another order, then none
    pages, table, totals = pool([10 * 1024 + last], 64, 2, d, 9)
    stay = torch.zeros(2, 10 * 1024 + last)
    g = torch.Generator().manual_seed(3)
    for i in range(64):
        k = 4 * i if i < 32 else 128 - 4 * (i - 32)
        for h in range(2):
            stay[h, 128 * i + torch.randperm(128, generator=g)[:k]] = 1.0 + i
    tok = torch.arange(10 * 1024 + last)
    totals[table[0][tok // 64].long(), :, tok % 64] = stay.T.contiguous()
    budget = int((stay[0] > 0).sum())
    assert budget == int((stay[1] > 0).sum())
    for b in (budget, budget - 37, 36, 35, 1):
        check([10 * 1024 + last], 64, 2, d, b, state=(pages, table, totals))


def test_more_keys_than_shared_memory_holds():
    # 8 CTAs hold 49152 keys each: the rest is read again for every pass
    n = 8 * 49152 + 4321
    pages, table, totals = pool([n], 256, 1, 64, 7)
    p, t = pages.cuda(), totals.cuda()
    new, kept = moe.kv_evict(p, table.cuda(), i32([n]), 150000, totals=t, page_size=256, n_kv_heads=1, head_dim=64, first=5, recent=1000)
    tok = torch.arange(n)
    v = totals[table[0][tok // 256].long(), 0, tok % 256]
    mid = v[5:n - 1000].sort(descending=True, stable=True).indices[:150000 - 1005] + 5
    want = torch.cat([torch.arange(5), mid.sort().values, torch.arange(n - 1000, n)])
    assert torch.equal(kept[0, 0].cpu().long(), want) and new.tolist() == [150000]
    k = torch.arange(150000)
    assert torch.equal(rows(p.cpu(), table[0], 150000, 256, 1, 64), rows(pages, table[0], n, 256, 1, 64)[want])
    t = t.cpu()[table[0][tok // 256].long(), 0, tok % 256]
    assert torch.equal(t[k], v[want]) and not bool(t[150000:].any())


def test_more_keys_than_sixteen_ctas_hold():
    n, budget = 16 * 49152 + 4321, 300000
    pages, table, totals = pool([n], 1024, 1, 64, 8)
    p, t = pages.cuda(), totals.cuda()
    new, kept = moe.kv_evict(p, table.cuda(), i32([n]), budget, totals=t, page_size=1024, n_kv_heads=1, head_dim=64, first=5, recent=1000)
    tok = torch.arange(n)
    v = totals[table[0][tok // 1024].long(), 0, tok % 1024]
    mid = v[5:n - 1000].sort(descending=True, stable=True).indices[:budget - 1005] + 5
    want = torch.cat([torch.arange(5), mid.sort().values, torch.arange(n - 1000, n)])
    assert torch.equal(kept[0, 0].cpu().long(), want) and new.tolist() == [budget]
    k = torch.arange(budget)
    assert torch.equal(rows(p.cpu(), table[0], budget, 1024, 1, 64), rows(pages, table[0], n, 1024, 1, 64)[want])
    t = t.cpu()[table[0][tok // 1024].long(), 0, tok % 1024]
    assert torch.equal(t[k], v[want]) and not bool(t[budget:].any())


def test_more_sequences_than_lanes():
    lens = [(37 * i) % 400 for i in range(130)]
    check(lens, 32, 2, 64, 120, 2, 10, seed=8)


def test_wide_tables_and_no_eviction():
    check([100, 50], 32, 2, 64, 64, 4, 4, seed=9, width=4000)
    pages, table, totals = pool([100, 50], 32, 2, 64, 10)
    p, t, new, kept = check([100, 50], 32, 2, 64, 128, seed=10)
    assert torch.equal(p, pages) and torch.equal(t, totals)


def test_bad_pages_and_lengths_leave_a_sequence_as_it_is():
    lens, ps = [400, 300], 32
    pages, table, totals = pool(lens, ps, 2, 64, 11)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    good = check(lens, ps, 2, 64, 100, state=(pages, table, totals))
    own = table[1][:10].long()
    for bad_page, bad_len, bit in ((-1, 400, moe.MOE_KV_BAD_PAGE), (pages.shape[0], 400, moe.MOE_KV_BAD_PAGE),
                                   (None, -5, moe.MOE_KV_BAD_LENGTH), (None, 13 * 32 + 1, moe.MOE_KV_BAD_LENGTH)):
        t2 = table.clone()
        if bad_page is not None:
            t2[0, 12] = bad_page
        status.zero_()
        p, t = pages.cuda(), totals.cuda()
        new, kept = moe.kv_evict(p, t2.cuda(), i32([bad_len, 300]), 100, totals=t, page_size=ps, n_kv_heads=2, head_dim=64, status=status)
        assert int(status) == bit and new.tolist() == [bad_len, 100]
        assert bool((kept[0] == -1).all()) and torch.equal(kept[1], good[3][1])
        p, t = p.cpu(), t.cpu()
        assert torch.equal(p[own], good[0][own]) and torch.equal(t[own], good[1][own])
        p[own], t[own] = pages[own], totals[own]
        assert torch.equal(p, pages) and torch.equal(t, totals)


def test_two_at_once():
    # on streams of their own, each with its own cache, again and again
    cases = []
    for seed, (lens, d, budget) in enumerate((([5000, 3000, 9000], 128, 2500), ([20000], 64, 9000))):
        pages, table, totals = pool(lens, 64, 2, d, 20 + seed)
        want, after = expect(pages, table, totals, lens, budget, 4, 64, 64, 2, d)
        cases.append((lens, d, budget, pages.cuda(), table.cuda(), totals.cuda(), i32(lens), want, after, torch.cuda.Stream()))
    torch.cuda.synchronize()
    done = []
    for _ in range(6):
        for lens, d, budget, pages, table, totals, n, want, after, stream in cases:
            with torch.cuda.stream(stream):
                p, t = pages.clone(), totals.clone()
                new, kept = moe.kv_evict(p, table, n, budget, totals=t, page_size=64, n_kv_heads=2, head_dim=d, first=4, recent=64)
                done.append((lens, d, table, want, after, p, t, kept))
    torch.cuda.synchronize()
    for lens, d, table, want, after, p, t, kept in done:
        assert torch.equal(kept.cpu(), want)
        for s, n in enumerate(lens):
            tok, row = torch.arange(n), table[s].cpu()
            assert torch.equal(rows(p.cpu(), row, n, 64, 2, d), after[s][0])
            assert same(t.cpu()[row[tok // 64].long(), :, tok % 64], after[s][1])


def test_streams_and_graphs():
    lens, ps = [500, 130, 700], 64
    pages, table, totals = pool(lens, ps, 2, 128, 12)
    args = dict(page_size=ps, n_kv_heads=2, head_dim=128, first=4, recent=16)
    s = torch.cuda.Stream()
    p, t, tab, ln = pages.cuda(), totals.cuda(), table.cuda(), i32(lens)
    s.wait_stream(torch.cuda.current_stream())
    a = moe.kv_evict(p, tab, ln, 128, totals=t, stream=s, **args)
    torch.cuda.current_stream().wait_stream(s)
    want = check(lens, ps, 2, 128, 128, 4, 16, state=(pages, table, totals))
    assert torch.equal(p.cpu(), want[0]) and torch.equal(t.cpu(), want[1]) and torch.equal(a[1], want[3])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        new, kept = moe.kv_evict(p, tab, ln, 128, totals=t, **args)
    for n in ([500, 130, 700], [129, 128, 1], [0, 129, 300]):
        p.copy_(pages), t.copy_(totals), ln.copy_(i32(n))
        g.replay()
        want = check(n, ps, 2, 128, 128, 4, 16, state=(pages, table, totals))
        assert torch.equal(p.cpu(), want[0]) and torch.equal(t.cpu(), want[1]) and torch.equal(kept, want[3]) and torch.equal(new, want[2])


def test_refusals():
    pages, table, totals = pool([100], 32, 2, 64, 13)
    good = dict(pages=pages.cuda(), page_table=table.cuda(), seq_lens=i32([100]), budget=50, totals=totals.cuda(), page_size=32,
                n_kv_heads=2, head_dim=64)
    moe.kv_evict(**good)
    for bad in (dict(budget=-1), dict(first=-1), dict(recent=-1), dict(first=30, recent=21), dict(budget=1 << 31),
                dict(totals=good["totals"].half()), dict(totals=good["totals"][:, :1]), dict(totals=good["totals"].cpu()),
                dict(page_size=33), dict(head_dim=96), dict(n_kv_heads=4), dict(seq_lens=i32([100, 1])), dict(pages=pages),
                dict(status=torch.zeros(2, dtype=torch.int32, device="cuda"))):
        with pytest.raises(moe.MoeError):
            moe.kv_evict(**dict(good, **bad))
    new, kept = moe.kv_evict(**dict(good, page_table=table.cuda()[:0], seq_lens=i32([])))
    assert new.shape == (0,) and kept.shape == (0, 2, 50)
