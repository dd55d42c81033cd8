"""Routing on the GPU against a 64-bit statement (tests/route_ref.py), and the layer with a choice made before.

Choices are equal, whatever is near a border (gaps are at least 1e-13 in 64 bits, or ties).  Weights: expf is good to 2
steps (2^-22), its argument's rounding counts 2^-24 of the argument, the sum over E <= 1024 has 32 + 5 additions (2^-24
each), quotient and scale a step each: 2^-24 (64 + span) relative."""
import numpy as np
import pytest
import torch

import oracle
import router_softmax_top_gb300 as moe
import synth
from tests import route_ref as R
from tests.gpu_util import DECODE_TOL, pinned_store, row_rel_err

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def check(x, k, score="softmax", bias=None, groups=1, kept=None, group_score="top2", renorm=False, scale=1.0):
    """x: a cuda tensor [T, E]."""
    ids, w = moe.route(x, k, score=score, bias=bias, n_groups=groups, top_groups=kept, group_score=group_score,
                       renormalise=renorm, scale=scale)
    rid, rw, span = R.route(x.double().cpu().numpy(), k, score, None if bias is None else bias.double().cpu().numpy(), groups,
                            kept or groups, group_score, renorm, float(np.float32(scale)))
    assert np.array_equal(ids.cpu().numpy(), rid)
    got = w.cpu().double().numpy()
    tol = np.abs(rw) * (64 + span[:, None]) * 2.0 ** -24 + 1e-37
    assert (np.abs(got - rw) <= tol).all(), float((np.abs(got - rw) / tol).max())
    return ids, w


@pytest.mark.parametrize("T,E,k,groups,kept", [
    (1, 1, 1, 1, 1), (1, 128, 8, 1, 1), (3, 7, 7, 1, 1), (5, 33, 3, 1, 1), (64, 256, 8, 8, 4), (9, 60, 4, 4, 2),
    (17, 1024, 32, 32, 3), (4, 1000, 32, 10, 1), (6, 512, 32, 16, 16), (130, 96, 6, 3, 2), (2, 32, 32, 32, 32), (7, 160, 6, 8, 3)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("group_score", ["max", "top2"])
def test_choice_and_weights(T, E, k, groups, kept, score, group_score):
    g = torch.Generator().manual_seed(T * E + k)
    x = torch.randn(T, E, generator=g) * 2
    b = (torch.randn(E, generator=g) * 0.1).cuda()
    for i, dt in enumerate(DT.values()):
        for bias in (None, b):
            check(x.to(dt).cuda(), k, score, bias, groups, kept, group_score, renorm=(i + (bias is None)) % 2 == 0, scale=2.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k,groups,kept", [(128, 8, 1, 1), (256, 8, 8, 4), (1000, 32, 10, 5)])
def test_values_next_to_a_border(score, E, k, groups, kept):
    # the bias takes every value to the same one, but for its own rounding
    g = torch.Generator().manual_seed(E)
    x = torch.randn(1, E, generator=g)
    p = torch.softmax(x.double(), -1) if score == "softmax" else torch.sigmoid(x.double())
    bias = (0.75 - p[0]).float().cuda()
    for gs in ("max", "top2"):
        check(x.repeat(5, 1).cuda(), k, score, bias, groups, kept, gs)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_ties_go_to_the_lowest(score):
    for E, groups, kept in ((64, 1, 1), (64, 8, 3), (300, 4, 2)):
        zero = torch.zeros(3, E, device="cuda")
        for bias in (None, torch.zeros(E, device="cuda"), torch.full((E,), 0.3, device="cuda")):
            ids, _ = check(zero, 5, score, bias, groups, kept, renorm=True)
            assert torch.equal(ids, torch.arange(5, dtype=torch.int32, device="cuda").repeat(3, 1))
        # few distinct values; -0 and 0 are one value
        x = torch.randint(-1, 2, (40, E), generator=torch.Generator().manual_seed(1)).float()
        x = torch.where((x == 0) & (torch.rand(40, E, generator=torch.Generator().manual_seed(2)) < 0.5), -0.0, x).cuda()
        for bias in (None, torch.zeros(E, device="cuda")):
            check(x, 7, score, bias, groups, kept)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_large_and_small_logits(score):
    g = torch.Generator().manual_seed(3)
    for size in (1e-30, 1e-6, 30.0, 90.0, 1e4, 3e38):
        x = (torch.rand(9, 100, generator=g) * 2 - 1) * size
        check(x.cuda(), 6, score)
        if size < 100:
            check(x.cuda(), 6, score, None, 4, 2, "top2", renorm=True)
        # a bias of nothing: values are the scores, down to those that 32 bits do not hold
        if size in (30.0, 90.0) and score == "softmax":
            check(x.cuda(), 6, score, torch.zeros(100, device="cuda"))
    x = torch.randn(4, 64, generator=g)
    check(x.cuda(), 8, score, (torch.randn(64, generator=g) * 1e30).cuda(), 8, 2, "top2")
    check(x.cuda(), 8, score, torch.full((64,), 3e38).cuda(), 8, 2, "top2")


def test_logits_below_the_normal_numbers():
    g = torch.Generator().manual_seed(4)
    for E, k in ((100, 6), (1024, 32), (40, 32)):
        x = (torch.rand(5, E, generator=g) * 2 - 1) * 1e-40
        for y in (x, x.abs(), -x.abs()):
            check(y.cuda(), k)
            check(y.cuda(), min(k, 8), "sigmoid", None, 4, 2, "max")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,kept", [(1, 1), (8, 2)])
def test_closed_experts(score, groups, kept):
    g = torch.Generator().manual_seed(5)
    x = torch.randn(20, 64, generator=g)
    for t in range(20):
        x[t, torch.randperm(64, generator=g)[:3 * t + 5]] = -float("inf")
    x[18], x[19] = -float("inf"), -float("inf")
    x[18, 40] = 1.0
    b = (torch.randn(64, generator=g) * 0.1).cuda()
    for bias in (None, b):
        for gs in ("max", "top2"):
            for renorm in (False, True):
                _, w = check(x.cuda(), 6, score, bias, groups, kept, gs, renorm)
                assert bool((w[19] == 0).all())


def test_rows_that_make_no_sense():
    x = torch.randn(6, 40, device="cuda")
    x[1, 3], x[3, 39] = float("nan"), float("inf")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ids, w = moe.route(x, 4, status=status)
    bad = torch.tensor([False, True, False, True, False, False], device="cuda")
    assert torch.equal(w.isnan().all(1), bad) and torch.equal(w.isnan().any(1), bad)
    assert ids[1].tolist() == ids[3].tolist() == [0, 1, 2, 3]
    assert int(status) == moe.MOE_ROUTE_BAD_LOGIT and "logit" in moe.status_message(status)
    ok, _ = moe.route(torch.where(bad[:, None], 0.0, x), 4)
    assert torch.equal(ids[~bad], ok[~bad])
    status.zero_()
    for v in (float("nan"), float("inf"), -float("inf")):
        b = torch.zeros(40, device="cuda")
        b[7] = v
        assert bool(moe.route(x, 4, bias=b, status=status)[1].isnan().all())
    assert int(status) == moe.MOE_ROUTE_BAD_LOGIT


def test_strides_streams_and_graphs():
    big = torch.randn(11, 300, device="cuda")
    for lo, n in ((0, 128), (3, 128), (1, 67), (100, 200)):
        check(big[:, lo:lo + n], 5, "sigmoid")
    check(big.bfloat16()[::3, 8:136], 5)
    x = torch.randn(33, 256, device="cuda")
    want = moe.route(x, 8, n_groups=8, top_groups=3)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = moe.route(x, 8, n_groups=8, top_groups=3, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    ids, w = torch.empty_like(want[0]), torch.empty_like(want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.route(x, 8, n_groups=8, top_groups=3, ids_out=ids, weights_out=w)
    for seed in range(3):
        x.copy_(torch.randn(33, 256, generator=torch.Generator().manual_seed(seed)))
        g.replay()
        assert all(torch.equal(a, b) for a, b in zip((ids, w), moe.route(x, 8, n_groups=8, top_groups=3)))
    empty = moe.route(x[:0], 8)
    assert empty[0].shape == (0, 8) and empty[1].shape == (0, 8)


def test_refusals():
    x = torch.randn(4, 64, device="cuda")
    for bad in (dict(top_k=0), dict(top_k=33), dict(top_k=65), dict(n_groups=5), dict(n_groups=64), dict(n_groups=8, top_groups=9),
                dict(n_groups=8, top_groups=0), dict(n_groups=8, top_groups=1, top_k=9), dict(score="relu"),
                dict(group_score="mean"), dict(scale=float("nan")), dict(scale=float("inf")),
                dict(bias=torch.zeros(63, device="cuda")), dict(bias=torch.zeros(64)), dict(bias=torch.zeros(64, device="cuda").half()),
                dict(ids_out=torch.zeros(4, 8, device="cuda")), dict(weights_out=torch.zeros(4, 7, device="cuda")),
                dict(top_k=1 << 40)):
        kw = dict(dict(top_k=8), **bad)
        with pytest.raises(moe.MoeError):
            moe.route(x, kw.pop("top_k"), **kw)
    for y in (x.cpu(), x.double(), x[0], x.t()):
        with pytest.raises(moe.MoeError):
            moe.route(y, 2)
    with pytest.raises(moe.MoeError):
        moe.route(torch.randn(2, 1025, device="cuda"), 2)


# ------------------------------------------------------------------- the layer with a choice made before
def _cache(store, sh, **kw):
    return moe.MoECache(n_layers=sh[0], n_experts=sh[1], top_k=sh[2], hidden=sh[3], ffn=sh[4], store=store, **kw)


@pytest.mark.parametrize("T,S,kw", [
    (1, 8, dict(fill_mode=1)), (4, 16, dict(fill_mode=1)), (4, 16, dict(fill_mode=0)), (4, 8, dict(fill_mode=1)),
    (1, 8, dict(fill_mode=1, policy=1)), (7, 4, dict(fill_mode=0, policy=2)), (40, 8, dict(fill_mode=1)),
    (40, 16, dict(fill_mode=0, act_dtype="bf16", gemm_min_tokens=16)), (300, 16, dict(fill_mode=1, act_dtype="bf16", gemm_min_tokens=16))])
def test_the_routers_own_choice_gives_the_same_layer(T, S, kw):
    sh = (2, 16, 4, 256, 512)
    store = pinned_store(*sh[:2], *sh[3:], seed=3)
    a, b = (_cache(store, sh, slots_per_layer=S, max_tokens=T, **kw) for _ in range(2))
    g = torch.Generator().manual_seed(T)
    for step in range(4):
        logits, x = torch.randn(T, 16, generator=g).cuda(), torch.randn(T, 256, generator=g).cuda()
        if kw.get("act_dtype") == "bf16":
            x = x.bfloat16()
        want = a.forward(step % 2, logits, x)
        plan = a.last_plan(step % 2, T)
        ids, w = torch.from_numpy(plan["ids"]).cuda(), torch.from_numpy(plan["w"]).cuda()
        got = b.forward_routed(step % 2, ids, w, x)
        assert torch.equal(want, got)
        other = b.last_plan(step % 2, T)
        assert all(np.array_equal(plan[n], other[n]) for n in ("ids", "w", "gpu_slot", "stage", "miss_expert", "miss_slot"))
        rid, rw = moe.route(logits, 4)
        assert torch.equal(rid, ids)
        np.testing.assert_allclose(rw.cpu(), plan["w"], rtol=2e-6)
    assert a.sync() == b.sync() == moe.MOE_OK
    assert a.stats() == b.stats()
    a.close(), b.close()


def test_grouped_routing_and_the_experts_products():
    L, E, k, H, F = 1, 16, 4, 256, 512
    store = pinned_store(L, E, H, F, seed=4)
    c = _cache(store, (L, E, k, H, F), slots_per_layer=8, max_tokens=4, fill_mode=1)
    eb = synth.expert_bytes(H, F)
    blocks = store.numpy().reshape(E, eb)
    g = torch.Generator().manual_seed(9)
    for _ in range(3):
        logits, x = torch.randn(4, E, generator=g), torch.randn(4, H, generator=g)
        bias = torch.randn(E, generator=g) * 0.2
        ids, w = moe.route(logits.cuda(), k, score="sigmoid", bias=bias.cuda(), n_groups=4, top_groups=2, renormalise=True, scale=2.0)
        out = c.forward_routed(0, ids, w, x.cuda())
        rid, rw, _ = R.route(logits.double().numpy(), k, "sigmoid", bias.double().numpy(), 4, 2, "top2", True, 2.0)
        assert np.array_equal(ids.cpu().numpy(), rid)
        want = np.stack([sum(rw[t, q] * oracle.expert_ffn(blocks[rid[t, q]], H, F, x[t].double().numpy()) for q in range(k))
                         for t in range(4)])
        assert row_rel_err(out.cpu().numpy(), want).max() <= DECODE_TOL
    assert c.sync() == moe.MOE_OK
    c.close()


@pytest.mark.parametrize("T", [1, 3, 20])
@pytest.mark.parametrize("what", ["high", "low", "twice", "nan"])
def test_choices_that_make_no_sense(T, what):
    sh = (1, 16, 4, 256, 512)
    store = pinned_store(1, 16, 256, 512, seed=5)
    c = _cache(store, sh, slots_per_layer=16, max_tokens=T, fill_mode=1)
    ids = torch.arange(4, dtype=torch.int32, device="cuda").repeat(T, 1)
    w, x = torch.full((T, 4), 0.25, device="cuda"), torch.randn(T, 256, device="cuda")
    c.forward_routed(0, ids, w, x)
    assert c.sync() == moe.MOE_OK
    if what == "nan":
        w[T - 1, 3] = float("nan")
    else:
        ids[T - 1, 3] = {"high": 16, "low": -1, "twice": 1}[what]
    try:
        c.forward_routed(0, ids, w, x)
        assert c.sync() == moe.MOE_ERR_INVALID_ARG
    except moe.MoeError as e:
        assert e.code == moe.MOE_ERR_INVALID_ARG
    with pytest.raises(moe.MoeError):
        c.forward_routed(0, ids.clamp(0, 3), w, x)
    assert c.stats()["poisoned"]
    c.close()
