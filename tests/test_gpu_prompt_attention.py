"""Causal attention over packed prompts on the GPU, against a plain 64-bit statement.

Tolerance.  With p the weights, A = sum p |v| / sum p and Z = max_j scale sum_d |q_d k_jd|
of a row: the kernel rounds each weight to the inputs' type (half a step, u), sums
D products in fp32 (2^-18 Z covers D = 256) and rounds the result once, so
|error| <= A (u + 2^-12 + 2^-17 Z) + u |result|."""
import pytest
import torch

import router_softmax_top_gb300 as moe
from tests import attention_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _seeded():
    torch.manual_seed(21)

DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def cu_of(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def inputs(nq, nk, hq, hkv, d, dt, seed, fused=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda n, h: torch.randn(n, h, d, generator=g, device="cuda").to(dt)  # noqa: E731
    if fused:
        return r(nq, hq + 2 * hkv).split([hq, hkv, hkv], 1)
    return r(nq, hq), r(nk, hkv), r(nk, hkv)


def check(q, k, v, lens, keys, window, rows=None):
    d = q.shape[2]
    out, lse = moe.prompt_attention(q, k, v, i32(cu_of(lens)), i32(cu_of(keys)), window=window, return_lse=True)
    o, l = out.cpu().double(), lse.cpu().double()
    qd, kd, vd = q.cpu().double(), k.cpu().double(), v.cpu().double()
    a = b = 0
    u = R.EPS[q.dtype]
    for n, m in zip(lens, keys):
        at = [m - n + i for i in range(n)]
        pick = list(range(n)) if rows is None or n <= rows else sorted({0, 1, 63, 64, 127, 128, n // 2, n - 2, n - 1})
        ix = torch.tensor([a + i for i in pick], dtype=torch.long)
        ro, rl, mag, z = R.attend(qd[ix], kd[b:b + m], vd[b:b + m], [at[i] for i in pick], m, d ** -0.5, window)
        tol = mag * (u + 2.0 ** -12 + 2.0 ** -17 * z[..., None]) + u * ro.abs() + 1e-30
        err = (o[ix] - ro).abs()
        assert bool((err <= tol).all()), (n, m, float((err / tol).max()))
        empty = torch.isinf(rl)
        assert torch.equal(torch.isinf(l[ix]) & (l[ix] < 0), empty)
        assert not bool(((l[ix] - rl).abs()[~empty] > (2.0 ** -17 * z + 2.0 ** -20 * (1 + rl.abs()))[~empty]).any())
        a, b = a + n, b + m
    return out, lse


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("hq,hkv,lens,extra,window", [
    (1, 1, [1], 0, 0),
    (4, 2, [37], 0, 0),
    (8, 2, [0, 1, 2, 31, 33, 64, 0, 65], 0, 0),
    (3, 1, [130, 129], 0, 0),
    (7, 1, [40, 300], 0, 0),
    (5, 5, [128, 256], 0, 0),
    (16, 1, [100], 0, 0),
    (4, 1, [17, 200], 333, 0),
    (4, 2, [150, 3], 0, 1),
    (4, 2, [300], 0, 50),
    (2, 1, [90, 260], 200, 130),
    (64, 1, [9], 40, 0)])
def test_prompts(d, dtype, hq, hkv, lens, extra, window):
    keys = [n + extra for n in lens]
    q, k, v = inputs(sum(lens), sum(keys), hq, hkv, d, DT[dtype], d + len(lens), fused=extra == 0)
    check(q, k, v, lens, keys, window)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_long_prompts(d):
    lens = [1500, 2300]
    q, k, v = inputs(sum(lens), sum(lens), 4, 2, d, torch.bfloat16, 3)
    a, la = check(q, k, v, lens, lens, 0, rows=10)
    for _ in range(3):
        b, lb = moe.prompt_attention(q, k, v, i32(cu_of(lens)), return_lse=True)
        assert torch.equal(a, b) and torch.equal(la, lb)
    check(q, k, v, lens, lens, 700, rows=10)


def test_fewer_keys_than_queries():
    # the first queries stand before the first key and see nothing
    q, k, v = inputs(50, 20, 4, 2, 64, torch.float16, 5)
    out, _ = check(q, k, v, [50], [20], 0)
    assert not bool(out[:30].any())
    q, k, v = inputs(8, 1, 4, 2, 128, torch.bfloat16, 5)
    out, lse = moe.prompt_attention(q, k[:0], v[:0], i32([0, 8]), i32([0, 0]), return_lse=True)
    assert not bool(out.any()) and bool((lse == -float("inf")).all())


def test_scores_far_apart_move_the_reference():
    n, d = 700, 128
    q, k, v = inputs(n, n, 2, 1, d, torch.bfloat16, 6)
    k = (k.float() * (1 + torch.arange(n, device="cuda") / 20)[:, None, None]).bfloat16()
    check((q.float() * 3).bfloat16(), k, v, [n], [n], 0)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_what_a_row_does_not_see_does_not_reach_it(d, value):
    lens = [150, 77]
    q, k, v = inputs(227, 227, 4, 2, d, torch.bfloat16, 7)
    clean = moe.prompt_attention(q, k, v, i32(cu_of(lens)))
    k2, v2 = k.clone(), v.clone()
    k2[100], v2[100] = value, value          # a later token of the first prompt
    got = moe.prompt_attention(q, k2, v2, i32(cu_of(lens)))
    near = R.EPS[torch.bfloat16] * 4
    assert bool(((got[:100].float() - clean[:100].float()).abs() <= near * (1 + clean[:100].float().abs())).all())
    assert bool((~torch.isfinite(got[100:150].float())).all())
    assert torch.equal(got[150:], clean[150:])   # and no row of the next prompt
    v2 = v.clone()
    v2[150:] = value                          # the next prompt's values, in the same tile of keys
    got = moe.prompt_attention(q, k, v2, i32(cu_of(lens)))
    assert bool(((got[:150].float() - clean[:150].float()).abs() <= near * (1 + clean[:150].float().abs())).all())
    if value == float("inf"):                 # a seen infinity is an infinity
        v2 = v.clone()
        v2[3, 0, 5] = value
        got = moe.prompt_attention(q, k, v2, i32(cu_of(lens)))
        assert bool(torch.isinf(got[3:150, :2, 5]).all()) and bool(torch.isfinite(got[3:150, :2, 6].float()).all())
    # outside the window
    k2, v2 = k.clone(), v.clone()
    k2[:20], v2[:20] = value, value
    w = moe.prompt_attention(q, k, v, i32(cu_of(lens)), window=30)
    got = moe.prompt_attention(q, k2, v2, i32(cu_of(lens)), window=30)
    assert bool(((got[49:].float() - w[49:].float()).abs() <= near * (1 + w[49:].float().abs())).all())


# Few rows with many keys: the keys of a tile are shared out over several CTAs, whose sums the last one joins (each join
# rounds in fp32, 2^-24 per part and so within the 2^-12 above).
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("d,hq,hkv,lens,extra,window", [
    (128, 8, 2, [5], 9000, 0),
    (64, 6, 2, [37], 3000, 0),
    (256, 4, 1, [1], 5001, 0),
    (256, 16, 4, [130], 2000, 0),
    (128, 4, 4, [300, 0, 2, 65], 1800, 0),
    (64, 3, 1, [1, 90, 700], 2500, 1024),
    (128, 7, 1, [33, 40], 4100, 1500),
    (128, 64, 1, [9, 3], 3333, 0)])
def test_keys_shared_out(d, dtype, hq, hkv, lens, extra, window):
    keys = [n + extra if n else 0 for n in lens]
    q, k, v = inputs(sum(lens), sum(keys), hq, hkv, d, DT[dtype], d + len(lens))
    ws = moe.prompt_attention_workspace(sum(lens), hq, sum(keys), hkv, d, len(lens), window)
    assert ws is not None                     # these sizes do share
    a, la = check(q, k, v, lens, keys, window)
    for own in (None, ws, ws):                # a result does not depend on which part is done last
        b, lb = moe.prompt_attention(q, k, v, i32(cu_of(lens)), i32(cu_of(keys)), window=window, return_lse=True,
                                     workspace=own)
        assert torch.equal(a, b) and torch.equal(la, lb)
    assert not bool(ws[:moe.MOE_KV_COUNTER_BYTES].any())


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_shared_keys_that_a_row_does_not_see(d, value):
    n, m = 40, 3000
    q, k, v = inputs(n, m, 4, 2, d, torch.bfloat16, 11)
    cu_q, cu_k = i32([0, n]), i32([0, m])
    assert moe.prompt_attention_workspace(n, 4, m, 2, d, 1, 2000) is not None
    clean = moe.prompt_attention(q, k, v, cu_q, cu_k, window=2000)
    near = R.EPS[torch.bfloat16] * 4
    k2, v2 = k.clone(), v.clone()
    k2[:970], v2[:970] = value, value         # before the window of all rows from 9 on, in its first block
    k2[m - 5:], v2[m - 5:] = value, value     # after all rows but the last five
    got = moe.prompt_attention(q, k2, v2, cu_q, cu_k, window=2000)
    assert bool(((got[9:n - 5].float() - clean[9:n - 5].float()).abs() <= near * (1 + clean[9:n - 5].float().abs())).all())
    assert bool((~torch.isfinite(got[n - 5:].float())).all())
    if value == float("inf"):                 # a seen infinity is an infinity
        v2 = v.clone()
        v2[2000, 0, 5] = value
        got = moe.prompt_attention(q, k, v2, cu_q, cu_k)
        assert bool(torch.isinf(got[:, :2, 5]).all()) and bool(torch.isfinite(got[:, :2, 6].float()).all())


def test_shared_keys_in_graphs_and_streams():
    n, m = 20, 4000
    q, k, v = inputs(n, m, 8, 2, 128, torch.bfloat16, 12)
    cu_q, cu_k = i32([0, n]), i32([0, m])
    want = moe.prompt_attention(q, k, v, cu_q, cu_k)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = moe.prompt_attention(q, k, v, cu_q, cu_k, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        one = moe.prompt_attention(q, k, v, cu_q, cu_k)
        two = moe.prompt_attention(one, k, v, cu_q, cu_k)
    for _ in range(2):
        q.mul_(0.5)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(one, moe.prompt_attention(q, k, v, cu_q, cu_k))
        assert torch.equal(two, moe.prompt_attention(one, k, v, cu_q, cu_k))


def test_workspaces_that_are_refused():
    n, m = 20, 4000
    q, k, v = inputs(n, m, 8, 2, 128, torch.bfloat16, 12)
    cu_q, cu_k = i32([0, n]), i32([0, m])
    ws = moe.prompt_attention_workspace(n, 8, m, 2, 128, 1)
    for bad in (ws[:-256], ws[128:], ws.cpu(), ws[::2]):
        with pytest.raises(moe.MoeError):
            moe.prompt_attention(q, k, v, cu_q, cu_k, workspace=bad)
    # sizes that do not share need none: few keys, many rows, many sequences
    assert moe.prompt_attention_workspace(n, 8, 200, 2, 128, 1) is None
    assert moe.prompt_attention_workspace(1 << 20, 8, 1 << 20, 2, 128, 1) is None
    assert moe.prompt_attention_workspace(n, 8, m, 2, 128, 33) is None


def test_bad_offsets_are_reported():
    q, k, v = inputs(100, 100, 4, 2, 64, torch.bfloat16, 8)
    clean = moe.prompt_attention(q, k, v, i32([0, 40, 100]))
    for cu_q, cu_k, same, dead in (([0, 40, 101], [0, 40, 100], slice(0, 40), None),
                                   ([0, 40, 20], [0, 40, 100], slice(0, 40), None),
                                   ([-5, 40, 100], [0, 40, 100], slice(40, 100), None),
                                   ([0, 40, 100], [0, 40, 101], slice(0, 40), slice(40, 100)),
                                   ([0, 40, 100], [0, 200, 100], slice(0, 0), slice(0, 100)),
                                   ([0, 40, 100], [-1, 40, 100], slice(40, 100), slice(0, 40))):
        status, out = i32([0]), torch.zeros_like(clean)
        moe.prompt_attention(q, k, v, i32(cu_q), i32(cu_k), out=out, status=status)
        assert int(status) == moe.MOE_KV_BAD_LENGTH
        assert torch.equal(out[same], clean[same])
        if dead is not None:
            assert bool(torch.isnan(out[dead]).all())


def test_many_short_prompts_and_streams():
    lens = [1 + i % 5 for i in range(400)]
    n = sum(lens)
    q, k, v = inputs(n, n, 4, 4, 128, torch.float16, 9)
    want, _ = check(q, k, v, lens, lens, 0)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = moe.prompt_attention(q, k, v, i32(cu_of(lens)), stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    cu = i32(cu_of(lens))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        res = moe.prompt_attention(q, k, v, cu)
    q.mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(res, moe.prompt_attention(q, k, v, cu))


def test_python_refusals():
    q, k, v = inputs(10, 10, 4, 2, 64, torch.bfloat16, 1)
    cu = i32([0, 10])
    for bad in (lambda: moe.prompt_attention(q.float(), k, v, cu), lambda: moe.prompt_attention(q, k.half(), v, cu),
                lambda: moe.prompt_attention(q, k, v[:5], cu), lambda: moe.prompt_attention(q, k, v, cu.long()),
                lambda: moe.prompt_attention(q, k, v, cu, i32([0, 5, 10])), lambda: moe.prompt_attention(q[:, :3], k, v, cu),
                lambda: moe.prompt_attention(q, k, v, cu, scale=0.0), lambda: moe.prompt_attention(q, k, v, cu, window=-1),
                lambda: moe.prompt_attention(q.cpu(), k, v, cu), lambda: moe.prompt_attention(q, k, v, cu[:0]),
                lambda: moe.prompt_attention(q, k, v, cu, out=torch.empty(10, 4, 64, device="cuda"))):
        with pytest.raises(moe.MoeError):
            bad()
    assert moe.prompt_attention(q[:0], k, v, cu).shape == (0, 4, 64)
