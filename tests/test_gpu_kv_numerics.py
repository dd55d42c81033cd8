"""Attention over the 4-bit cache where scales and weights lie far apart, against 64 bits on the GPU.

Bound.  Of a row with weights w_j (sum 1), a product of a weight with a value's scale is
rounded once to fp16: off by at most 2^-11 of itself, or by 2^-25 of the unit in which the
row's largest such product is at least 2^10.  A value is at most 8 scales, so n keys are off by at
most n 2^-35 T beside the relative part, T = max_j w_j max_d |v_jd|; where T is below 2^-70 of the
weights the unit is tied to the largest weight instead, n 2^-92.  Scores are fp32 sums (2^-17 Z, Z = max_j
scale sum |q k|), the result is rounded once.  Hence
|error| <= sum_j w_j |v_j| (2^-11 + 2^-12 + 2^-17 Z) + n (2^-35 T + 2^-92) + half a step of the result.
(Beside that the accumulators' own rounding, where single keys of exact value 0 have most of the weight: see
tests/test_gpu_kv_ragged.py.)"""
import pytest
import torch

import router_softmax_top_gb300 as moe
from tests import attention_ref as R

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float16]
LEAST = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}     # half a step of results below the normal numbers


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def cached(k, v, ps=64):
    """A cache of one sequence."""
    n, hkv, d = k.shape
    pages = moe.kv_pages(-(-n // ps), hkv, d, ps)
    table = torch.randperm(pages.shape[0], generator=torch.Generator().manual_seed(n)).to(torch.int32)[None].cuda()
    moe.kv_append(pages, table, i32([0]), i32([0, n]), k, v, page_size=ps)
    return pages, table


def check(q, pages, table, n, hkv, ps=64, window=0, scale=1.0, z_extra=0.0):
    d, hq, rows = q.shape[2], q.shape[1], q.shape[0]
    out, lse = moe.kv_attention(q, pages, table, i32([n]), page_size=ps, n_kv_heads=hkv, q_tokens=rows, window=window,
                                scale=scale, return_lse=True)
    k, v = [x.double() for x in moe.kv_read(pages, table, i32([0]), i32([0, n]), n, page_size=ps, n_kv_heads=hkv, head_dim=d,
                                            dtype=torch.float32)]
    for r in range(rows):
        at = n - rows + r
        lo = max(0, at - window + 1) if window else 0
        for h in range(hq):
            kk, vv = k[lo:at + 1, h * hkv // hq], v[lo:at + 1, h * hkv // hq]
            s = kk @ q[r, h].double() * scale
            z = float((kk.abs() @ q[r, h].double().abs()).max()) * scale
            w = torch.softmax(s, 0)
            ref, mag, top = w @ vv, w @ vv.abs(), float((w * vv.abs().amax(1)).max())
            m = len(w)
            tol = mag * (2.0 ** -11 + 2.0 ** -12 + 2.0 ** -17 * z) + m * (2.0 ** -35 * top + 2.0 ** -92)
            tol = tol + torch.clamp(R.EPS[q.dtype] * ref.abs(), min=LEAST[q.dtype])
            err = (out[r, h].double() - ref).abs()
            assert bool((err <= tol).all()), (r, h, float((err / tol).max()))
            want = float(torch.logsumexp(s, 0))
            assert abs(float(lse[r, h]) - want) <= 2.0 ** -17 * z + 2.0 ** -20 * (1 + abs(want))
    return out


def scored(t, d, hkv=1):
    """Keys whose score with a query of ones is t (exactly where t / 32 is one of a block's codes)."""
    k = torch.zeros(len(t), hkv, d, device="cuda")
    k[:, :, :32] = (t / 32)[:, None, None]
    return k


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("outlier", [0.0, 1.0, 5e5])
def test_many_small_weights_beside_a_large_one_and_a_large_value(d, dtype, outlier):
    # a key of weight one third, 65536 of 2^-15 of it, and one of no weight whose value's scale is the largest there is
    n = 65600
    g = torch.Generator(device="cuda").manual_seed(d)
    t = torch.full((n,), 0.0, device="cuda")
    t[3], t[40000] = 10.5, -60.0
    v = 0.5 + 0.25 * torch.randn(n, 1, d, generator=g, device="cuda")
    v[40000] = outlier
    pages, table = cached(scored(t, d), v)
    check(torch.ones(1, 2, d, device="cuda", dtype=dtype), pages, table, n, 1)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("every", [1, 32, 33])
def test_large_values_of_no_weight_in_many_tiles(dtype, every):
    n, d = 20000, 128
    g = torch.Generator(device="cuda").manual_seed(every)
    t = torch.zeros(n, device="cuda")
    t[5] = 9.0
    v = 0.5 + 0.25 * torch.randn(n, 1, d, generator=g, device="cuda")
    if every > 1:
        t[7::every], v[7::every, :, :32] = -50.0, 4e5
    pages, table = cached(scored(t, d), v)
    check(torch.ones(1, 1, d, device="cuda", dtype=dtype), pages, table, n, 1)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("size", [2.0 ** -18, 2.0 ** -12, 2.0 ** -6])
@pytest.mark.parametrize("heavy", [0.0, 1.0])
def test_small_values_of_small_weights(dtype, size, heavy):
    # a heavy first key, of value 0 or like the others, and 30000 light ones whose values are small
    n, d = 30000, 64
    g = torch.Generator(device="cuda").manual_seed(7)
    t = torch.zeros(n, device="cuda")
    t[0] = 14.0
    v = size * (1 + 0.5 * torch.randn(n, 1, d, generator=g, device="cuda"))
    v[0] *= heavy
    pages, table = cached(scored(t, d), v)
    check(torch.ones(1, 2, d, device="cuda", dtype=dtype), pages, table, n, 1)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", [64, 256])
@pytest.mark.parametrize("heavy", [30.0, 100.0, 400.0])
def test_the_heaviest_key_has_no_value(dtype, d, heavy):
    n = 900
    g = torch.Generator(device="cuda").manual_seed(8)
    t = torch.randn(n, generator=g, device="cuda")
    t[100] = heavy
    v = torch.randn(n, 1, d, generator=g, device="cuda")
    v[100] = 0
    pages, table = cached(scored(t, d), v)
    check(torch.ones(1, 1, d, device="cuda", dtype=dtype), pages, table, n, 1)


@pytest.mark.parametrize("dtype", DTYPES)
def test_no_values_at_all_then_some(dtype):
    n, d = 700, 128
    t = torch.linspace(-20, 20, n, device="cuda")
    v = torch.zeros(n, 1, d, device="cuda")
    v[650:] = torch.randn(50, 1, d, device="cuda", generator=torch.Generator(device="cuda").manual_seed(9))
    pages, table = cached(scored(t, d), v)
    check(torch.ones(1, 1, d, device="cuda", dtype=dtype), pages, table, n, 1)
    check(torch.ones(1, 1, d, device="cuda", dtype=dtype), pages, table, 640, 1)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", [64, 128, 256])
def test_large_values_that_a_row_does_not_see(dtype, d):
    n, ps = 70, 32
    g = torch.Generator(device="cuda").manual_seed(d)
    k, v = [torch.randn(n, 1, d, generator=g, device="cuda") for _ in range(2)]
    q = torch.randn(2, 4, d, generator=g, device="cuda").to(dtype)
    kw = dict(page_size=ps, n_kv_heads=1, q_tokens=2, return_lse=True)
    for window, hidden in ((20, slice(33, 48)), (20, slice(0, 49)), (0, slice(0, 0))):
        pages, table = cached(k, v, ps)
        clean = moe.kv_attention(q, pages, table, i32([n]), window=window, **kw)
        after = torch.full_like(v[:20], 3e5)
        pages, table = cached(torch.cat([k, after]), torch.cat([v, after]), ps)     # and after the sequence
        v2, k2 = v.clone(), k.clone()
        v2[hidden], k2[hidden] = -4e5, 1e4
        moe.kv_append(pages, table, i32([0]), i32([0, n]), k2, v2, page_size=ps)
        got = moe.kv_attention(q, pages, table, i32([n]), window=window, **kw)
        assert torch.equal(got[0], clean[0]) and torch.equal(got[1], clean[1])
        # the last token, which the second row sees and the first one does not
        v2, k2 = v2.clone(), k2.clone()
        v2[n - 1], k2[n - 1] = 4e5, 50 * q[1, 0].float()
        moe.kv_append(pages, table, i32([0]), i32([0, n]), k2, v2, page_size=ps)
        got = moe.kv_attention(q, pages, table, i32([n]), window=window, **kw)
        assert torch.equal(got[0][0], clean[0][0]) and torch.equal(got[1][0], clean[1][0])
        assert not torch.equal(got[0][1], clean[0][1])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", [64, 70])
def test_a_value_that_is_not_finite_shows_whatever_its_weight(dtype, n):
    # in a tile that the row sees whole, and in one that it sees in part
    d, at = 64, n - 3
    t = torch.zeros(n, device="cuda")
    t[at] = -80.0
    v = torch.randn(n, 1, d, device="cuda", generator=torch.Generator(device="cuda").manual_seed(n))
    v[at, 0, 40] = float("nan")
    pages, table = cached(scored(t, d), v, 32)
    out = moe.kv_attention(torch.ones(1, 1, d, device="cuda", dtype=dtype), pages, table, i32([n]), page_size=32,
                           n_kv_heads=1, scale=1.0)
    assert bool(torch.isnan(out[0, 0, 32:]).all()) and bool(torch.isfinite(out[0, 0, :32]).all())
