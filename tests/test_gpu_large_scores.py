"""Scores of any finite size, and the scales that are refused.

Where the scores of a row lie further apart than the weights can tell, all the weight is one key's, and the result is its
value (exactly a weight of 1, rounded once)."""
import pytest
import torch

import router_softmax_top_gb300 as moe
from tests.test_gpu_kv_numerics import cached, i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("top", [2.0 ** 110, 2.0 ** 119, 2.0 ** 120, 3e38])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_queries_of_any_finite_size(top, d):
    # far apart, or all 0, which shares the weight evenly
    n = 300
    g = torch.Generator(device="cuda").manual_seed(d)
    v = torch.randn(n, 1, d, generator=g, device="cuda")
    k = torch.zeros(n, 1, d, device="cuda")
    k[:, 0, :32] = 2.0 ** -10 * (torch.randperm(n, generator=g, device="cuda") + 1)[:, None] / n
    pages, table = cached(k, v)
    q = torch.zeros(1, 3, d, device="cuda")
    q[0, 0, :32], q[0, 1, 40], q[0, 2, :32] = top, -top, 1.0
    q = q.bfloat16()
    out, lse = moe.kv_attention(q, pages, table, i32([n]), page_size=64, n_kv_heads=1, return_lse=True)
    kr, vr = [x[:, 0].double() for x in moe.kv_read(pages, table, i32([0]), i32([0, n]), n, page_size=64, n_kv_heads=1,
                                                    head_dim=d, dtype=torch.float32)]
    best = int(kr[:, 0].argmax())
    assert bool(((out[0, 0].double() - vr[best]).abs() <= 2.0 ** -8 * vr[best].abs() + 2.0 ** -10 * vr[best].abs()).all())
    mean, size = vr.mean(0), vr.abs().mean(0)
    assert bool(((out[0, 1].double() - mean).abs() <= 2.0 ** -8 * mean.abs() + 2.0 ** -10 * size).all())
    assert bool(torch.isfinite(out).all()) and bool(torch.isfinite(lse).all())
    assert float(lse[0, 0]) == pytest.approx(float(kr[best] @ q[0, 0].double()) * d ** -0.5, rel=2.0 ** -14)


@pytest.mark.parametrize("scale", [2.5e38, 3.4e38])
def test_scales_whose_exponent_overflows_are_refused(scale):
    pages, table = cached(*[torch.randn(40, 1, 64, device="cuda") for _ in range(2)])
    q = torch.zeros(1, 2, 64, device="cuda").bfloat16()
    with pytest.raises(moe.MoeError):
        moe.kv_attention(q, pages, table, i32([40]), page_size=64, n_kv_heads=1, scale=scale)
    with pytest.raises(moe.MoeError):
        moe.prompt_attention(q, q[:, :1], q[:, :1], i32([0, 1]), scale=scale)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("dtype,size", [(torch.bfloat16, 3e4), (torch.bfloat16, 1e10), (torch.bfloat16, 3e38), (torch.float16, 60000.0)])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("n,m", [(200, 200), (3, 200)])
def test_prompts_of_any_finite_size(d, dtype, size, sign, n, m):
    g = torch.Generator(device="cuda").manual_seed(d)
    c = (torch.randperm(m, generator=g, device="cuda") + 1).float()          # whole numbers: exact in both types
    k = (c * (2.0 ** -20 if size > 1e30 else 1.0))[:, None, None].expand(m, 1, d).to(dtype).contiguous()
    v = torch.randn(m, 1, d, generator=g, device="cuda").to(dtype)
    q = torch.full((n, 2, d), sign * size, device="cuda").to(dtype)
    q[:, 1] = 0                                                              # a head beside it whose scores are 0
    cu_q, cu_k = i32([0, n]), i32([0, m])
    out, lse = moe.prompt_attention(q, k, v, cu_q, cu_k, return_lse=True)
    for i in range(n):
        hi = m - n + i + 1
        best = int((sign * c[:hi]).argmax())
        assert torch.equal(out[i, 0], v[best, 0]), i
        mean, mag = v[:hi, 0].double().mean(0), v[:hi, 0].double().abs().mean(0)
        u = torch.finfo(dtype).eps / 2
        assert bool(((out[i, 1].double() - mean).abs() <= u * mean.abs() + (u + 2.0 ** -12) * mag).all()), i
    assert bool(torch.isfinite(lse).all())
