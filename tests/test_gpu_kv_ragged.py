"""Attention over the cache for ragged batches of every size, type and window, log-sums among the outputs, against 64 bits on
the GPU.  Tolerances: those of tests/test_gpu_kv_cache.py, the part that is not relative as tests/test_gpu_kv_numerics.py
has it; and, as a value's code passes through the accumulators as it is and its -8 as a product of its own, sums of up to
16 w d (w a weight, d its value's scale) are rounded in fp32, four times per 32 keys: 2^-16 sum_j w_j d_j covers that
(queries of the first rows are the first keys here, so that single keys have most of the weight)."""
import pytest
import torch

import router_softmax_top_gb300 as moe
from tests import attention_ref as R
from tests.test_gpu_kv_cache import filled, i32

pytestmark = pytest.mark.gpu


def check(lens, d, hq, hkv, q_tokens, window, dtype, seed):
    pages, table = filled(lens, 64, hkv, d, seed)
    td, n = table.cuda(), len(lens)
    g = torch.Generator(device="cuda").manual_seed(seed)
    q = torch.randn(n * q_tokens, hq, d, generator=g, device="cuda").to(dtype)
    out, lse = moe.kv_attention(q, pages, td, i32(lens), page_size=64, n_kv_heads=hkv, q_tokens=q_tokens, window=window,
                                return_lse=True)
    for s, m in enumerate(lens):
        rows = slice(s * q_tokens, (s + 1) * q_tokens)
        if m == 0:
            assert not bool(out[rows].any()) and bool((lse[rows] == -float("inf")).all())
            continue
        k, v = [x.double().repeat_interleave(hq // hkv, 1) for x in moe.kv_read(
            pages, td[s:s + 1], i32([0]), i32([0, m]), m, page_size=64, n_kv_heads=hkv, head_dim=d, dtype=torch.float32)]
        z = torch.einsum("rhd,nhd->hrn", q[rows].double(), k) * d ** -0.5
        at = (m - q_tokens + torch.arange(q_tokens, device="cuda"))[None, :, None]
        key = torch.arange(m, device="cuda")
        hide = key > at
        if window:
            hide = hide | (key <= at - window)
        z.masked_fill_(hide, -float("inf"))
        w = torch.nan_to_num(torch.softmax(z, -1))
        ref, mag = torch.einsum("hrn,nhd->rhd", w, v), torch.einsum("hrn,nhd->rhd", w, v.abs())
        size = (torch.einsum("rhd,nhd->hrn", q[rows].double().abs(), k.abs()) * d ** -0.5).amax(-1).T
        tol = mag * (2.0 ** -10 + 2.0 ** -12 + 2.0 ** -17 * size[..., None]) + R.EPS[dtype] * ref.abs() + 1e-30
        big = v.unflatten(-1, (-1, 32)).abs().amax(-1)                                    # 8 d at most, 7 d at least
        top = torch.einsum("hrn,nhb->rhb", w, big / 7).repeat_interleave(32, -1)
        most = (w * big.amax(-1).T[:, None]).amax(-1).T[..., None]
        tol = tol + 2.0 ** -16 * top + m * (2.0 ** -35 * most + 2.0 ** -92)
        assert bool(((out[rows].double() - ref).abs() <= tol).all()), (s, m)
        want, got = torch.logsumexp(z, -1).T, lse[rows].double()
        none = torch.isinf(want)
        assert torch.equal(torch.isinf(got) & (got < 0), none)
        assert bool(((got - want).abs() <= 2.0 ** -17 * size + 2.0 ** -20 * (1 + want.abs()))[~none].all()), (s, m)


@pytest.mark.parametrize("d,hq,hkv,q_tokens", [(64, 8, 8, 1), (128, 16, 8, 1), (256, 16, 8, 2), (128, 24, 2, 1), (64, 32, 2, 2)])
@pytest.mark.parametrize("n,longest", [(2, 9000), (9, 8000), (70, 3000)])
@pytest.mark.parametrize("window,dtype", [(0, torch.bfloat16), (1, torch.bfloat16), (700, torch.float16), (33, torch.bfloat16)])
def test_ragged_batches(d, hq, hkv, q_tokens, n, longest, window, dtype):
    g = torch.Generator().manual_seed(n + d + window)
    lens = [int(x) for x in torch.randint(0, longest, (n,), generator=g)]
    lens[n // 2] = longest
    check(lens, d, hq, hkv, q_tokens, window, dtype, n + window)


@pytest.mark.parametrize("n", [1025, 1500, 2100])
@pytest.mark.parametrize("hkv", [1, 4])
def test_more_sequences_than_lanes_look_at_in_one_turn(n, hkv):
    # a lane counts n / 32 sequences: from 1025 on its share is found in a second look
    g = torch.Generator().manual_seed(n)
    lens = [int(x) for x in torch.randint(0, 90, (n,), generator=g)]
    for at in (0, n // 3, n - 1):
        lens[at] = 2500
    check(lens, 64, 4, hkv, 1, 0, torch.bfloat16, n)
