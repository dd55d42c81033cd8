"""How the attention operators are called: streams, sizes of nothing, arguments at their ends."""
import pytest
import torch

import router_softmax_top_gb300 as moe

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def some_cache(n, ps=32, hkv=2, d=64):
    pages = moe.kv_pages(-(-n // ps), hkv, d, ps)
    table = torch.arange(pages.shape[0], dtype=torch.int32, device="cuda")[None]
    k, v = [torch.randn(n, hkv, d, device="cuda").bfloat16() for _ in range(2)]
    moe.kv_append(pages, table, i32([0]), i32([0, n]), k, v, page_size=ps)
    return pages, table


@pytest.mark.parametrize("rot", [0, 32, 64])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rows_without_a_place_are_nan_whatever_is_rotated(rot, interleaved):
    x = torch.randn(6, 2, 64, device="cuda")
    cos, sin = moe.rope_table(34, rot) if rot else (None, None)
    for starts, cu, bit, dead in (([-1], [0, 6], moe.MOE_KV_BAD_LENGTH, range(6)),
                                  ([0], [0, 4], moe.MOE_KV_BAD_LENGTH, [4, 5]),
                                  ([30], [0, 6], moe.MOE_KV_BAD_POSITION, [4, 5])):
        if not rot and bit == moe.MOE_KV_BAD_POSITION:
            continue
        pages, status = moe.kv_pages(2, 2, 64, 32), i32([0])
        q, k = moe.kv_append(pages, i32([[0, 1]]), i32(starts), i32(cu), x, x, page_size=32, q=x, cos=cos, sin=sin,
                             interleaved=interleaved, status=status)
        assert int(status) == bit
        gone = torch.zeros(6, dtype=torch.bool, device="cuda")
        gone[list(dead)] = True
        for y in (q, k):
            assert bool(torch.isnan(y[gone]).all()) and bool(torch.isfinite(y[~gone]).all())


def test_a_step_of_no_sequences():
    pages = moe.kv_pages(1, 2, 64, 32)
    table, none, cu = i32([[0]])[:0], i32([]), i32([0])
    q, k = [torch.zeros(0, h, 64, device="cuda", dtype=torch.bfloat16) for h in (4, 2)]
    a, b = moe.kv_append(pages, table, none, cu, k, k, page_size=32, q=q)
    assert a.shape == (0, 4, 64) and b.shape == (0, 2, 64)
    for t in moe.kv_read(pages, table, none, cu, 0, page_size=32, n_kv_heads=2, head_dim=64):
        assert t.shape == (0, 2, 64)
    assert moe.kv_attention(q, pages, table, none, page_size=32, n_kv_heads=2).shape == (0, 4, 64)
    assert moe.prompt_attention(q, k, k, cu).shape == (0, 4, 64)
    one = torch.zeros(1, 2, 64, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(moe.MoeError):       # tokens without a sequence
        moe.kv_append(pages, table, none, cu, one, one, page_size=32)
    with pytest.raises(moe.MoeError):
        moe.kv_read(pages, table, none, cu, 1, page_size=32, n_kv_heads=2, head_dim=64)
