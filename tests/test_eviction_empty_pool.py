"""A cache without pages: the smallest that the checks of a cache take.  The refusals checked here never reach a GPU."""
import ctypes

import pytest
import torch

import router_softmax_top_gb300 as moe
from router_softmax_top_gb300 import attention as A
from tests.test_eviction_calls import AT, UNSUPPORTED, evict, lib, prompt, weigh  # noqa: F401
from tests.test_kv_layout import _cache


def test_no_totals_are_wanted_where_there_are_no_pages(lib):  # noqa: F811
    # each call has something else that is refused, by another code and after the totals are looked at
    c = _cache(n_pages=0, pages=0)
    assert weigh(lib, c, totals=None, dtype=0) == UNSUPPORTED
    assert evict(lib, c, totals=None, budget=(1 << 30) + 1) == UNSUPPORTED
    assert prompt(lib, totals=None, pages=0, q=A.MoeTensor(AT + 2, 2048, 128)) == UNSUPPORTED
    # and with pages they are
    assert prompt(lib, totals=None, q=A.MoeTensor(AT + 2, 2048, 128)) == moe.MOE_ERR_INVALID_ARG
    assert lib.moe_kv_evict_workspace(ctypes.byref(c)) > 0


@pytest.mark.gpu
@pytest.mark.parametrize("width", [0, 3])
def test_calls_on_an_empty_pool(width):
    hkv, d, ps = 2, 64, 32
    pages, totals = moe.kv_pages(0, hkv, d, ps), moe.kv_totals(0, hkv, ps)
    table = torch.full((4, width), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(4, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    q = torch.randn(4, 4, d, device="cuda").bfloat16()
    args = dict(page_size=ps, n_kv_heads=hkv, status=status)
    o, lse = moe.kv_attention(q, pages, table, lens, return_lse=True, **args)
    assert moe.kv_weigh(q, pages, table, lens, lse, totals=totals, **args) is totals
    new, kept = moe.kv_evict(pages, table, lens, 8, totals=totals, head_dim=d, **args)
    assert new.tolist() == [0] * 4 and bool((kept == -1).all()) and int(status) == 0
    cu = torch.zeros(5, dtype=torch.int32, device="cuda")
    k = torch.randn(4, hkv, d, device="cuda").bfloat16()
    assert moe.prompt_weigh(q, k, lse, cu, totals=totals, page_table=table, status=status) is totals
    assert int(status) == 0
    if width:
        # tokens without pages: a status, and nothing else
        lens += 40
        moe.kv_weigh(q, pages, table, lens, lse, totals=totals, **args)
        assert int(status) == moe.MOE_KV_BAD_PAGE
        status.zero_()
        new, kept = moe.kv_evict(pages, table, lens, 8, totals=totals, head_dim=d, **args)
        assert new.tolist() == [40] * 4 and bool((kept == -1).all()) and int(status) == moe.MOE_KV_BAD_PAGE
