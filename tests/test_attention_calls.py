"""Calls of the attention operators that never reach a GPU."""
import ctypes

import pytest

import router_softmax_top_gb300 as moe
from router_softmax_top_gb300 import attention as A
from router_softmax_top_gb300 import build as moe_build
from tests.test_kv_layout import _cache


@pytest.fixture(scope="module")
def lib():
    moe_build.build()
    return A._lib()


@pytest.mark.parametrize("table", [0, 1 << 20])
def test_a_step_of_no_sequences(lib, table):
    c = ctypes.byref(_cache(n_seqs=0, page_table=table))
    t = ctypes.byref(A.MoeTensor(1 << 20, 1024, 128))
    for n, code in ((0, moe.MOE_OK), (2, moe.MOE_ERR_INVALID_ARG)):
        assert lib.moe_kv_append(c, 1 << 20, 1 << 20, n, None, 0, t, t, None, None, 0, 0, 0, None, 1 << 20, 1, None) == code
        assert lib.moe_kv_read(c, 1 << 20, 1 << 20, n, 1 << 20, 1 << 20, 1, None) == code
    assert lib.moe_kv_attention(c, 1 << 20, t, 8, 1, 1.0, 0, 1 << 20, None, 1, 1 << 20, 1 << 30, None) == moe.MOE_OK
    assert lib.moe_prompt_attention(t, 0, 8, t, t, 0, 8, 128, 1 << 20, 1 << 20, 0, 0.1, 0, 1 << 20, None, 1, None, None) == moe.MOE_OK
