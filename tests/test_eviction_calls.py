"""Refusals of the attention sums' and the eviction's entry points that never reach a GPU."""
import ctypes

import pytest

import router_softmax_top_gb300 as moe
from router_softmax_top_gb300 import attention as A
from router_softmax_top_gb300 import build as moe_build
from router_softmax_top_gb300 import eviction
from tests.test_kv_layout import BAD_CACHES, _cache

AT = 1 << 20


@pytest.fixture(scope="module")
def lib():
    moe_build.build()
    A._lib()
    return eviction._lib()


def weigh(lib, c=None, **kw):
    a = dict(lens=AT, q=A.MoeTensor(AT, 2048, 128), hq=16, j=1, scale=1.0, window=0, lse=AT, totals=AT, dtype=1)
    a.update(kw)
    return lib.moe_kv_weigh(ctypes.byref(c or _cache()), a["lens"], ctypes.byref(a["q"]), a["hq"], a["j"], a["scale"], a["window"],
                            a["lse"], a["totals"], 0, a["dtype"], None)


def prompt(lib, **kw):
    a = dict(q=A.MoeTensor(AT, 2048, 128), n=4, hq=16, k=A.MoeTensor(AT, 1024, 128), nk=4, hkv=8, d=128, cu=AT, cu_k=AT, seqs=1,
             scale=1.0, window=0, lse=AT, table=AT, stride=4, width=4, pages=3, ps=64, totals=AT, restart=0, dtype=1)
    a.update(kw)
    return lib.moe_prompt_weigh(ctypes.byref(a["q"]), a["n"], a["hq"], ctypes.byref(a["k"]), a["nk"], a["hkv"], a["d"], a["cu"],
                                a["cu_k"], a["seqs"], a["scale"], a["window"], a["lse"], a["table"], a["stride"], a["width"],
                                a["pages"], a["ps"], a["totals"], a["restart"], a["dtype"], None, None)


def evict(lib, c=None, **kw):
    a = dict(lens=AT, totals=AT, budget=64, first=4, recent=8, new=AT, kept=AT, ws=AT, size=1 << 30)
    a.update(kw)
    return lib.moe_kv_evict(ctypes.byref(c or _cache()), a["lens"], a["totals"], a["budget"], a["first"], a["recent"], a["new"],
                            a["kept"], a["ws"], a["size"], None)


@pytest.mark.parametrize("change,code", BAD_CACHES)
def test_bad_caches(lib, change, code):
    c = _cache(**change)
    assert weigh(lib, c) == evict(lib, c) == code
    assert lib.moe_kv_evict_workspace(ctypes.byref(c)) == 0


INVALID, UNSUPPORTED = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED


@pytest.mark.parametrize("kw,code", [
    (dict(lens=None), INVALID), (dict(lse=None), INVALID), (dict(totals=None), INVALID), (dict(totals=AT + 2), INVALID),
    (dict(lse=AT + 1), INVALID), (dict(hq=0), INVALID), (dict(hq=12), INVALID), (dict(j=0), INVALID), (dict(j=1025), UNSUPPORTED),
    (dict(window=-1), INVALID), (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(scale=3e38), INVALID), (dict(dtype=0), UNSUPPORTED), (dict(hq=2048), UNSUPPORTED), (dict(q=A.MoeTensor(0, 2048, 128)), INVALID),
    (dict(q=A.MoeTensor(AT + 2, 2048, 128)), UNSUPPORTED), (dict(q=A.MoeTensor(AT, 2047, 128)), UNSUPPORTED)])
def test_kv_weigh(lib, kw, code):
    assert weigh(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(n=-1), INVALID), (dict(nk=-1), INVALID), (dict(seqs=-1), INVALID), (dict(hkv=0), INVALID), (dict(hq=12), INVALID),
    (dict(d=96), UNSUPPORTED), (dict(hkv=8, hq=520), UNSUPPORTED), (dict(dtype=0), UNSUPPORTED), (dict(ps=48), UNSUPPORTED),
    (dict(cu=None), INVALID), (dict(cu_k=None), INVALID), (dict(lse=None), INVALID), (dict(totals=None), INVALID),
    (dict(table=None), INVALID), (dict(stride=3), INVALID), (dict(width=-1), INVALID), (dict(pages=-1), INVALID),
    (dict(scale=0.0), INVALID), (dict(window=-1), INVALID), (dict(k=A.MoeTensor(0, 1024, 128)), INVALID),
    (dict(k=A.MoeTensor(AT + 2, 1024, 128)), UNSUPPORTED), (dict(q=A.MoeTensor(AT, 2048, 127)), UNSUPPORTED),
    (dict(width=1 << 25, stride=1 << 25), UNSUPPORTED), (dict(n=1 << 30), UNSUPPORTED),
    (dict(seqs=0), moe.MOE_OK), (dict(nk=0), moe.MOE_OK), (dict(n=0, lse=None), moe.MOE_OK)])
def test_prompt_weigh(lib, kw, code):
    assert prompt(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(lens=None), INVALID), (dict(totals=None), INVALID), (dict(totals=AT + 8), INVALID), (dict(new=None), INVALID),
    (dict(kept=None), INVALID), (dict(budget=-1), INVALID), (dict(first=-1), INVALID), (dict(recent=-1), INVALID),
    (dict(first=60), INVALID), (dict(first=2147483647, recent=2147483647), INVALID), (dict(ws=None), INVALID), (dict(ws=AT + 128), INVALID),
    (dict(size=100), INVALID), (dict(kept=AT + 2), INVALID)])
def test_kv_evict(lib, kw, code):
    assert evict(lib, **kw) == code


def test_kv_evict_of_budgets_that_counts_do_not_hold(lib):
    assert evict(lib, budget=(1 << 30) + 1) == evict(lib, budget=2147483647) == UNSUPPORTED
    assert evict(lib, budget=1 << 30, size=100) == INVALID


def test_kv_evict_of_lengths_written_over_themselves(lib):
    assert evict(lib, lens=AT + 64, new=AT + 64) == INVALID


def test_tables_wider_than_is_supported(lib):
    c = _cache(table_width=1 << 25, table_stride=1 << 25)
    assert weigh(lib, c) == evict(lib, c) == UNSUPPORTED
    assert lib.moe_kv_evict_workspace(ctypes.byref(c)) == 0
    assert lib.moe_kv_evict_workspace(ctypes.byref(_cache())) > 0


def test_no_sequences(lib):
    c = _cache(n_seqs=0, page_table=0)
    assert weigh(lib, c) == evict(lib, c) == moe.MOE_OK


def test_append_at_refuses_what_append_refuses(lib):
    t = ctypes.byref(A.MoeTensor(AT, 1024, 128))
    for c, code in ((_cache(), INVALID), (_cache(head_dim=96), UNSUPPORTED)):   # no offsets; a head size that is not supported
        assert A._lib().moe_kv_append_at(ctypes.byref(c), AT, AT, None, 2, None, 0, t, t, None, None, 0, 0, 0, None, AT, 1, None) == code
