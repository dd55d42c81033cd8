"""Refusals of the routing entry points that never reach a GPU."""
import ctypes

import pytest

import router_softmax_top_gb300 as moe
from router_softmax_top_gb300 import build as moe_build
from router_softmax_top_gb300 import routing


@pytest.fixture(scope="module")
def lib():
    moe_build.build()
    return routing._lib()


GOOD = dict(n_experts=64, top_k=8, score=0, n_groups=8, top_groups=4, group_score=1, renormalise=1, scale=1.0)


def call(lib, n=4, logits=1 << 20, ids=1 << 20, weights=1 << 20, dtype=0, bias=None, **kw):
    r = routing.MoeRouting(**dict(GOOD, **kw))
    return lib.moe_route(ctypes.byref(r), logits, 64, n, bias, ids, weights, dtype, None, None)


@pytest.mark.parametrize("kw", [
    dict(n_experts=0), dict(n_experts=-8), dict(top_k=0), dict(top_k=33, top_groups=4), dict(n_groups=0), dict(n_groups=7),
    dict(top_groups=0), dict(top_groups=9), dict(top_groups=1, top_k=9), dict(score=2), dict(score=-1), dict(group_score=2),
    dict(group_score=-1), dict(scale=float("nan")), dict(scale=float("inf")), dict(dtype=3), dict(dtype=-1), dict(n=-1),
    dict(logits=None), dict(ids=None), dict(weights=None), dict(logits=(1 << 20) + 2), dict(ids=(1 << 20) + 1),
    dict(bias=(1 << 20) + 2)])
def test_arguments_that_make_no_sense(lib, kw):
    assert call(lib, **kw) == moe.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(n_experts=1032), dict(top_k=33, top_groups=8), dict(n_experts=640, n_groups=64, top_groups=4)])
def test_sizes_that_are_not_supported(lib, kw):
    assert call(lib, **kw) == moe.MOE_ERR_UNSUPPORTED


def test_no_tokens_and_no_struct(lib):
    assert call(lib, n=0, logits=None, ids=None, weights=None) == moe.MOE_OK
    assert lib.moe_route(None, 1 << 20, 64, 4, None, 1 << 20, 1 << 20, 0, None, None) == moe.MOE_ERR_INVALID_ARG
    assert lib.moe_layer_forward_routed(None, 0, None, None, None, 1, None, None) == moe.MOE_ERR_INVALID_ARG


def test_the_struct_is_the_headers(tmp_path):
    import os
    import subprocess
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    (tmp_path / "s.c").write_text('#include <stdio.h>\n#include <stddef.h>\n#include "moe_route.h"\nint main(void) '
                                  '{ printf("%zu %zu\\n", sizeof(moe_routing), offsetof(moe_routing, scale)); return 0; }')
    subprocess.run(["gcc", "-I", os.path.join(root, "include"), str(tmp_path / "s.c"), "-o", str(tmp_path / "s")], check=True)
    a = subprocess.run([str(tmp_path / "s")], capture_output=True, text=True, check=True).stdout.split()
    assert [int(v) for v in a] == [ctypes.sizeof(routing.MoeRouting), routing.MoeRouting.scale.offset] == [routing._ROUTING.size, 28]
