"""Calls of the attention operators that never reach a GPU."""
import ctypes
import threading

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


# ------------------------------------------------------------------- the workspaces that are kept
@pytest.fixture
def kept(monkeypatch):
    monkeypatch.setattr(A.torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(A, "_workspaces", {})
    made = []

    def get(*key):
        return A._kept(key, lambda: made.append(key) or object())
    return get, made


def test_a_stream_keeps_its_workspaces(kept):
    get, made = kept
    a, b, c = get(0, 5, 64), get(0, 5, "prompt", 64), get(0, 6, 64)
    assert len({id(x) for x in (a, b, c)}) == 3
    assert get(0, 5, 64) is a and get(0, 5, "prompt", 64) is b and len(made) == 3


def test_threads_do_not_share_the_workspace_of_the_stream_each_has(kept):
    # handle 2 is another stream in every thread, and two of them may run at once
    get, _ = kept
    mine, theirs = [get(0, 2, 64)], []
    t = threading.Thread(target=lambda: theirs.append(get(0, 2, 64)))
    t.start()
    t.join()
    assert theirs[0] is not mine[0] and get(0, 2, 64) is mine[0]
    # of any other stream the threads share one
    mine = get(0, 7, 64)
    t = threading.Thread(target=lambda: theirs.append(get(0, 7, 64)))
    t.start()
    t.join()
    assert theirs[1] is mine


def test_workspaces_of_streams_that_come_and_go_are_given_up(kept):
    get, made = kept
    for s in range(1000):
        get(0, 16 * s + 16, 128)
    assert len(made) == 1000 and len(A._workspaces) <= A._MOST_KEPT <= 64
    get(0, 16 * 1000, 128)               # the last one is still there
    assert len(made) == 1000
