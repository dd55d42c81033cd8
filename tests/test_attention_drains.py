"""What the attention kernels wait for before they give memory back, on the CPU.

A role that leaves early (its own wait gave up, or another role's did) sets a flag that
cuts other waits short; a wait for copies or products in flight must not be one of them.
The wait functions are taken out of the kernels' header and run on a barrier and a
clock of the test's own."""
import ctypes
import os
import re
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "router_softmax_top_gb300", "csrc")
STUBS = r'''
#include <stdint.h>
#define __device__
#define __forceinline__ inline
static long polls, done_after, clock_ns;
static uint64_t a_now_ns() { return clock_ns += 1000; }
static bool a_mbar_try(uint64_t *, uint32_t) { return ++polls > done_after; }
constexpr uint64_t kAttnWaitNs = 2000000000ull;
constexpr uint32_t kAttnSpin = 1u << 26;
'''
CALLS = r'''
extern "C" int wait_with(long after, int failed) {
  polls = clock_ns = 0; done_after = after;
  uint64_t bar = 0;
  return a_mbar_wait(&bar, 0, &failed);
}
extern "C" int drain(long after) {
  polls = clock_ns = 0; done_after = after;
  uint64_t bar = 0;
  return a_mbar_drain(&bar, 0);
}
'''


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return f.read()


@pytest.fixture(scope="module")
def waits(tmp_path_factory):
    text = source("attn_common.cuh")
    parts = []
    for fn in ("a_mbar_wait", "a_mbar_drain"):
        m = re.search(r"__device__ __forceinline__ bool " + fn + r"\([^\n]*(?:\}\n|\{\n.*?\n\}\n)", text, re.S)
        assert m, fn
        parts.append(m.group(0))
    d = tmp_path_factory.mktemp("waits")
    (d / "w.cpp").write_text(STUBS + "".join(parts) + CALLS)
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-o", str(d / "w.so"), str(d / "w.cpp")], check=True)
    lib = ctypes.CDLL(str(d / "w.so"))
    lib.wait_with.argtypes, lib.drain.argtypes = [ctypes.c_long, ctypes.c_int], [ctypes.c_long]
    return lib


def test_a_failure_cuts_waits_short_but_not_drains(waits):
    assert waits.wait_with(100000, 0) == 1 and waits.wait_with(100000, 1) == 0
    assert waits.drain(100000) == 1
    assert waits.drain(1 << 40) == 0        # bounded all the same


def test_products_are_drained_before_tensor_memory_is_given_back():
    text = source("prompt_attention.cu")
    end = text[text.index("commit(&done);"):]
    first_wait = re.search(r"\b(a_mbar_drain|a_mbar_wait|wait)\(([^;]*)\);", end)
    assert first_wait.group(1) == "a_mbar_drain" and first_wait.group(2) == "&done, 0"
    assert end.index("a_mbar_drain(&done, 0)") < end.index("tcgen05.dealloc")


def test_copies_are_drained_before_the_loader_leaves():
    text = source("prompt_attention.cu")
    tail = text[text.index("no copy may be in flight when the CTA leaves"):]
    lines = tail[:tail.index("kMmaWarp")].split("\n")
    waits = [x for x in lines if "_full[" in x or "q_bar" in x]
    assert len(waits) == 3 and all("a_mbar_drain(" in x and "a_mbar_wait(" not in x for x in waits)
