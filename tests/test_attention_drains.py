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


# ------------------------------------------------------------------- a warp's ring of tiles
RING = r'''
#include <stdint.h>
#include <stdlib.h>
#include <vector>
#include "kv_layout.h"
using namespace moe;

// Barriers of one arrival per phase and copies that land when the clock says so, as the kernel's warp uses them.
struct Bar { uint32_t phase = 0; int pending = 1; long landing = -1; };
struct Model {
  static constexpr int S = 2;
  Bar bar[S];
  long now = 0, limit;
  int faults = 0;    // arrivals on a phase that has had its own, or copies into a stage that one is on its way to
  explicit Model(long limit) : limit(limit) {}
  void settle() {
    for (Bar &b : bar)
      if (b.pending == 0 && b.landing >= 0 && now >= b.landing) { b.landing = -1; b.pending = 1; ++b.phase; }
  }
  void ask(uint32_t x, long delay) {   // delay 0: the tile has no page, an arrival without a copy
    settle();
    Bar &b = bar[TileRing<S>::stage(x)];
    if (b.pending == 0 || b.phase != x / S) ++faults;
    b.pending = 0;
    b.landing = now + delay;
  }
  bool there(uint32_t x) {
    settle();
    return (bar[TileRing<S>::stage(x)].phase & 1u) != TileRing<S>::parity(x);   // what a test of a phase's parity says
  }
  bool wait(uint32_t x) {
    const long end = now + limit;
    for (;; ++now) {
      if (there(x)) return true;
      if (now >= end) return false;
    }
  }
  int on_way() { settle(); int n = 0; for (Bar &b : bar) n += b.pending == 0; return n; }
};

// A share of `tiles`; copies take delay[x].  Out: faults, copies on their way when the part is written, tiles that came,
// and the clock.
extern "C" void run(int tiles, const long *delay, long limit, long *out) {
  Model m(limit);
  TileRing<Model::S> ring;
  auto issue = [&](uint32_t x) {
    if (!ring.dead && (int)x < tiles) m.ask(x, delay[x]);
  };
  for (int i = 0; i < Model::S; ++i) issue(i);
  long came = 0;
  for (int t = 0; t < tiles; ++t) {
    const uint32_t x = ring.used;
    ring.take([&](uint32_t y) { return m.there(y); }, [&](uint32_t y) { return m.wait(y); });
    came += !ring.dead;
    m.now += 3;
    issue(x + Model::S);
  }
  out[0] = m.faults; out[1] = m.on_way(); out[2] = came; out[3] = m.now;
}
'''


@pytest.fixture(scope="module")
def ring(tmp_path_factory):
    d = tmp_path_factory.mktemp("ring")
    (d / "r.cpp").write_text(RING)
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-I", CSRC, "-o", str(d / "r.so"), str(d / "r.cpp")],
                   check=True)
    lib = ctypes.CDLL(str(d / "r.so"))

    def run(delays, limit):
        out = (ctypes.c_long * 4)()
        lib.run(len(delays), (ctypes.c_long * len(delays))(*delays), ctypes.c_long(limit), out)
        return list(out)
    return run


def test_a_ring_whose_copies_come(ring):
    import random
    rng = random.Random(1)
    for _ in range(2000):
        n = rng.randrange(0, 12)
        delays = [rng.choice([0, 1, 5, 40]) for _ in range(n)]
        assert ring(delays, 100)[:3] == [0, 0, n]


def test_a_ring_whose_copy_is_late(ring):
    # a copy that lands after the wait for it gave up, but within the wait after that
    import random
    rng = random.Random(2)
    for _ in range(2000):
        n = rng.randrange(1, 12)
        delays = [rng.choice([0, 1, 5, 40]) for _ in range(n)]
        late = rng.randrange(n)
        delays[late] = rng.randrange(150, 190)
        faults, on_way, came, _ = ring(delays, 100)
        assert faults == 0 and on_way == 0 and came <= n and (came == late or came == n)


def test_a_ring_whose_copies_never_come_ends(ring):
    for n in (1, 2, 3, 9):
        for lost in range(n):
            delays = [1 << 40 if x >= lost else 5 for x in range(n)]
            faults, on_way, came, clock = ring(delays, 100)
            assert faults == 0 and came == lost and on_way <= 2
            assert clock <= 4 * 100 + 20 * n     # one wait, and one more for each stage
