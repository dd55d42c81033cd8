"""Raising a kernel's shared memory limit from several threads at once, on the CPU: the limit that is set is never below the
one on record.  The header is compiled behind a setter of the test's own, which holds the first thread up until another has
been through, or half a second."""
import ctypes
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "router_softmax_top_gb300", "csrc")
CODE = r'''
#include <chrono>
#include <thread>
#include "dyn_smem.h"
using namespace moe;

// The first thread asks for `first` bytes and is held up where it sets them; the second for `second`, once the first is there.
extern "C" void two_threads(long first, long second, int dev, long *out) {
  DynSmemLimit limit;
  std::atomic<long> attribute{0}, sets{0};
  std::atomic<bool> inside{false}, through{false};
  auto wait = [](std::atomic<bool> &flag) {
    for (int i = 0; i < 500 && !flag.load(); ++i) std::this_thread::sleep_for(std::chrono::milliseconds(1));
  };
  std::thread a([&] {
    limit.raise(dev, (size_t)first, [&](size_t want) {
      inside = true;
      wait(through);
      ++sets;
      attribute = (long)want;
      return 0;
    });
  });
  std::thread b([&] {
    wait(inside);
    limit.raise(dev, (size_t)second, [&](size_t want) { ++sets; attribute = (long)want; return 0; });
    through = true;
  });
  a.join();
  b.join();
  // a launch of the larger size comes after both
  const long most = first > second ? first : second;
  limit.raise(dev, (size_t)most, [&](size_t want) { ++sets; attribute = (long)want; return 0; });
  out[0] = attribute;
  out[1] = sets;
  out[2] = dev >= 0 && dev < DynSmemLimit::kDevices ? (long)limit.bytes[dev].load() : -1;
}

extern "C" int failing(long *record) {
  DynSmemLimit limit;
  const int e = limit.raise(0, 1000, [](size_t) { return 7; });
  *record = (long)limit.bytes[0].load();
  return e;
}
'''


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("limit")
    (d / "l.cpp").write_text(CODE)
    subprocess.run(["g++", "-O1", "-std=c++17", "-pthread", "-shared", "-fPIC", "-I", CSRC, "-o", str(d / "l.so"), str(d / "l.cpp")],
                   check=True)
    return ctypes.CDLL(str(d / "l.so"))


@pytest.mark.parametrize("first,second", [(80000, 196608), (196608, 80000), (100000, 100000)])
@pytest.mark.parametrize("dev", [0, 63])
def test_two_threads(lib, first, second, dev):
    out = (ctypes.c_long * 3)()
    lib.two_threads(ctypes.c_long(first), ctypes.c_long(second), dev, out)
    most = max(first, second)
    assert out[0] >= most and out[2] == most


def test_a_limit_that_is_not_taken_is_not_on_record(lib):
    record = ctypes.c_long(-1)
    assert lib.failing(ctypes.byref(record)) == 7 and record.value == 0


def test_every_kernel_goes_by_the_record():
    # nobody sets the attribute beside it (the allocation-free entry point has a lock and a record of its own)
    for name in os.listdir(CSRC):
        with open(os.path.join(CSRC, name)) as f:
            text = f.read()
        assert text.count("cudaFuncAttributeMaxDynamicSharedMemorySize") == (1 if name in ("common.cuh", "noalloc.cu") else 0), name
