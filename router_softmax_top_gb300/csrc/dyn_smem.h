// The dynamic shared memory limit that a kernel has been raised to, per device:
// plain C++ that the library and the host tests share.
#pragma once

#include <atomic>
#include <mutex>
#include <stddef.h>

namespace moe {

// (The attribute belongs to the kernel on each device.)
struct DynSmemLimit {
  static constexpr int kDevices = 64;
  std::atomic<size_t> bytes[kDevices] = {};
  std::mutex lock;

  // Raises the limit on device `dev` to `want` bytes by set(want) unless it is there already; 0, or what set returned.
  // set puts the attribute to its value, lower or not, so between the look and the record nobody else may set it: a
  // smaller one that came in between would leave a record that is above the limit, and launches that fail.
  template <typename Set>
  int raise(int dev, size_t want, Set set) {
    std::atomic<size_t> *cur = (dev >= 0 && dev < kDevices) ? &bytes[dev] : nullptr;
    if (cur && want <= cur->load(std::memory_order_acquire)) return 0;
    const std::lock_guard<std::mutex> held(lock);
    if (cur && want <= cur->load(std::memory_order_relaxed)) return 0;
    const int e = set(want);
    if (e == 0 && cur && want > cur->load(std::memory_order_relaxed)) cur->store(want, std::memory_order_release);
    return e;
  }
};

}  // namespace moe
