// Work that is done once for each device of the process: a kernel's attributes
// (its limit of dynamic shared memory, say) belong to the device that was
// current when they were set. Plain C++, no CUDA headers.
#pragma once

#include <stdint.h>

#include <atomic>

namespace sv {

class DeviceOnce {
 public:
  // f() until it has returned 0 once for this device; returns what it returned,
  // or 0. Devices past the 64th run it every time.
  template <typename Err, typename F>
  Err run(int dev, F f) {
    const uint64_t bit = dev >= 0 && dev < 64 ? 1ull << dev : 0;
    if (done_.load(std::memory_order_acquire) & bit) return Err(0);
    const Err e = f();
    if (e == Err(0)) done_.fetch_or(bit, std::memory_order_release);
    return e;
  }

 private:
  std::atomic<uint64_t> done_{0};
};

}  // namespace sv
