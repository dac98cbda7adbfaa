// Work that has to be done once on every device in use: an attribute of a kernel,
// for one, belongs to the device that is current when it is set.
#pragma once

#include <atomic>
#include <cstdint>

class OncePerDevice {
 public:
  // Runs set() unless it has succeeded on this device before; false where it fails
  // (the next call tries again).  Threads that come at the same time may both run it.
  template <class Set>
  bool ensure(int device, Set set) {
    const uint64_t bit = device >= 0 && device < 64 ? 1ull << device : 0ull;
    if (done_.load(std::memory_order_acquire) & bit) return true;
    if (!set()) return false;
    done_.fetch_or(bit, std::memory_order_release);
    return true;
  }

 private:
  std::atomic<uint64_t> done_{0};
};
