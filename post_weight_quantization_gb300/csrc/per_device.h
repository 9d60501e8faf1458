// What is done once for every device of the process, such as a kernel's shared-memory limit: a
// function's attributes belong to the device that was current when they were set.
#pragma once

#include <atomic>
#include <cstdint>

namespace gptq {

class PerDevice {
 public:
  static constexpr int kMaxDevices = 64;
  // f() for a device that it has not succeeded for; true once it has.
  template <typename F>
  bool once(int device, F&& f) {
    const uint64_t bit = 1ull << device;
    if (done_.load(std::memory_order_acquire) & bit) return true;
    if (!f()) return false;
    done_.fetch_or(bit, std::memory_order_release);
    return true;
  }

 private:
  std::atomic<uint64_t> done_{0};
};

}  // namespace gptq
