// launch_limits.h -- attributes of a kernel that are raised before a launch
// (the dynamic shared memory it may take).  Host code without any CUDA call, so
// that it can be checked with a fake of the setter.
#pragma once

#include <stddef.h>

#include <atomic>
#include <mutex>

namespace wql {

// The largest value set so far for one kernel, on each device: an attribute
// belongs to the device that was current when it was set.  raise() calls
// set(value) only when the device's value is smaller, one thread at a time, so
// that no thread lowers it under another's launch.  set() returns 0 for
// success, as cudaError_t does.
class LargestPerDevice {
 public:
  template <typename Set>
  auto raise(int device, size_t value, Set set) -> decltype(set(value)) {
    using Error = decltype(set(value));
    const bool known = device >= 0 && device < kDevices;
    if (known && value <= set_[device].load(std::memory_order_acquire)) return Error(0);
    std::lock_guard<std::mutex> lock(mutex_);
    if (!known) return set(value > other_ ? other_ = value : other_);
    if (value <= set_[device].load(std::memory_order_relaxed)) return Error(0);
    const Error e = set(value);
    if (e == Error(0)) set_[device].store(value, std::memory_order_release);
    return e;
  }

 private:
  static constexpr int kDevices = 64;
  std::mutex mutex_;
  std::atomic<size_t> set_[kDevices] = {};
  size_t other_ = 0;                   // of devices past those: set every time
};

// The value set last for one kernel, on each device, of an attribute that only
// gives a preference: two threads that want different ones may each launch with
// the other's.
class LastPerDevice {
 public:
  template <typename Set> auto want(int device, int value, Set set) -> decltype(set(value)) {
    using Error = decltype(set(value));
    if (device < 0 || device >= kDevices) return set(value);
    if (last_[device].load(std::memory_order_acquire) == value + 1) return Error(0);
    const Error e = set(value);
    if (e == Error(0)) last_[device].store(value + 1, std::memory_order_release);
    return e;
  }

 private:
  static constexpr int kDevices = 64;
  std::atomic<int> last_[kDevices] = {};     // the value + 1; 0: none yet
};

}  // namespace wql
