// Values that are asked of the runtime once per device and then shared by all host threads.
#pragma once

#include <atomic>

namespace moe {

// N ints for each of the first kDevices devices.  The values are published with release
// order after all of them are stored, and read only after the flag was seen with acquire
// order, so that no thread meets a device's values half written (plain stores may become
// visible in any order on a weakly ordered CPU).  Threads that come before the first is
// done each make the values themselves, which are the same.
template <int N>
class PerDevice {
 public:
  static constexpr int kDevices = 64;

  // Fills out with the values of `device`, from make(out) where none are kept yet.  What
  // make() fails to find (false) is not kept and not returned.
  template <class Make>
  bool get(int device, int (&out)[N], Make make) {
    const bool known = device >= 0 && device < kDevices;
    if (known && ready_[device].load(std::memory_order_acquire)) {
      for (int i = 0; i < N; ++i) out[i] = value_[device][i].load(std::memory_order_relaxed);
      return true;
    }
    if (!make(out)) return false;
    if (known) {
      for (int i = 0; i < N; ++i) value_[device][i].store(out[i], std::memory_order_relaxed);
      ready_[device].store(true, std::memory_order_release);
    }
    return true;
  }

 private:
  std::atomic<int> value_[kDevices][N] = {};
  std::atomic<bool> ready_[kDevices] = {};
};

}  // namespace moe
