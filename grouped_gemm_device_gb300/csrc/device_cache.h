// A number that is asked of a device (how many blocks of a kernel fit an SM, its registers) and kept
// for that device once it has been answered.
#pragma once

#include <atomic>

namespace moe {

class DeviceCache {
 public:
  // ask() returns the number of the current device, which is `device`, or 0 if it could not be had:
  // then the next call asks again.
  template <class F>
  int get(int device, F&& ask) {
    if (device < 0 || device >= kDevices) return ask();
    int n = value_[device].load(std::memory_order_relaxed);
    if (n <= 0) {
      n = ask();
      if (n > 0) value_[device].store(n, std::memory_order_relaxed);
    }
    return n;
  }

 private:
  static constexpr int kDevices = 64;
  std::atomic<int> value_[kDevices] = {};
};

}  // namespace moe
