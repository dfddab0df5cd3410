// A positive number that is found out once per device (a kernel's attribute
// that has been set, a count of resident clusters), kept by device number.
#pragma once

#include <atomic>

namespace moe {

constexpr int kMaxDevices = 64;

class PerDevice {
 public:
  // The number of device `dev`: make()'s result, called until it is positive.
  // Threads that come together may each call it; they find the same number.
  template <typename F>
  int get(int dev, F&& make) {
    if (dev < 0 || dev >= kMaxDevices) return make();
    int v = of_[dev].load(std::memory_order_acquire);
    if (v > 0) return v;
    v = make();
    if (v > 0) of_[dev].store(v, std::memory_order_release);
    return v;
  }

 private:
  std::atomic<int> of_[kMaxDevices] = {};
};

}  // namespace moe
