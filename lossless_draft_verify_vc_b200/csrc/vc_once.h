// vc_once.h -- values looked up once per device (kernel attributes, resident
// blocks) by calls that may run in several host threads.  Host code only.
#pragma once

#include <atomic>
#include <mutex>

namespace vc {

template <class T>
class PerDevice {
 public:
  // The device's value; the first call runs fill(value) alone, later ones cost one load.
  template <class Fill>
  const T& get(int dev, const Fill& fill) {
    Slot& s = slots_[dev >= 0 && dev < kDevices ? dev : 0];
    if (!s.ready.load(std::memory_order_acquire)) {
      std::lock_guard<std::mutex> lock(mu_);
      if (!s.ready.load(std::memory_order_relaxed)) {
        fill(s.value);
        s.ready.store(true, std::memory_order_release);
      }
    }
    return s.value;
  }

 private:
  static constexpr int kDevices = 64;
  struct Slot {
    std::atomic<bool> ready{false};
    T value{};
  } slots_[kDevices];
  std::mutex mu_;
};

}  // namespace vc
