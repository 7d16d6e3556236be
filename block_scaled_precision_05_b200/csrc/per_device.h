// per_device.h -- what a launcher looks up once per device (host side, no CUDA).
#pragma once

#include <atomic>

namespace bsp {

constexpr int kMaxDevices = 64;

// A value for each device, 0 until it is known.  Launches come from any thread (the bindings release the interpreter);
// two that look the same value up at once store the same one, so each load and store being atomic is enough.
class PerDevice {
 public:
  int get(int device) const { return value_[device].load(std::memory_order_relaxed); }
  void set(int device, int value) { value_[device].store(value, std::memory_order_relaxed); }

 private:
  std::atomic<int> value_[kMaxDevices] = {};
};

}  // namespace bsp
