// Numbers that the host learns once per device of the process: a kernel's
// attributes are set on, and its occupancy belongs to, the device that is
// current.  Plain C++, no CUDA types.
#pragma once

#include <atomic>

namespace moe {

class PerDevice {
 public:
  static constexpr int kMaxDevices = 256;

  // *value: device's number (not negative), from make(value) where it is not
  // known yet.  make returns an error, 0 for none; after an error nothing is
  // kept.  Threads may make it at the same time; it is published after make has
  // returned, so a thread that finds it finds what make set up too.
  template <typename Make>
  auto get(int device, int* value, Make make) -> decltype(make(value)) {
    std::atomic<int>* slot = device >= 0 && device < kMaxDevices ? &known_[device] : nullptr;
    const int known = slot ? slot->load(std::memory_order_acquire) : 0;
    if (known > 0) {
      *value = known - 1;
      return {};
    }
    const auto error = make(value);
    if (error == decltype(make(value)){} && slot) slot->store(*value + 1, std::memory_order_release);
    return error;
  }

 private:
  std::atomic<int> known_[kMaxDevices] = {};   // number + 1; 0: not known
};

}  // namespace moe
