// State that is made once for each device.  Function attributes (a kernel's
// dynamic shared memory limit) and occupancies belong to the device that was
// current when they were set or asked for, so a launcher that keeps one of
// each for the process would launch on a second GPU without them.
#pragma once

#include <mutex>

namespace gbo {

constexpr int kMaxDevices = 64;

template <typename State>
class PerDevice {
 public:
  // The state of device `dev`, made by make(State &) at the first call for it;
  // NULL for an index outside 0 .. kMaxDevices - 1.
  template <typename Make>
  const State *of(int dev, Make make) {
    if (dev < 0 || dev >= kMaxDevices) return nullptr;
    std::call_once(slot_[dev].once, [&] { make(slot_[dev].state); });
    return &slot_[dev].state;
  }

 private:
  struct Slot {
    std::once_flag once;
    State state;
  };
  Slot slot_[kMaxDevices];
};

}  // namespace gbo
