// device_once.h -- set-up that each device needs once (a kernel's attributes), from any
// number of host threads: the entry points run without the interpreter's lock.
#pragma once

#include <atomic>

namespace losa {

// N devices; one object per thing to set up.
template <int N>
class DeviceOnce {
 public:
  // setup() -- 0 if it succeeded -- unless a call of it has succeeded for this device.
  // Threads that come at the same time each call it, so it has to stand being repeated;
  // a device past N is set up every time.
  template <typename F>
  auto run(int dev, F setup) -> decltype(setup()) {
    const bool kept = dev >= 0 && dev < N;
    if (kept && done_[dev].load(std::memory_order_acquire)) return decltype(setup())(0);
    const auto rc = setup();
    if (kept && rc == decltype(setup())(0)) done_[dev].store(true, std::memory_order_release);
    return rc;
  }

 private:
  std::atomic<bool> done_[N] = {};
};

}  // namespace losa
