// What is asked once a device.
#pragma once

#include <atomic>
#include <mutex>

namespace sanatan {

// get(device, out, ask): the device's value, from ask(&value) (which returns 0 for
// success) the first time that this succeeds.  A failure is the call's own: the next call
// asks again.  Any thread may call; devices from kDevices on are asked every time.
template <typename Value, int kDevices = 16>
class PerDevice {
 public:
  template <typename Ask>
  auto get(int device, Value* out, Ask ask) -> decltype(ask(out)) {
    using Error = decltype(ask(out));
    if (device < 0 || device >= kDevices) return ask(out);
    if (!known_[device].load(std::memory_order_acquire)) {
      std::lock_guard<std::mutex> hold(lock_);
      if (!known_[device].load(std::memory_order_relaxed)) {
        Value answer{};
        const Error e = ask(&answer);
        if (e != Error{}) return e;
        value_[device] = answer;
        known_[device].store(true, std::memory_order_release);
      }
    }
    *out = value_[device];
    return Error{};
  }

 private:
  std::mutex lock_;
  std::atomic<bool> known_[kDevices] = {};
  Value value_[kDevices] = {};
};

}  // namespace sanatan
