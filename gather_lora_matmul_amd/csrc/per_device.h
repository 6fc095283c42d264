// A setting of a process that each device needs once (internal).
#pragma once

#include <atomic>
#include <cstdint>

namespace lora {

// done(device, set) calls set() unless it has succeeded (returned 0) for this device
// before; devices from 64 on are not remembered.  Threads may call it at the same
// time: a setting may then be made twice, never not at all.
class PerDevice {
 public:
  template <typename F>
  auto done(int device, F set) -> decltype(set()) {
    const uint64_t bit = device >= 0 && device < 64 ? (uint64_t)1 << device : 0;
    using R = decltype(set());
    if (bit && (set_.load(std::memory_order_acquire) & bit)) return R{};
    const R r = set();
    if (r == R{}) set_.fetch_or(bit, std::memory_order_release);
    return r;
  }

 private:
  std::atomic<uint64_t> set_{0};
};

}  // namespace lora
