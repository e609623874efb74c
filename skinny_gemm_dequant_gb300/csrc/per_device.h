// Work that is done once on each device of a process (plain C++: no CUDA header).
#pragma once
#include <atomic>
#include <cstdint>

namespace ql {

// `act` runs until it has returned `ok` once on a device; on devices past the 64th at every call.
class OncePerDevice {
 public:
  template <class E, class F>
  E run(int dev, E ok, F&& act) {
    const uint64_t bit = dev >= 0 && dev < 64 ? uint64_t(1) << dev : 0;
    if (done_.load(std::memory_order_acquire) & bit) return ok;
    const E e = act();
    if (e == ok) done_.fetch_or(bit, std::memory_order_release);
    return e;
  }

 private:
  std::atomic<uint64_t> done_{0};
};

}  // namespace ql
