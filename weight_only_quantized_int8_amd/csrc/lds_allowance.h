// lds_allowance.h -- LDS of a launch above the 64 KiB that every kernel may use.  Host code only.
#pragma once

#include <stdint.h>

#include <atomic>

namespace int8w {

// Whether a launch has to be allowed its LDS first: what counts is the dynamic part together with
// the kernel's own arrays.
constexpr bool needs_lds_allowance(uint32_t dynamic_bytes, uint32_t static_bytes) {
  return (uint64_t)dynamic_bytes + static_bytes > 64u << 10;
}

// One kernel's allowance.  It holds for a device, so a process that uses several asks on each of
// them, and host threads may launch at the same time: two that find nothing done both ask, which
// does no harm, and none launches before its own or an earlier request has succeeded.
class LdsAllowance {
 public:
  // ask() once a device; returns what it returned, or `ok` where an earlier one did.
  template <class Error, class Ask>
  Error once(int device, Error ok, Ask ask) {
    const uint64_t bit = device >= 0 && device < 64 ? 1ull << device : 0ull;  // others ask each time
    if (done_.load(std::memory_order_acquire) & bit) return ok;
    const Error e = ask();
    if (e == ok) done_.fetch_or(bit, std::memory_order_release);
    return e;
  }

 private:
  std::atomic<uint64_t> done_{0};
};

}  // namespace int8w
