// lds_allowance.h -- LDS of a launch above the 64 KiB that every kernel may use.  Host code only.
#pragma once

#include <stdint.h>

namespace int8w {

// Whether a launch has to be allowed its LDS first: what counts is the dynamic part together with
// the kernel's own arrays.
constexpr bool needs_lds_allowance(uint32_t dynamic_bytes, uint32_t static_bytes) {
  return (uint64_t)dynamic_bytes + static_bytes > 64u << 10;
}

}  // namespace int8w
