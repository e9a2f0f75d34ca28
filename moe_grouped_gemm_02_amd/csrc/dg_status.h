// Error reporting and argument checks shared by the C ABI files.
#pragma once

#include <stdint.h>

namespace dg {

// Sets the calling thread's last error text and returns `status`.
int fail(int status, const char* fmt, ...);
// Clears the last error text and returns DG_SUCCESS.
int ok();

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// count * stride * elem < lim, for count, stride >= 0 and elem, lim > 0,
// decided without forming the product (strides come from the caller).
inline bool below(int64_t count, int64_t stride, int64_t elem, int64_t lim) {
  if (count == 0 || stride == 0) return true;
  return stride <= (lim - 1) / elem / count;
}

}  // namespace dg
