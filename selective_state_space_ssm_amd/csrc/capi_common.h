// What the C ABI's source files share: the calling thread's error text and
// the host-side argument checks.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <string>

#include "ssm_scan.h"

namespace ssm {
namespace capi {

inline thread_local std::string g_err;

inline int fail(int code, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  g_err = buf;
  return code;
}

inline int hip_fail(hipError_t e, const char* what) {
  return fail(SSM_EHIP, "%s: %s", what, hipGetErrorString(e));
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Byte range [p, p + n) of a possibly-null pointer.
struct Range {
  uintptr_t lo, hi;
  bool valid;
};
inline Range range_of(const void* p, uint64_t bytes) {
  Range r;
  r.valid = p != nullptr && bytes > 0;
  r.lo = reinterpret_cast<uintptr_t>(p);
  r.hi = r.lo + bytes;
  return r;
}
inline bool overlap(const Range& a, const Range& b) { return a.valid && b.valid && a.lo < b.hi && b.lo < a.hi; }

// x*y with an overflow check against 2^62.
inline bool mul_ok(int64_t x, int64_t y, int64_t* out) {
  const int64_t lim = int64_t(1) << 62;
  if (x < 0 || y < 0) return false;
  if (x != 0 && y > lim / x) return false;
  *out = x * y;
  return true;
}

}  // namespace capi
}  // namespace ssm
