// Host helpers shared by the C ABI sources: the per-thread error string, status
// returns and argument checks.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <cstdarg>
#include <cstdio>
#include <string>

#include "../../include/vggt3.h"

namespace vggt3 {
namespace api {

inline std::string& last_error() {
  thread_local std::string e;
  return e;
}

inline int fail(int status, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
inline int fail(int status, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  last_error() = buf;
  return status;
}

inline int ok() {
  last_error().clear();
  return VGGT3_OK;
}

inline int check_hip(hipError_t e, const char* what) {
  if (e != hipSuccess) return fail(VGGT3_EHIP, "%s: %s", what, hipGetErrorString(e));
  return VGGT3_OK;
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline bool overlap(const void* a, size_t an, const void* b, size_t bn) {
  if (a == nullptr || b == nullptr || an == 0 || bn == 0) return false;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  return a0 < b0 + bn && b0 < a0 + an;
}

inline bool valid_dtype(int32_t dt) { return dt == VGGT3_BF16 || dt == VGGT3_F32; }
inline size_t elem_size(int32_t dt) { return dt == VGGT3_BF16 ? 2 : 4; }
inline size_t round256(size_t b) { return (b + 255) / 256 * 256; }

}  // namespace api
}  // namespace vggt3
