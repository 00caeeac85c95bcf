// ssm_host.hpp -- what the library's host files share: the error message of the
// calling thread, size arithmetic, and the alias and alignment checks.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ssm_scan.h"

namespace ssmh {

// The detail ssm_last_error_message() returns lives in ssm_scan.hip, one for
// each thread: every call clears it first.
__attribute__((visibility("hidden"))) void clear_message();

// Keeps the message and returns the status.
__attribute__((visibility("hidden"), format(printf, 2, 3))) ssm_status_t fail(ssm_status_t s,
                                                                              const char* fmt, ...);

constexpr int64_t kMaxGrid = (int64_t(1) << 31) - 1;

inline size_t dtype_size(int32_t dt) { return dt == SSM_BF16 ? 2 : 4; }

inline bool mul_ok(int64_t a, int64_t b, int64_t* out) {
  if (a < 0 || b < 0) return false;
  if (a != 0 && b > INT64_MAX / a) return false;
  *out = a * b;
  return true;
}

inline size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

struct Range {
  const void* p;
  size_t bytes;
};

inline bool overlap(Range a, Range b) {
  if (!a.p || !b.p || a.bytes == 0 || b.bytes == 0) return false;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
  return a0 < b0 + b.bytes && b0 < a0 + a.bytes;
}

inline bool misaligned(const void* p, size_t align) {
  return p && (reinterpret_cast<uintptr_t>(p) % align) != 0;
}

inline ssm_status_t launch_status(const char* what) {
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(SSM_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
  return SSM_OK;
}

}  // namespace ssmh
