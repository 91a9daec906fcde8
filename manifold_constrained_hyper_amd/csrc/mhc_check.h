// Host-side argument checks shared by the translation units of the C ABI.
#pragma once

#include "mhc.h"

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace mhc {

// Largest problem accepted: B*n*C elements below 2^40 and K = n*C below 2^30
// keep every byte offset and every 32-bit kernel index in range.
constexpr int64_t kMaxElems = int64_t(1) << 40;
constexpr int64_t kMaxK = int64_t(1) << 30;
constexpr int64_t kMaxB = (int64_t(1) << 31) - 1;

struct Span {
  uintptr_t lo, hi;  // [lo, hi)
};

inline Span span(const void *p, size_t bytes) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  return Span{a, a + bytes};
}

inline bool overlaps(Span a, Span b) { return a.lo < a.hi && b.lo < b.hi && a.lo < b.hi && b.lo < a.hi; }

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline bool supported_n(int32_t n) { return n == 1 || n == 2 || n == 4 || n == 8; }

// Shape checks common to every call.  Returns MHC_OK when the shape is
// acceptable (B may be 0).
inline int check_shape(int64_t B, int32_t n, int64_t C) {
  if (B < 0 || n < 1 || C < 1) return MHC_ERR_INVALID_ARG;
  if (!supported_n(n) || C % 8 != 0) return MHC_ERR_UNSUPPORTED;
  // C is compared before it is multiplied: n * C itself could overflow.
  if (B > kMaxB || C > kMaxK / n || (B > 0 && B > kMaxElems / ((int64_t)n * C)))
    return MHC_ERR_UNSUPPORTED;
  return MHC_OK;
}

inline int64_t ncoef(int32_t n) { return (int64_t)n * n + 2 * (int64_t)n; }

inline int from_hip(hipError_t e) { return e == hipSuccess ? MHC_OK : MHC_ERR_HIP; }

}  // namespace mhc
