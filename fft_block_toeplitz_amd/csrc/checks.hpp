// Argument checks that the C entry points of the sequence operators share.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fftmv.h"

namespace fftmv {

inline int status_of(hipError_t e) {
  if (e == hipSuccess) return FFTMV_SUCCESS;
  if (e == hipErrorInvalidConfiguration) return FFTMV_ERR_UNSUPPORTED_SIZE;  // a grid above 2^32 work-items
  if (e == hipErrorInvalidValue) return FFTMV_ERR_INVALID_ARG;
  if (e == hipErrorOutOfMemory) return FFTMV_ERR_OUT_OF_MEMORY;
  return FFTMV_ERR_HIP;
}

inline bool aligned(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline bool field(const void *p, size_t es) { return p && aligned(p, es); }
inline bool floats(const void *p) { return aligned(p, 4); }  // NULL passes

inline size_t elem_bytes(int dtype) { return dtype == FFTMV_F32 ? 4 : 2; }

// The kernels count samples, rows of a sample and channels in 32 bits, and run
// up to a few thousand rows past the last one.
constexpr int64_t kMost = INT32_MAX - (1 << 16);
inline bool sizes_fit(int64_t batch, int64_t rows, int64_t channels) {
  return batch <= kMost && rows <= kMost && channels <= kMost;
}

// Rows r * step apart, the last of them `channels` long, stay inside 63 bits.
inline bool strides_ok(int64_t n, int64_t stride, int64_t m, int64_t step, int64_t channels) {
  int64_t a = 0, b = 0, c = 0;
  if (stride < 0 || step < 0) return false;
  return !__builtin_mul_overflow(n, stride, &a) && !__builtin_mul_overflow(m, step, &b) &&
         !__builtin_add_overflow(a, b, &c) && !__builtin_add_overflow(c, channels, &a) &&
         !__builtin_mul_overflow(a, int64_t(8), &b);
}

}  // namespace fftmv
