// Rows in 8 bits with a float32 scale each: what the kernels share.
#pragma once

#include <hip/hip_runtime.h>

#include "orbit_internal.h"

namespace orbit {

struct Int8RowArgs {
  const void* in;
  const int32_t* perm;
  const uint32_t* sign_bits;
  int8_t* q_out;
  float* s_out;
  long long rows, stride;  // stride in elements
  int d, h;
  int vec;      // rows in 16-byte words
  int lds_row;  // bytes of the row's copy in LDS
  float inv_sqrt_h;
};

// A row's scale, and how its codes are made of x' sqrt(h): the low bytes of
// fma(x pre, inv, 1.5 * 2^23).  pre lifts rows whose 127 / max would leave
// float32's range (2^64 below 2^-100).
struct Int8Scale {
  float s, pre, inv;
  uint32_t keep;  // 0: the row holds an infinity or a NaN (s is NaN)
};
__device__ __forceinline__ Int8Scale int8_scale(unsigned top, float inv_sqrt_h) {
  const float m = __builtin_bit_cast(float, top);
  const bool fine = top < 0x7f800000u;
  Int8Scale r;
  r.pre = top < 0x0d800000u ? 18446744073709551616.0f : 1.0f;
  r.s = fine ? m * inv_sqrt_h / 127.0f : __builtin_nanf("");
  r.inv = r.s > 0.0f ? 127.0f / (m * r.pre) : 0.0f;
  r.keep = fine ? 0xffffffffu : 0u;
  return r;
}
__device__ __forceinline__ uint32_t int8_codes(const float* x, const Int8Scale& s) {
  uint32_t b[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) b[j] = __builtin_bit_cast(uint32_t, __builtin_fmaf(x[j], s.inv, 12582912.0f));
  const uint32_t lo = __builtin_amdgcn_perm(b[1], b[0], 0x0c0c0400u), hi = __builtin_amdgcn_perm(b[3], b[2], 0x04000c0cu);
  return (lo | hi) & s.keep;
}

hipError_t launch_int8_rows(const Int8RowArgs& a, int dtype, bool rotated, hipStream_t stream);

}  // namespace orbit
