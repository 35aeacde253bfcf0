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
  double inv_sqrt_h;
};

hipError_t launch_int8_rows(const Int8RowArgs& a, int dtype, bool rotated, hipStream_t stream);

}  // namespace orbit
