// Shared device helpers of the operators between a block's quantized
// projections: element types, vectors of eight, and reductions over a wave.
#pragma once

#include <hip/hip_runtime.h>

#include <stdint.h>

#include <type_traits>

#include "orbit_internal.h"

namespace orbit {
namespace block {

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// Compute units that a launch should fill (the whole device; splits are
// chosen from sizes alone, so that workspaces can be sized without asking it).
constexpr int kUnits = 256;

// Eight neighbouring elements, loaded and stored as 16-byte words.
template <class T>
struct alignas(16) Vec8 {
  T e[8];
};

inline int64_t dtype_bytes(int dt) { return dt == ORBIT_F32 ? 4 : 2; }
inline bool is_dtype(int dt) { return dt == ORBIT_F32 || dt == ORBIT_BF16 || dt == ORBIT_F16; }
inline bool aligned_to(const void* p, int64_t bytes) { return ((uintptr_t)p & (uintptr_t)(bytes - 1)) == 0; }
// Rows that eight-element vectors may read: 16-byte base, strides in whole
// vectors.
inline bool vector_rows(const void* p, int64_t stride) { return aligned_to(p, 16) && stride % 8 == 0; }

// One 16x16x32 product.  Lane l holds row (A) or column (B) l % 16 at k = 8
// (l / 16) + 0 .. 7, and of the result column l % 16, rows 4 (l / 16) + 0 .. 3.
__device__ __forceinline__ f32x4 mma(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mma(f16x8 a, f16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}
template <class T>
struct Vec8Of;
template <>
struct Vec8Of<__bf16> {
  typedef bf16x8 V;
};
template <>
struct Vec8Of<_Float16> {
  typedef f16x8 V;
};

template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) {
  const int o = __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true);
  return v + __builtin_bit_cast(float, o);
}
template <int CTRL>
__device__ __forceinline__ float dpp_max(float v) {
  const int o = __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true);
  return fmaxf(v, __builtin_bit_cast(float, o));
}
constexpr int kXor1 = 0xB1, kXor2 = 0x4E;               // quad_perm [1,0,3,2], [2,3,0,1]
constexpr int kHalfMirror = 0x141, kRowMirror = 0x140;  // after the quads: lanes 4 and 8 apart

// Sums of the two halves (32 lanes) or the neighbouring rows (16 lanes) of a
// wave, in every lane: the swap puts one half's values beside the other's.
__device__ __forceinline__ float add_rows16(float v) {
  const unsigned u = __builtin_bit_cast(unsigned, v);
  const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  return __builtin_bit_cast(float, (unsigned)r[0]) + __builtin_bit_cast(float, (unsigned)r[1]);
}
__device__ __forceinline__ float add_rows32(float v) {
  const unsigned u = __builtin_bit_cast(unsigned, v);
  const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return __builtin_bit_cast(float, (unsigned)r[0]) + __builtin_bit_cast(float, (unsigned)r[1]);
}
__device__ __forceinline__ float max_rows16(float v) {
  const unsigned u = __builtin_bit_cast(unsigned, v);
  const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  return fmaxf(__builtin_bit_cast(float, (unsigned)r[0]), __builtin_bit_cast(float, (unsigned)r[1]));
}
__device__ __forceinline__ float max_rows32(float v) {
  const unsigned u = __builtin_bit_cast(unsigned, v);
  const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return fmaxf(__builtin_bit_cast(float, (unsigned)r[0]), __builtin_bit_cast(float, (unsigned)r[1]));
}

// Sum over each row of 16 lanes, and over the wave: the same bits in every
// lane of the row, of the wave.
__device__ __forceinline__ float row_sum(float v) {
  v = dpp_add<kXor1>(v);
  v = dpp_add<kXor2>(v);
  v = dpp_add<kHalfMirror>(v);
  return dpp_add<kRowMirror>(v);
}
__device__ __forceinline__ float wave_sum(float v) { return add_rows32(add_rows16(row_sum(v))); }

}  // namespace block
}  // namespace orbit
