// Norms around a residual sum (orbit_block_norm):
//   b^ = post(branch) * post_weight;  r = rho x + gate b^;
//   y = norm(r) * weight * (1 + scale) + shift.
//
// Bound: memory (12 or so float operations per element against 6 .. 12
// bytes).  One pass: a row stays in the registers of the waves that loaded
// it, so x and the branch are read once and r and y written once, whatever
// the number of norms.  A layer norm centres the registers' values before it
// squares them (no E[v^2] - mean^2 cancellation).
#pragma once

#include "block_common.h"

namespace orbit {
namespace block {

struct NormArgs {
  const char *x, *branch;
  char *r, *y;
  const char *weight, *post_weight, *gate, *scale, *shift;
  const int32_t* group_ids;
  long long xs, bs, rs, ys, gs, scs, shs;  // row strides, elements
  uint32_t rows, groups, rows_per_group;
  int dim, waves;  // waves per row
  int p_dtype, norm, post;
  float rho, eps, width;  // width: dim as a float
};

// A vector of parameters as loaded: 16-bit types take `a` alone.
struct ParamRaw {
  u32x4 a, b;
};

template <bool VEC>
__device__ __forceinline__ ParamRaw load_param(const char* p, long long off, int e0, int step, int dim, int dt) {
  ParamRaw r;
  if constexpr (VEC) {
    if (dt == ORBIT_F32) {
      const u32x4* q = (const u32x4*)(p + 4 * (off + e0));
      r.a = q[0];
      r.b = q[1];
    } else {
      r.a = *(const u32x4*)(p + 2 * (off + e0));
    }
  } else {
    float f[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int e = e0 + j * step;
      f[j] = 0.0f;
      if (e < dim)
        f[j] = dt == ORBIT_F32    ? ((const float*)p)[off + e]
               : dt == ORBIT_BF16 ? (float)((const __bf16*)p)[off + e]
                                  : (float)((const _Float16*)p)[off + e];
    }
    r.a = __builtin_bit_cast(u32x4, f32x4{f[0], f[1], f[2], f[3]});
    r.b = __builtin_bit_cast(u32x4, f32x4{f[4], f[5], f[6], f[7]});
  }
  return r;
}

__device__ __forceinline__ void param_f32(const ParamRaw& r, int dt, float (&f)[8]) {
  if (dt == ORBIT_F32) {
    const f32x4 a = __builtin_bit_cast(f32x4, r.a), b = __builtin_bit_cast(f32x4, r.b);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f[j] = a[j];
      f[4 + j] = b[j];
    }
  } else if (dt == ORBIT_BF16) {
    const bf16x8 h = __builtin_bit_cast(bf16x8, r.a);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = (float)h[j];
  } else {
    const f16x8 h = __builtin_bit_cast(f16x8, r.a);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = (float)h[j];
  }
}

template <class T, bool VEC>
__device__ __forceinline__ Vec8<T> load_row(const char* p, long long off, int e0, int step, int dim) {
  Vec8<T> v;
  if constexpr (VEC) {
    v = *(const Vec8<T>*)((const T*)p + off + e0);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int e = e0 + j * step;
      v.e[j] = e < dim ? ((const T*)p)[off + e] : (T)0.0f;
    }
  }
  return v;
}

template <class T, bool VEC>
__device__ __forceinline__ void store_row(char* p, long long off, int e0, int step, int dim, const float (&f)[8]) {
  Vec8<T> v;
#pragma unroll
  for (int j = 0; j < 8; ++j) v.e[j] = (T)f[j];
  if constexpr (VEC) {
    *(Vec8<T>*)((T*)p + off + e0) = v;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int e = e0 + j * step;
      if (e < dim) ((T*)p)[off + e] = v.e[j];
    }
  }
}

// ITEMS vectors of eight per thread.  VEC: a thread's eight elements lie side
// by side (16-byte accesses; dim and every stride whole vectors); otherwise
// neighbouring threads take neighbouring elements, one at a time.
template <class XT, class BT, class YT, int ITEMS, bool VEC>
__global__ __launch_bounds__(ITEMS == 1 ? 512 : 1024) void norm_kernel(NormArgs a) {
  __shared__ float red[4][16];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int W = a.waves;
  const int wr = W == 1 ? 0 : wave;  // this wave among its row's
  const uint32_t row = W == 1 ? blockIdx.x * (blockDim.x >> 6) + wave : blockIdx.x;
  if (row >= a.rows) return;  // W == 1 only: no barrier follows
  const int T = W << 6, t = (wr << 6) + lane;
  const int step = VEC ? 1 : T;
  const int dt = VEC ? a.p_dtype : (int)ORBIT_F32;
  int e0[ITEMS];
  bool on[ITEMS];
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    e0[i] = VEC ? (i * T + t) * 8 : i * 8 * T + t;
    on[i] = e0[i] < a.dim;
  }

  Vec8<XT> xv[ITEMS];
  Vec8<BT> bv[ITEMS];
#pragma unroll
  for (int i = 0; i < ITEMS; ++i)
    if (on[i]) xv[i] = load_row<XT, VEC>(a.x, row * a.xs, e0[i], step, a.dim);
  if (a.branch) {
#pragma unroll
    for (int i = 0; i < ITEMS; ++i)
      if (on[i]) bv[i] = load_row<BT, VEC>(a.branch, row * a.bs, e0[i], step, a.dim);
  }
  uint32_t g = a.group_ids ? (uint32_t)a.group_ids[row] : row / a.rows_per_group;
  const bool modulated = g < a.groups;
  const char* const gate = modulated ? a.gate : nullptr;
  const char* const scale = modulated ? a.scale : nullptr;
  const char* const shift = modulated ? a.shift : nullptr;

  // the parameters' loads are in flight during the reductions
  ParamRaw wraw[ITEMS], praw[ITEMS], graw[ITEMS], craw[ITEMS], hraw[ITEMS];
  auto fetch = [&](ParamRaw (&raw)[ITEMS], const char* p, long long off) {
    if (p) {
#pragma unroll
      for (int i = 0; i < ITEMS; ++i)
        if (on[i]) raw[i] = load_param<VEC>(p, off, e0[i], step, a.dim, a.p_dtype);
    }
  };
  fetch(praw, a.post_weight, 0);
  fetch(graw, gate, g * a.gs);
  if (ITEMS == 1) {
    fetch(wraw, a.weight, 0);
    fetch(craw, scale, g * a.scs);
    fetch(hraw, shift, g * a.shs);
  }

  int round = 0;
  auto row_sum = [&](float v) {
    v = wave_sum(v);
    if (W > 1) {
      if (lane == 0) red[round][wave] = v;
      __syncthreads();
      v = red[round][0];
      for (int w = 1; w < W; ++w) v += red[round][w];
      ++round;
    }
    return v;
  };
  // v becomes v / sqrt(mean v^2 + eps), centred first for a layer norm
  auto normalize = [&](float (&v)[ITEMS][8], int kind) {
    if (kind == ORBIT_NORM_LAYER) {
      float s = 0.0f;
#pragma unroll
      for (int i = 0; i < ITEMS; ++i)
        if (on[i]) {
#pragma unroll
          for (int j = 0; j < 8; ++j) s += v[i][j];
        }
      const float mean = row_sum(s) / a.width;  // a quotient: exact for equal values
#pragma unroll
      for (int i = 0; i < ITEMS; ++i)
        if (on[i]) {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            v[i][j] = VEC || e0[i] + j * step < a.dim ? v[i][j] - mean : 0.0f;
        }
    }
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i)
      if (on[i]) {
#pragma unroll
        for (int j = 0; j < 8; ++j) s = fmaf(v[i][j], v[i][j], s);
      }
    const float inv = 1.0f / sqrtf(row_sum(s) / a.width + a.eps);
#pragma unroll
    for (int i = 0; i < ITEMS; ++i)
      if (on[i]) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] *= inv;
      }
  };

  float v[ITEMS][8];
  float f[8];
  if (a.branch) {
#pragma unroll
    for (int i = 0; i < ITEMS; ++i)
      if (on[i]) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = (float)bv[i].e[j];
      }
    if (a.post != ORBIT_NORM_NONE) normalize(v, a.post);
#pragma unroll
    for (int i = 0; i < ITEMS; ++i)
      if (on[i]) {
        if (a.post_weight) {
          param_f32(praw[i], dt, f);
#pragma unroll
          for (int j = 0; j < 8; ++j) v[i][j] *= f[j];
        }
        if (gate) {
          param_f32(graw[i], dt, f);
#pragma unroll
          for (int j = 0; j < 8; ++j) v[i][j] *= f[j];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = fmaf(a.rho, (float)xv[i].e[j], v[i][j]);
        store_row<XT, VEC>(a.r, row * a.rs, e0[i], step, a.dim, v[i]);
      }
  } else {
#pragma unroll
    for (int i = 0; i < ITEMS; ++i)
      if (on[i]) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = (float)xv[i].e[j];
      }
  }
  if (a.norm == ORBIT_NORM_NONE) return;
  if (ITEMS > 1) {
    fetch(wraw, a.weight, 0);
    fetch(craw, scale, g * a.scs);
    fetch(hraw, shift, g * a.shs);
  }
  normalize(v, a.norm);
#pragma unroll
  for (int i = 0; i < ITEMS; ++i)
    if (on[i]) {
      if (a.weight) {
        param_f32(wraw[i], dt, f);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] *= f[j];
      }
      if (scale) {
        param_f32(craw[i], dt, f);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = fmaf(v[i][j], f[j], v[i][j]);
      }
      if (shift) {
        param_f32(hraw[i], dt, f);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] += f[j];
      }
      store_row<YT, VEC>(a.y, row * a.ys, e0[i], step, a.dim, v[i]);
    }
}

// One wave takes a row of up to 512 elements (four rows to a workgroup),
// more waves share a longer one.
template <class XT, class BT, class YT, bool VEC>
hipError_t launch_norm_t(NormArgs& a, hipStream_t stream) {
  const int chunks = (a.dim + 511) / 512;  // waves with one vector per lane
  if (chunks <= 8) {
    a.waves = chunks;
    const unsigned threads = chunks == 1 ? 256u : 64u * chunks;
    const unsigned blocks = chunks == 1 ? (a.rows + 3) / 4 : a.rows;
    norm_kernel<XT, BT, YT, 1, VEC><<<dim3(blocks), dim3(threads), 0, stream>>>(a);
  } else {
    a.waves = (chunks + 1) / 2;
    norm_kernel<XT, BT, YT, 2, VEC><<<dim3(a.rows), dim3(64u * a.waves), 0, stream>>>(a);
  }
  return hipGetLastError();
}

template <class XT, class BT, class YT>
hipError_t launch_norm(NormArgs& a, bool vec, hipStream_t stream) {
  return vec ? launch_norm_t<XT, BT, YT, true>(a, stream) : launch_norm_t<XT, BT, YT, false>(a, stream);
}

// x F32: any branch and output type (block_norm_f32.hip).
hipError_t launch_norm_f32(NormArgs& a, int b_dtype, int y_dtype, bool vec, hipStream_t stream);

}  // namespace block
}  // namespace orbit
