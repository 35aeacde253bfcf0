// Norms around a residual sum (orbit_block_norm):
//   b^ = post(branch) * post_weight;  r = rho x + gate b^;
//   y = norm(r) * weight * (1 + scale) + shift.
//
// Bound: memory (12 or so float operations per element against 6 .. 12
// bytes).  One pass: a row stays in the registers of the waves that loaded
// it, so x and the branch are read once and r and y written once, whatever
// the number of norms.  A lane holds one vector of eight neighbouring
// elements (two, past 4096), so that registers stay few and many waves have
// their loads in flight: with up to eight vectors per lane and one wave per
// row, without any barrier, 16384 rows of 3072 took 133 us.  The parameters'
// loads go out before the reductions and come from L1 or L2.  4096 x 3072
// bf16 with gate, scale and shift: 21 us (4.8 TB/s, a copy's rate); 32768 x
// 2048 float32 with float32 parameters and a norm on both sides: 188 us (4.3
// TB/s: a row's parameters are 40 KB from L2 beside its 24 KB).
//
// A layer norm centres the values before it squares them: each wave about
// its own mean, joined by M2 = sum M2_w + sum n_w (mean_w - mean)^2, which
// takes one exchange through LDS instead of two and cancels nothing.
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

// Eight elements as loaded, 16 or 32 bytes: kept as they came until they are
// used, so that no load waits for another.
template <int BYTES>
struct Raw {
  u32x4 w[BYTES / 16];
};

// A vector of a row at any address its type allows (16-byte accesses need no
// alignment on this device).  The load is unconditional: a lane past the end
// reads the row's last eight elements.  TAIL: rows may end inside a vector;
// that vector is read from the row's last eight and moved down, zeros behind.
template <class T, bool TAIL>
__device__ __forceinline__ Raw<8 * sizeof(T)> load_eight(const T* row, int e0, int dim) {
  Raw<8 * sizeof(T)> v;
  if (TAIL && dim < 8) {
    T e[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) e[j] = e0 + j < dim ? row[e0 + j] : (T)0;
    __builtin_memcpy(&v, e, sizeof v);
    return v;
  }
  const int at = min(e0, dim - 8);
  __builtin_memcpy(&v, row + at, sizeof v);
  if constexpr (TAIL) {
    constexpr int kWords = 2 * sizeof(T);
    const int shift = min(e0 - at, 8);
    uint32_t w[kWords];
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = v.w[i / 4][i % 4];
    const int words = sizeof(T) == 4 ? shift : shift >> 1;
#pragma unroll
    for (int by = 1; by <= kWords; by *= 2)
#pragma unroll
      for (int i = 0; i < kWords; ++i) w[i] = words & by ? (i + by < kWords ? w[i + by] : 0u) : w[i];
    if (sizeof(T) == 2) {
#pragma unroll
      for (int i = 0; i < kWords; ++i) w[i] = shift & 1 ? (w[i] >> 16) | (i + 1 < kWords ? w[i + 1] << 16 : 0u) : w[i];
    }
#pragma unroll
    for (int i = 0; i < kWords; ++i) v.w[i / 4][i % 4] = w[i];
  }
  return v;
}
template <class T>
__device__ __forceinline__ void unpack(const Raw<8 * sizeof(T)>& v, float (&f)[8]) {
  const Vec8<T> t = __builtin_bit_cast(Vec8<T>, v);
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] = (float)t.e[j];
}
template <bool TAIL, class T>
__device__ __forceinline__ void store_eight(T* p, int n, const float (&f)[8]) {
  Vec8<T> v;
#pragma unroll
  for (int j = 0; j < 8; ++j) v.e[j] = (T)f[j];
  if (!TAIL || n >= 8) {
    __builtin_memcpy(p, &v, sizeof v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) p[j] = v.e[j];
  }
}

// Eight parameters (P32: float32; otherwise bf16 or fp16 by dtype).
template <bool P32>
__device__ __forceinline__ void param(const Raw<P32 ? 32 : 16>& v, int dtype, float (&f)[8]) {
  if constexpr (P32) unpack<float>(v, f);
  else if (dtype == ORBIT_BF16) unpack<__bf16>(v, f);
  else unpack<_Float16>(v, f);
}

template <class XT, class BT, class YT, bool P32, int ITEMS, bool TAIL>
__global__ __launch_bounds__(ITEMS == 1 ? 512 : 1024) void norm_kernel(NormArgs a) {
  __shared__ float2 red[2][16];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int W = a.waves;
  const int wr = W == 1 ? 0 : wave;  // this wave among its row's
  const uint32_t row = W == 1 ? blockIdx.x * (blockDim.x >> 6) + wave : blockIdx.x;
  if (row >= a.rows) return;  // W == 1 only: no barrier follows
  int e0[ITEMS], n[ITEMS];    // a vector's first element; how many of its eight exist
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    e0[i] = ((i * W + wr) * 64 + lane) * 8;
    n[i] = a.dim - e0[i];
  }

  Raw<8 * sizeof(XT)> xv[ITEMS];
  Raw<8 * sizeof(BT)> bv[ITEMS];
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) xv[i] = load_eight<XT, TAIL>((const XT*)a.x + row * a.xs, e0[i], a.dim);
  if (a.branch) {
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) bv[i] = load_eight<BT, TAIL>((const BT*)a.branch + row * a.bs, e0[i], a.dim);
  }
  const uint32_t g = a.group_ids ? (uint32_t)a.group_ids[row] : row / a.rows_per_group;
  const bool modulated = g < a.groups;
  const char* const gate = modulated ? a.gate : nullptr;
  const char* const scale = modulated ? a.scale : nullptr;
  const char* const shift = modulated ? a.shift : nullptr;
  typedef typename std::conditional<P32, float, unsigned short>::type PT;
  Raw<8 * sizeof(PT)> wp[ITEMS], pp[ITEMS], gp[ITEMS], cp[ITEMS], hp[ITEMS];
  auto fetch = [&](Raw<8 * sizeof(PT)> (&to)[ITEMS], const char* p, long long at) {
    if (p) {
#pragma unroll
      for (int i = 0; i < ITEMS; ++i) to[i] = load_eight<PT, TAIL>((const PT*)p + at, e0[i], a.dim);
    }
  };
  fetch(pp, a.post_weight, 0);
  fetch(gp, gate, g * a.gs);
  fetch(wp, a.weight, 0);
  fetch(cp, scale, g * a.scs);
  fetch(hp, shift, g * a.shs);

  int round = 0;
  // v becomes v / sqrt(mean v^2 + eps), centred first for a layer norm
  auto normalize = [&](float (&v)[ITEMS][8], int kind) {
    float mean = 0.0f, sum = 0.0f, square = 0.0f;
    int count = 0;  // of this wave's elements
    if (kind == ORBIT_NORM_LAYER) {
#pragma unroll
      for (int i = 0; i < ITEMS; ++i) {
        count += min(max(a.dim - (i * W + wr) * 512, 0), 512);
        if (n[i] > 0) {
#pragma unroll
          for (int j = 0; j < 8; ++j) sum += v[i][j];  // zeros past the row's end
        }
      }
      sum = wave_sum(sum);
      mean = sum / (float)count;  // a quotient: exact for equal values
    }
#pragma unroll
    for (int i = 0; i < ITEMS; ++i)
      if (n[i] > 0) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float d = !TAIL || j < n[i] ? v[i][j] - mean : 0.0f;
          square = fmaf(d, d, square);
        }
      }
    square = wave_sum(square);
    if (W > 1) {
      if (lane == 0) red[round][wave] = make_float2(sum, square);
      __syncthreads();
      // every row of 16 lanes adds up the waves' parts, a lane to each
      const int w = lane & 15;
      float2 q = red[round][w];
      if (w >= W) q = make_float2(0.0f, 0.0f);
      if (kind == ORBIT_NORM_LAYER) {
        mean = row_sum(q.x) / a.width;
        int m = 0;
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) m += min(max(a.dim - (i * W + w) * 512, 0), 512);
        const float d = w < W ? q.x / (float)m - mean : 0.0f;
        q.y = fmaf((float)m * d, d, q.y);
      }
      square = row_sum(q.y);
      ++round;
    }
    const float inv = 1.0f / sqrtf(square / a.width + a.eps);
#pragma unroll
    for (int i = 0; i < ITEMS; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = (v[i][j] - mean) * inv;
  };

  float v[ITEMS][8], f[8];
  if (a.branch) {
#pragma unroll
    for (int i = 0; i < ITEMS; ++i)
      unpack<BT>(bv[i], v[i]);
    if (a.post != ORBIT_NORM_NONE) normalize(v, a.post);
#pragma unroll
    for (int i = 0; i < ITEMS; ++i)
      if (n[i] > 0) {
        if (a.post_weight) {
          param<P32>(pp[i], a.p_dtype, f);
#pragma unroll
          for (int j = 0; j < 8; ++j) v[i][j] *= f[j];
        }
        if (gate) {
          param<P32>(gp[i], a.p_dtype, f);
#pragma unroll
          for (int j = 0; j < 8; ++j) v[i][j] *= f[j];
        }
        // past the row's end zeros, for the sums of the next norm
        unpack<XT>(xv[i], f);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = !TAIL || j < n[i] ? fmaf(a.rho, f[j], v[i][j]) : 0.0f;
        store_eight<TAIL>((XT*)a.r + row * a.rs + e0[i], n[i], v[i]);
      }
  } else {
#pragma unroll
    for (int i = 0; i < ITEMS; ++i)
      unpack<XT>(xv[i], v[i]);
  }
  if (a.norm == ORBIT_NORM_NONE) return;
  normalize(v, a.norm);
#pragma unroll
  for (int i = 0; i < ITEMS; ++i)
    if (n[i] > 0) {
      if (a.weight) {
        param<P32>(wp[i], a.p_dtype, f);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] *= f[j];
      }
      if (scale) {
        param<P32>(cp[i], a.p_dtype, f);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = fmaf(v[i][j], f[j], v[i][j]);
      }
      if (shift) {
        param<P32>(hp[i], a.p_dtype, f);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] += f[j];
      }
      store_eight<TAIL>((YT*)a.y + row * a.ys + e0[i], n[i], v[i]);
    }
}

// One wave takes a row of up to 512 elements (four rows to a workgroup),
// eight a row of up to 4096, sixteen of up to 16384.
template <class XT, class BT, class YT, bool P32>
hipError_t launch_norm_p(NormArgs& a, hipStream_t stream) {
  const int vectors = (a.dim + 511) / 512;  // per lane of one wave
  a.waves = vectors <= 8 ? vectors : (vectors + 1) / 2;
  const dim3 block(a.waves == 1 ? 256u : 64u * a.waves), grid(a.waves == 1 ? (a.rows + 3) / 4 : a.rows);
  if (a.dim % 8 == 0) {
    if (vectors <= 8) norm_kernel<XT, BT, YT, P32, 1, false><<<grid, block, 0, stream>>>(a);
    else norm_kernel<XT, BT, YT, P32, 2, false><<<grid, block, 0, stream>>>(a);
  } else {
    if (vectors <= 8) norm_kernel<XT, BT, YT, P32, 1, true><<<grid, block, 0, stream>>>(a);
    else norm_kernel<XT, BT, YT, P32, 2, true><<<grid, block, 0, stream>>>(a);
  }
  return hipGetLastError();
}

template <class XT, class BT, class YT>
hipError_t launch_norm(NormArgs& a, hipStream_t stream) {
  return a.p_dtype == ORBIT_F32 ? launch_norm_p<XT, BT, YT, true>(a, stream) : launch_norm_p<XT, BT, YT, false>(a, stream);
}

// x F32: any branch and output type (block_norm_f32.hip).
hipError_t launch_norm_f32(NormArgs& a, int b_dtype, int y_dtype, hipStream_t stream);

}  // namespace block
}  // namespace orbit
