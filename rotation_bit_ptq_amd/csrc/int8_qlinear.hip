// orbit_int8_qlinear: the product of 8-bit integers with a scale for each
// token and each channel,
//   y[m, n] = act(sx[m] sw[n] sum_k qx[m, k] qw[n, k] + bias[n]),
// on the int8 matrix cores; the sums are exact (int32), the scales, the bias
// and the activation float32, and y is rounded once.
//
// Two kernels.
// * tile_kernel, for products with enough tiles to fill the chip.  Bound: the
//   matrix cores.
// * thin_kernel, for few tokens or few tiles.  Bound: the weights' bytes, or
//   latency.
// Everywhere the weights are the matrix instruction's A operand (rows) and
// the tokens its B operand (columns), so that a lane's results are
// neighbouring channels of one token.
//
// K is a multiple of 16.  What lies past a row's end inside a 64-byte chunk is
// read at an address that is valid and multiplied as zero.
#include "block_common.h"

using namespace orbit;
using namespace orbit::block;

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));

struct ProductArgs {
  const char *x, *w;
  const float *sx, *sw;
  const void* bias;
  char* out;
  long long M, N;
  int K;
  int bias_dtype, out_dtype, act;
  int vec;  // output rows in 16-byte words
  int tiles_m, tiles_n;
};

__device__ __forceinline__ float bias_of(const ProductArgs& a, long long n) {
  if (!a.bias) return 0.0f;
  switch (a.bias_dtype) {
    case ORBIT_BF16: return (float)((const __bf16*)a.bias)[n];
    case ORBIT_F16: return (float)((const _Float16*)a.bias)[n];
    default: return ((const float*)a.bias)[n];
  }
}
// GELU in its erf form.
__device__ __forceinline__ float activate(float y, int act) {
  return act == ORBIT_ACT_GELU ? 0.5f * y * (1.0f + erff(y * 0.70710678118f)) : y;
}
template <class OT>
__device__ __forceinline__ void store8(OT* p, const float (&f)[8]) {
  Vec8<OT> v;
#pragma unroll
  for (int j = 0; j < 8; ++j) v.e[j] = (OT)f[j];
  *(Vec8<OT>*)p = v;
}

// Sums of `rows` tokens (from m0) and `cols` channels (from n0) that lie in
// LDS as int32 [rows][pitch], finished and stored by `threads` threads of
// which this is number t.
template <class OT>
__device__ __forceinline__ void finish(const ProductArgs& a, const int* sums, int pitch, int rows, int cols, long long m0,
                                       long long n0, int t, int threads) {
  if (a.vec) {
    const int per = cols / 8;            // vectors of a row
    const int at_once = threads / per;   // rows
    const int r0 = t / per, c = (t - r0 * per) * 8;
    const long long n = n0 + c;
    if (r0 >= at_once || n >= a.N) return;  // vec: N is a multiple of 8
    float sw[8], b[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      sw[j] = a.sw[n + j];
      b[j] = bias_of(a, n + j);
    }
    for (int r = r0; r < rows && m0 + r < a.M; r += at_once) {
      const float sx = a.sx[m0 + r];
      const i32x4 x = *(const i32x4*)(sums + r * pitch + c), y = *(const i32x4*)(sums + r * pitch + c + 4);
      float f[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = activate(fmaf((float)(j < 4 ? x[j & 3] : y[j & 3]), sx * sw[j], b[j]), a.act);
      store8((OT*)a.out + (m0 + r) * a.N + n, f);
    }
  } else {
    for (int i = t; i < rows * cols; i += threads) {
      const int r = i / cols, c = i - r * cols;
      if (m0 + r < a.M && n0 + c < a.N)
        ((OT*)a.out)[(m0 + r) * a.N + n0 + c] =
            (OT)activate(fmaf((float)sums[r * pitch + c], a.sx[m0 + r] * a.sw[n0 + c], bias_of(a, n0 + c)), a.act);
    }
  }
}

// ---- few tokens, few tiles ---------------------------------------------------
//
// A workgroup of eight waves takes 16 RB channels and up to 16 MB tokens;
// the waves take the 128-byte chunks w, w + 8, ... of K, two in flight ahead
// of the one that is multiplied, and add their sums in LDS (integers: the
// order does not matter).
template <class OT, int RB, int MB>
__global__ __launch_bounds__(512) void thin_kernel(ProductArgs a) {
  constexpr int kPitch = 16 * RB + 4;
  __shared__ __align__(16) int sums[16 * MB * kPitch];
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int r16 = lane & 15, kq = (lane >> 4) * 16;
  const long long n0 = (long long)blockIdx.x * (16 * RB), m0 = (long long)blockIdx.y * (16 * MB);
  const char *wrow[RB], *xrow[MB];
#pragma unroll
  for (int i = 0; i < RB; ++i) wrow[i] = a.w + min(n0 + 16 * i + r16, a.N - 1) * a.K;
#pragma unroll
  for (int i = 0; i < MB; ++i) xrow[i] = a.x + min(m0 + 16 * i + r16, a.M - 1) * a.K;
  for (int i = t; i < 16 * MB * kPitch; i += 512) sums[i] = 0;
  i32x4 acc[RB][MB];
#pragma unroll
  for (int i = 0; i < RB; ++i)
#pragma unroll
    for (int j = 0; j < MB; ++j) acc[i][j] = i32x4{0, 0, 0, 0};

  constexpr int kAhead = 2;
  i32x4 wv[kAhead][2][RB], xv[kAhead][2][MB];
  auto load = [&](int slot, int c) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int k = c * 128 + s * 64 + kq, at = min(k, a.K - 16);
#pragma unroll
      for (int i = 0; i < RB; ++i) wv[slot][s][i] = *(const i32x4*)(wrow[i] + at);
#pragma unroll
      for (int i = 0; i < MB; ++i) xv[slot][s][i] = *(const i32x4*)(xrow[i] + at);
    }
  };
  auto compute = [&](int slot, int c) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      if (c * 128 + s * 64 + 64 > a.K) {
        const bool in = c * 128 + s * 64 + kq < a.K;
#pragma unroll
        for (int i = 0; i < RB; ++i) wv[slot][s][i] = in ? wv[slot][s][i] : i32x4{0, 0, 0, 0};
      }
#pragma unroll
      for (int i = 0; i < RB; ++i)
#pragma unroll
        for (int j = 0; j < MB; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wv[slot][s][i], xv[slot][s][j], acc[i][j], 0, 0, 0);
    }
  };
  const int chunks = (a.K + 127) / 128;
#pragma unroll
  for (int p = 0; p < kAhead; ++p) load(p, wave + 8 * p);
  for (int c = wave; c < chunks; c += 8 * kAhead) {
#pragma unroll
    for (int p = 0; p < kAhead; ++p) {
      compute(p, c + 8 * p);  // a chunk past the end is all zeros
      load(p, c + 8 * (p + kAhead));
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < RB; ++i)
#pragma unroll
    for (int j = 0; j < MB; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        atomicAdd(&sums[(16 * j + r16) * kPitch + 16 * i + (lane >> 4) * 4 + q], acc[i][j][q]);
  __syncthreads();
  finish<OT>(a, sums, kPitch, 16 * MB, 16 * RB, m0, n0, t, 512);
}

template <class OT>
hipError_t launch_thin(const ProductArgs& a, hipStream_t stream) {
  const int mb = a.M <= 16 ? 1 : a.M <= 32 ? 2 : 4;
  const int64_t gm = (a.M + 16 * mb - 1) / (16 * mb);
  const bool wide = (a.N + 31) / 32 * gm >= kUnits;  // 32 channels a workgroup: half the token reads
  const dim3 grid((unsigned)((a.N + (wide ? 31 : 15)) / (wide ? 32 : 16)), (unsigned)gm), block(512);
  if (wide) {
    if (mb == 1) thin_kernel<OT, 2, 1><<<grid, block, 0, stream>>>(a);
    else if (mb == 2) thin_kernel<OT, 2, 2><<<grid, block, 0, stream>>>(a);
    else thin_kernel<OT, 2, 4><<<grid, block, 0, stream>>>(a);
  } else {
    if (mb == 1) thin_kernel<OT, 1, 1><<<grid, block, 0, stream>>>(a);
    else if (mb == 2) thin_kernel<OT, 1, 2><<<grid, block, 0, stream>>>(a);
    else thin_kernel<OT, 1, 4><<<grid, block, 0, stream>>>(a);
  }
  return hipGetLastError();
}

}  // namespace

extern "C" orbit_status orbit_int8_qlinear(const orbit_int8_qlinear_args* p, hipStream_t stream) {
  if (!p) return ORBIT_E_ARG;
  if (p->M < 0 || p->M >= ORBIT_MAX_ROWS || p->N < 0 || p->N >= ORBIT_MAX_ROWS) return ORBIT_E_SHAPE;
  if (p->K < 16 || p->K > 65536 || p->K % 16) return ORBIT_E_SHAPE;
  if (!is_dtype(p->out_dtype) || (p->bias && !is_dtype(p->bias_dtype))) return ORBIT_E_DTYPE;
  if (p->act != ORBIT_ACT_NONE && p->act != ORBIT_ACT_GELU) return ORBIT_E_ARG;
  if (p->M == 0 || p->N == 0) return ORBIT_OK;
  if (!p->qx || !p->qw || !p->sx || !p->sw || !p->out) return ORBIT_E_ARG;
  if (!aligned_to(p->qx, 16) || !aligned_to(p->qw, 16) || !aligned_to(p->sx, 4) || !aligned_to(p->sw, 4)) return ORBIT_E_ARG;
  if (!aligned_to(p->out, dtype_bytes(p->out_dtype)) || (p->bias && !aligned_to(p->bias, dtype_bytes(p->bias_dtype)))) return ORBIT_E_ARG;
  ProductArgs a = {};
  a.x = (const char*)p->qx;
  a.w = (const char*)p->qw;
  a.sx = p->sx;
  a.sw = p->sw;
  a.bias = p->bias;
  a.out = (char*)p->out;
  a.M = p->M;
  a.N = p->N;
  a.K = (int)p->K;
  a.bias_dtype = p->bias_dtype;
  a.out_dtype = p->out_dtype;
  a.act = p->act;
  a.vec = vector_rows(p->out, p->N);
  hipError_t e;
  switch (p->out_dtype) {
    case ORBIT_BF16: e = launch_thin<__bf16>(a, stream); break;
    case ORBIT_F16: e = launch_thin<_Float16>(a, stream); break;
    default: e = launch_thin<float>(a, stream);
  }
  return hip_status(e);
}
