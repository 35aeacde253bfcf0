// orbit_adapter_add: low-rank adapters of many requests beside a shared
// projection, out[m] = y[m] + s_a B_a (A_a x[m]), a = ids[m].
//
// Bound: memory (x, y and out once; the adapters in use once, then from L2).
// Two launches: v = A x into the workspace, then out = y + s B v; v stays in
// float32.
#include "block_common.h"

using namespace orbit;
using namespace orbit::block;

namespace {

struct AdapterArgs {
  const char *x, *A, *B, *y;
  char* out;
  const int32_t *ids, *ranks;
  const float* scale;
  float* v;
  long long xs, ys, os;
  uint32_t M, adapters;
  int K, N, R;
};

// The adapter's rank, 0 where there is none.
__device__ __forceinline__ int rank_of(const AdapterArgs& a, int id) {
  if ((uint32_t)id >= a.adapters) return 0;
  const int r = a.ranks ? a.ranks[id] : a.R;
  return r < 0 ? 0 : r < a.R ? r : a.R;
}

// v[m][r] = A[id][r] . x[m]: a wave per (row, rank).
template <class T>
__global__ __launch_bounds__(256) void shrink_rows_kernel(AdapterArgs a) {
  const uint32_t m = blockIdx.x;
  const int r = blockIdx.y * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int id = a.ids[m];
  if (r >= rank_of(a, id)) return;
  const T* const x = (const T*)a.x + m * a.xs;
  const T* const w = (const T*)a.A + ((long long)id * a.R + r) * a.K;
  float s = 0.0f;
#pragma unroll 4
  for (int k = lane * 8; k < a.K; k += 512) {
    const Vec8<T> p = *(const Vec8<T>*)(x + k), q = *(const Vec8<T>*)(w + k);
#pragma unroll
    for (int j = 0; j < 8; ++j) s = fmaf((float)p.e[j], (float)q.e[j], s);
  }
  s = wave_sum(s);
  if (lane == 0) a.v[(long long)m * a.R + r] = s;
}

// out[m][n] = y[m][n] + s B[id][n] . v[m]: a thread per column.
template <class T, class YT>
__global__ __launch_bounds__(256) void expand_rows_kernel(AdapterArgs a) {
  __shared__ float v[128];
  const uint32_t m = blockIdx.x;
  const int n = blockIdx.y * 256 + threadIdx.x;
  const int id = a.ids[m], rank = rank_of(a, id);
  if (rank > 0) {
    const float s = a.scale ? a.scale[id] : 1.0f;
    if ((int)threadIdx.x < a.R) v[threadIdx.x] = (int)threadIdx.x < rank ? a.v[(long long)m * a.R + threadIdx.x] * s : 0.0f;
  }
  __syncthreads();
  if (n >= a.N) return;
  float f = (float)((const YT*)a.y)[m * a.ys + n];
  if (rank > 0) {
    const T* const w = (const T*)a.B + ((long long)id * a.N + n) * a.R;
    float d = 0.0f;
    for (int r = 0; r < rank; r += 8) {
      const Vec8<T> q = *(const Vec8<T>*)(w + r);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (r + j < rank) d = fmaf((float)q.e[j], v[r + j], d);
    }
    f += d;
  }
  ((YT*)a.out)[m * a.os + n] = (YT)f;
}

template <class T>
hipError_t launch(const AdapterArgs& a, int y_dtype, hipStream_t stream) {
  shrink_rows_kernel<T><<<dim3(a.M, (a.R + 3) / 4), dim3(256), 0, stream>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const dim3 grid(a.M, (a.N + 255) / 256);
  switch (y_dtype) {
    case ORBIT_BF16: expand_rows_kernel<T, __bf16><<<grid, dim3(256), 0, stream>>>(a); break;
    case ORBIT_F16: expand_rows_kernel<T, _Float16><<<grid, dim3(256), 0, stream>>>(a); break;
    default: expand_rows_kernel<T, float><<<grid, dim3(256), 0, stream>>>(a);
  }
  return hipGetLastError();
}

bool sizes_ok(int64_t M, int64_t K, int64_t rank) {
  return M >= 0 && M < ORBIT_MAX_ROWS && K >= 8 && K <= 65536 && K % 8 == 0 && rank >= 8 && rank <= 128 && rank % 8 == 0;
}

}  // namespace

extern "C" int64_t orbit_adapter_workspace(int64_t M, int64_t K, int64_t rank) {
  if (!sizes_ok(M, K, rank)) return -1;
  return M * rank * 4;
}

extern "C" orbit_status orbit_adapter_add(const orbit_adapter_args* p, hipStream_t stream) {
  if (!p) return ORBIT_E_ARG;
  if (!sizes_ok(p->M, p->K, p->rank) || p->N < 0 || p->N > (1LL << 22)) return ORBIT_E_SHAPE;
  if (p->adapters < 0 || p->adapters >= (1LL << 31)) return ORBIT_E_SHAPE;
  if (p->x_dtype != ORBIT_BF16 && p->x_dtype != ORBIT_F16) return ORBIT_E_DTYPE;
  if (!is_dtype(p->y_dtype)) return ORBIT_E_DTYPE;
  if (p->x_stride < 0 || p->y_stride < 0) return ORBIT_E_SHAPE;
  if (p->M == 0 || p->N == 0) return ORBIT_OK;
  const int64_t yb = dtype_bytes(p->y_dtype);
  if (!p->x || !p->y || !p->out || !p->ids || !aligned_to(p->ids, 4)) return ORBIT_E_ARG;
  if (!vector_rows(p->x, p->x_stride) || !aligned_to(p->y, yb) || !aligned_to(p->out, yb)) return ORBIT_E_ARG;
  if (p->adapters > 0 && (!p->A || !p->B || !aligned_to(p->A, 16) || !aligned_to(p->B, 16))) return ORBIT_E_ARG;
  if ((p->ranks && !aligned_to(p->ranks, 4)) || (p->scale && !aligned_to(p->scale, 4))) return ORBIT_E_ARG;
  if (p->M > 1 && p->out_stride < p->N) return ORBIT_E_SHAPE;  // output rows that overlap would race
  if (!p->workspace || !aligned_to(p->workspace, 16) ||
      p->workspace_bytes < orbit_adapter_workspace(p->M, p->K, p->rank))
    return ORBIT_E_ARG;
  AdapterArgs a = {};
  a.x = (const char*)p->x;
  a.A = (const char*)p->A;
  a.B = (const char*)p->B;
  a.y = (const char*)p->y;
  a.out = (char*)p->out;
  a.ids = p->ids;
  a.ranks = p->ranks;
  a.scale = p->scale;
  a.v = (float*)p->workspace;
  a.xs = p->x_stride;
  a.ys = p->y_stride;
  a.os = p->out_stride;
  a.M = (uint32_t)p->M;
  a.adapters = (uint32_t)p->adapters;
  a.K = (int)p->K;
  a.N = (int)p->N;
  a.R = (int)p->rank;
  return hip_status(p->x_dtype == ORBIT_BF16 ? launch<__bf16>(a, p->y_dtype, stream) : launch<_Float16>(a, p->y_dtype, stream));
}
