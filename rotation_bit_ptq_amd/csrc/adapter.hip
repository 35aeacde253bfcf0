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
  int parts, k_part;  // K in parts of k_part, a workgroup each
  int columns;        // blocks of 256 columns per workgroup
};

constexpr int kWaves = 4;
constexpr int kRowsAtMost = 64;   // tokens up to which rows go one by one
constexpr int kPartsAtMost = 16;  // parts of K

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

// The distinct adapters of a tile of up to 64 rows, one after the other.
// Lane l holds row l's adapter (-1: none, or past the tile).
struct Requests {
  unsigned long long rest;
  int id, rank;
  unsigned long long rows;  // the rows of `id`

  __device__ __forceinline__ void begin(int mine) { rest = __ballot(mine >= 0); }
  __device__ __forceinline__ bool next(const AdapterArgs& a, int mine) {
    if (rest == 0) return false;
    id = __builtin_amdgcn_readlane(mine, __builtin_ctzll(rest));
    rows = __ballot(mine == id);
    rest &= ~rows;
    rank = rank_of(a, id);
    return true;
  }
};

// This lane's row's adapter if it has one of rank > 0, else -1.
template <int TM>
__device__ __forceinline__ int my_request(const AdapterArgs& a, uint32_t m0, int lane) {
  if (lane >= TM || m0 + lane >= a.M) return -1;
  const int id = a.ids[m0 + lane];
  return rank_of(a, id) > 0 ? id : -1;
}

// v = A x for tiles of 16 MB rows, ranks up to 16 RB, on the matrix cores:
// rows of x are the A operand, rows of the adapter's A the B operand, both
// straight from memory (16 contiguous bytes of a lane are an operand's
// slots).  The four waves share the workgroup's part of K, so each loads
// its piece of x once for all RB blocks of ranks; their sums meet in LDS.
// blockIdx.y takes part blockIdx.y of K: the parts are summed, in a fixed
// order, by the second kernel, so no atomics.  A tile of several requests
// runs once over its part of K for each, on the row blocks that hold the
// request alone; loads of P steps are in flight, also across requests.
template <class T, int MB, int RB, int P>
__global__ __launch_bounds__(256) void shrink_tiles_kernel(AdapterArgs a) {
  typedef typename Vec8Of<T>::V V8;
  constexpr int TM = 16 * MB, RP = 16 * RB;
  __shared__ float red[kWaves][TM][RP];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, r16 = lane & 15, lg = lane >> 4;
  const uint32_t m0 = blockIdx.x * TM;
  const int mine = my_request<TM>(a, m0, lane);
  const int k0 = (int)blockIdx.y * a.k_part + wave * (a.k_part / kWaves);
  const int k1 = min(a.K, k0 + a.k_part / kWaves);
  const int steps = k1 > k0 ? (k1 - k0 + 31) / 32 : 0;

  const T* xrow[MB];
#pragma unroll
  for (int mb = 0; mb < MB; ++mb) {
    const uint32_t m = m0 + mb * 16 + r16;
    xrow[mb] = (const T*)a.x + (long long)(m < a.M ? m : a.M - 1) * a.xs + lg * 8;
  }
  u32x4 xf[P][MB], wf[P][RB];
  f32x4 acc[MB][RB];
  auto clear = [&]() {
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
      for (int rb = 0; rb < RB; ++rb) acc[mb][rb] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  };
  auto holds = [&](unsigned long long rows, int mb) { return MB == 1 || ((rows >> (mb * 16)) & 0xffffull) != 0; };

  Requests ld, cp;  // the requests being loaded and multiplied
  ld.begin(mine);
  cp.begin(mine);
  int ls = 0, cs = 0;
  bool more = steps > 0 && ld.next(a, mine);
  if (more) cp.next(a, mine);
  bool left = more;
  auto load = [&](int p) {
    if (!more) return;
    const int k = k0 + ls * 32;
    const bool in = k + lg * 8 < k1;
    const u32x4 zero = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) {
      xf[p][mb] = zero;
      if (holds(ld.rows, mb) && in) xf[p][mb] = *(const u32x4*)(xrow[mb] + k);
    }
    const T* const w = (const T*)a.A + (long long)ld.id * a.R * a.K + k + lg * 8;
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
      const int r = rb * 16 + r16;
      wf[p][rb] = zero;
      if (r < ld.rank && in) wf[p][rb] = *(const u32x4*)(w + (long long)r * a.K);
    }
    if (++ls == steps) {
      ls = 0;
      more = ld.next(a, mine);
    }
  };
  auto multiply = [&](int p) {
    if (!left) return;
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
      if (holds(cp.rows, mb)) {
#pragma unroll
        for (int rb = 0; rb < RB; ++rb)
          acc[mb][rb] = mma(__builtin_bit_cast(V8, xf[p][mb]), __builtin_bit_cast(V8, wf[p][rb]), acc[mb][rb]);
      }
    if (++cs == steps) {
      cs = 0;
#pragma unroll
      for (int mb = 0; mb < MB; ++mb)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = mb * 16 + lg * 4 + i;
          if ((cp.rows >> row) & 1ull) {
#pragma unroll
            for (int rb = 0; rb < RB; ++rb) red[wave][row][rb * 16 + r16] = acc[mb][rb][i];
          }
        }
      clear();
      left = cp.next(a, mine);
    }
  };
  clear();
#pragma unroll
  for (int p = 0; p < P; ++p) load(p);
  while (left) {
#pragma unroll
    for (int p = 0; p < P; ++p) {
      multiply(p);
      load(p);
    }
  }
  __syncthreads();
  // waves without a step of their own wrote nothing
  const int part = a.k_part / kWaves;
  const int used = min(kWaves, (min(a.K, (int)blockIdx.y * a.k_part + a.k_part) - (int)blockIdx.y * a.k_part + part - 1) / part);
  for (int i = threadIdx.x; i < TM * RP; i += 256) {
    const int row = i / RP, r = i - row * RP;
    if (r >= a.R || m0 + row >= a.M) continue;
    float s = red[0][row][r];
    for (int w = 1; w < used; ++w) s += red[w][row][r];
    a.v[((long long)blockIdx.y * a.M + m0 + row) * a.R + r] = s;  // of rows without an adapter: never read
  }
}

// out = y + s B v for tiles of 16 MB rows and 256 J columns, on the matrix
// cores with the product transposed: rows of B are the A operand, straight
// from memory, and their order is chosen so that a lane ends up with 16
// neighbouring columns of one row, read and written in whole vectors.  v
// enters as a pair of 16-bit numbers (hi + lo, two products; for fp16 scaled
// by a power of two per row), so it keeps float32's range and 16 (bf16) or
// 21 (fp16) bits.  A tile's y is read once and held in float32 while its
// requests are added, each to its own rows.
template <class T, class YT, int MB, int KB, int VW, int P>
__global__ __launch_bounds__(256) void expand_tiles_kernel(AdapterArgs a) {
  typedef typename Vec8Of<T>::V V8;
  constexpr int TM = 16 * MB, RP = 32 * KB;
  constexpr int kRow = RP + 8;  // 16 bytes further per row: the operand reads spread over the banks
  __shared__ __align__(16) T vhi[TM][kRow], vlo[TM][kRow];
  __shared__ float up[TM];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, r16 = lane & 15, lg = lane >> 4;
  const uint32_t m0 = blockIdx.x * TM;
  const int mine = my_request<TM>(a, m0, lane);

  // v of the tile: the parts of K summed, the adapter's scale applied, split
  constexpr int kPer = RP / 8;  // threads on a row, within a wave
  for (int i = threadIdx.x; i < TM * kPer; i += 256) {
    const int row = i / kPer, r0 = (i - row * kPer) * 8;
    const uint32_t m = m0 + row;
    float f[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    const int id = m < a.M ? a.ids[m] : -1;
    const int rank = rank_of(a, id);
    if (r0 < rank) {
      const float* const v = a.v + (long long)m * a.R + r0;
#pragma unroll 4
      for (int s = 0; s < a.parts; ++s) {
        const f32x4* const q = (const f32x4*)(v + (long long)s * a.M * a.R);
        const f32x4 p0 = q[0], p1 = q[1];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          f[j] += p0[j];
          f[4 + j] += p1[j];
        }
      }
      const float s = a.scale ? a.scale[id] : 1.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = r0 + j < rank ? f[j] * s : 0.0f;
    }
    int e = 0;
    if (sizeof(T) == 2 && !__is_same(T, __bf16)) {
      float m8 = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) m8 = fmaxf(m8, fabsf(f[j]));
#pragma unroll
      for (int d = 1; d < kPer; d *= 2) m8 = fmaxf(m8, __shfl_xor(m8, d));
      e = m8 > 0.0f && m8 < __builtin_inff() ? __builtin_amdgcn_frexp_expf(m8) : 0;
    }
    Vec8<T> hi, lo;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float x = ldexpf(f[j], -e);
      hi.e[j] = (T)x;
      const float h = (float)hi.e[j];
      lo.e[j] = (T)(fabsf(h) < __builtin_inff() ? x - h : 0.0f);
    }
    *(Vec8<T>*)&vhi[row][r0] = hi;
    *(Vec8<T>*)&vlo[row][r0] = lo;
    if (r0 == 0) up[row] = ldexpf(1.0f, e);
  }
  __syncthreads();

  for (int j = 0; j < a.columns; ++j) {
    const int n0 = ((int)blockIdx.y * a.columns + j) * 256 + wave * 64;
    if (n0 >= a.N) return;
    const int nl = n0 + lg * 16;  // this lane's 16 columns
    float f[MB][16];
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) {
      const uint32_t m = m0 + mb * 16 + r16;
      const YT* const y = (const YT*)a.y + (long long)m * a.ys + nl;
#pragma unroll
      for (int c = 0; c < 16; c += VW) {
        struct alignas(VW * sizeof(YT)) {
          YT e[VW];
        } v;
        const bool in = m < a.M && nl + c < a.N;  // N a multiple of VW
        if (in) v = *(const decltype(v)*)(y + c);
#pragma unroll
        for (int i = 0; i < VW; ++i) f[mb][c + i] = in ? (float)v.e[i] : 0.0f;
      }
    }
    // B's rows: slot r16 of block nb is column 16 (r16 / 4) + 4 nb + r16 % 4
    u32x4 bf[P][4][KB];
    Requests ld, cp;
    ld.begin(mine);
    cp.begin(mine);
    bool more = ld.next(a, mine), left = cp.next(a, mine);
    auto load = [&](int p) {
      if (!more) return;
#pragma unroll
      for (int nb = 0; nb < 4; ++nb) {
        const int n = n0 + (r16 >> 2) * 16 + nb * 4 + (r16 & 3);
        const T* const w = (const T*)a.B + ((long long)ld.id * a.N + n) * a.R;
#pragma unroll
        for (int kk = 0; kk < KB; ++kk) {
          const int r = kk * 32 + lg * 8;
          u32x4 v = {0u, 0u, 0u, 0u};
          if (n < a.N && r < ld.rank) v = *(const u32x4*)(w + r);
          bf[p][nb][kk] = v;
        }
      }
      if (ld.rank & 7) {  // the last vector holds values past the adapter's rank
#pragma unroll
        for (int kk = 0; kk < KB; ++kk) {
          const int left_over = ld.rank - (kk * 32 + lg * 8);  // values of this lane's vector in use
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const uint32_t keep = left_over >= 2 * w + 2 ? 0xffffffffu : left_over == 2 * w + 1 ? 0xffffu : 0u;
#pragma unroll
            for (int nb = 0; nb < 4; ++nb) bf[p][nb][kk][w] &= keep;
          }
        }
      }
      more = ld.next(a, mine);
    };
    auto add = [&](int p) {
      if (!left) return;
#pragma unroll
      for (int mb = 0; mb < MB; ++mb) {
        const uint32_t rows = (uint32_t)(cp.rows >> (mb * 16)) & 0xffffu;
        if (MB > 1 && rows == 0) continue;
        f32x4 acc[4];
#pragma unroll
        for (int nb = 0; nb < 4; ++nb) acc[nb] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int kk = 0; kk < KB; ++kk) {
          const V8 hi = *(const V8*)&vhi[mb * 16 + r16][kk * 32 + lg * 8];
          const V8 lo = *(const V8*)&vlo[mb * 16 + r16][kk * 32 + lg * 8];
#pragma unroll
          for (int nb = 0; nb < 4; ++nb) {
            acc[nb] = mma(__builtin_bit_cast(V8, bf[p][nb][kk]), hi, acc[nb]);
            acc[nb] = mma(__builtin_bit_cast(V8, bf[p][nb][kk]), lo, acc[nb]);
          }
        }
        const bool own = (rows >> r16) & 1u;
        const float s = up[mb * 16 + r16];
#pragma unroll
        for (int c = 0; c < 16; ++c) f[mb][c] = own ? fmaf(acc[c >> 2][c & 3], s, f[mb][c]) : f[mb][c];
      }
      left = cp.next(a, mine);
    };
#pragma unroll
    for (int p = 0; p < P; ++p) load(p);
    while (left) {
#pragma unroll
      for (int p = 0; p < P; ++p) {
        add(p);
        load(p);
      }
    }
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) {
      const uint32_t m = m0 + mb * 16 + r16;
      YT* const out = (YT*)a.out + (long long)m * a.os + nl;
#pragma unroll
      for (int c = 0; c < 16; c += VW) {
        struct alignas(VW * sizeof(YT)) {
          YT e[VW];
        } v;
#pragma unroll
        for (int i = 0; i < VW; ++i) v.e[i] = (YT)f[mb][c + i];
        if (m < a.M && nl + c < a.N) *(decltype(v)*)(out + c) = v;
      }
    }
  }
}

// How a call is cut.  Few tokens: a wave per (token, rank) and a thread per
// (token, column).  More: tiles of 64 rows, or of 16 where 64 would leave
// compute units without work, and K in parts for the same reason.
struct Cut {
  bool tiles;
  int mb_shrink, mb_expand, parts, k_part, columns;
};

Cut cut_of(int64_t M, int64_t K, int64_t N, int64_t rank) {
  Cut cut, *const c = &cut;
  c->tiles = M > kRowsAtMost;
  c->parts = 1;
  c->k_part = (int)K;
  c->columns = 1;
  c->mb_shrink = c->mb_expand = 1;
  if (!c->tiles) return cut;
  const int big = rank > 64 ? 2 : 4;
  c->mb_shrink = (M + 16 * big - 1) / (16 * big) >= kUnits / 4 ? big : 1;
  const int64_t tiles = (M + 16 * c->mb_shrink - 1) / (16 * c->mb_shrink);
  int64_t parts = (4 * kUnits + tiles - 1) / tiles;
  const int64_t round = 32 * kWaves;  // a step of every wave
  if (parts > (K + 2 * round - 1) / (2 * round)) parts = (K + 2 * round - 1) / (2 * round);
  if (parts > kPartsAtMost) parts = kPartsAtMost;
  if (parts < 1) parts = 1;
  c->k_part = (int)(((K + parts - 1) / parts + round - 1) / round * round);
  c->parts = (int)((K + c->k_part - 1) / c->k_part);
  const int64_t across = (N + 255) / 256;
  c->mb_expand = ((M + 63) / 64) * across >= 4 * kUnits ? 4 : 1;
  const int64_t work = ((M + 16 * c->mb_expand - 1) / (16 * c->mb_expand)) * across;
  c->columns = work >= 16 * kUnits ? 4 : work >= 8 * kUnits ? 2 : 1;
  return cut;
}

template <class T>
hipError_t launch_shrink(const AdapterArgs& a, int mb, hipStream_t stream) {
  const dim3 grid((a.M + 16 * mb - 1) / (16 * mb), a.parts), block(256);
  const int rb = (a.R + 15) / 16;
  if (mb == 1) {
    if (rb == 1) shrink_tiles_kernel<T, 1, 1, 8><<<grid, block, 0, stream>>>(a);
    else if (rb == 2) shrink_tiles_kernel<T, 1, 2, 6><<<grid, block, 0, stream>>>(a);
    else if (rb <= 4) shrink_tiles_kernel<T, 1, 4, 4><<<grid, block, 0, stream>>>(a);
    else shrink_tiles_kernel<T, 1, 8, 2><<<grid, block, 0, stream>>>(a);
  } else {
    if (rb == 1) shrink_tiles_kernel<T, 4, 1, 4><<<grid, block, 0, stream>>>(a);
    else if (rb == 2) shrink_tiles_kernel<T, 4, 2, 3><<<grid, block, 0, stream>>>(a);
    else if (rb <= 4) shrink_tiles_kernel<T, 4, 4, 2><<<grid, block, 0, stream>>>(a);
    else shrink_tiles_kernel<T, 2, 8, 2><<<grid, block, 0, stream>>>(a);
  }
  return hipGetLastError();
}

template <class T, class YT, int VW>
hipError_t launch_expand(const AdapterArgs& a, int mb, hipStream_t stream) {
  const dim3 grid((a.M + 16 * mb - 1) / (16 * mb), (a.N + 256 * a.columns - 1) / (256 * a.columns)), block(256);
  const int kb = (a.R + 31) / 32;
  if (mb == 1) {
    if (kb == 1) expand_tiles_kernel<T, YT, 1, 1, VW, 4><<<grid, block, 0, stream>>>(a);
    else if (kb == 2) expand_tiles_kernel<T, YT, 1, 2, VW, 2><<<grid, block, 0, stream>>>(a);
    else expand_tiles_kernel<T, YT, 1, 4, VW, 1><<<grid, block, 0, stream>>>(a);
  } else {
    if (kb == 1) expand_tiles_kernel<T, YT, 4, 1, VW, 1><<<grid, block, 0, stream>>>(a);
    else if (kb == 2) expand_tiles_kernel<T, YT, 4, 2, VW, 1><<<grid, block, 0, stream>>>(a);
    else expand_tiles_kernel<T, YT, 4, 4, VW, 1><<<grid, block, 0, stream>>>(a);
  }
  return hipGetLastError();
}

template <class T, class YT>
hipError_t launch_y(AdapterArgs& a, const Cut& c, hipStream_t stream) {
  if (!c.tiles) {
    expand_rows_kernel<T, YT><<<dim3(a.M, (a.N + 255) / 256), dim3(256), 0, stream>>>(a);
    return hipGetLastError();
  }
  // y's and out's rows in vectors of eight, four or single elements
  const auto whole = [&](int w) {
    return a.N % w == 0 && a.ys % w == 0 && a.os % w == 0 && aligned_to(a.y, w * (int)sizeof(YT) > 16 ? 16 : w * (int)sizeof(YT)) &&
           aligned_to(a.out, w * (int)sizeof(YT) > 16 ? 16 : w * (int)sizeof(YT));
  };
  constexpr int kWide = 16 / sizeof(YT);  // elements of 16 bytes
  if (whole(kWide)) return launch_expand<T, YT, kWide>(a, c.mb_expand, stream);
  if (kWide > 4 && whole(4)) return launch_expand<T, YT, 4>(a, c.mb_expand, stream);
  return launch_expand<T, YT, 1>(a, c.mb_expand, stream);
}

template <class T>
hipError_t launch(AdapterArgs& a, const Cut& c, int y_dtype, hipStream_t stream) {
  hipError_t e;
  if (c.tiles) {
    e = launch_shrink<T>(a, c.mb_shrink, stream);
  } else {
    shrink_rows_kernel<T><<<dim3(a.M, (a.R + 3) / 4), dim3(256), 0, stream>>>(a);
    e = hipGetLastError();
  }
  if (e != hipSuccess) return e;
  switch (y_dtype) {
    case ORBIT_BF16: return launch_y<T, __bf16>(a, c, stream);
    case ORBIT_F16: return launch_y<T, _Float16>(a, c, stream);
    default: return launch_y<T, float>(a, c, stream);
  }
}

bool sizes_ok(int64_t M, int64_t K, int64_t rank) {
  return M >= 0 && M < ORBIT_MAX_ROWS && K >= 8 && K <= 65536 && K % 8 == 0 && rank >= 8 && rank <= 128 && rank % 8 == 0;
}

}  // namespace

extern "C" int64_t orbit_adapter_workspace(int64_t M, int64_t K, int64_t rank) {
  if (!sizes_ok(M, K, rank)) return -1;
  return M * rank * 4 * cut_of(M, K, 1, rank).parts;
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
  const Cut c = cut_of(p->M, p->K, p->N, p->rank);
  a.parts = c.parts;
  a.k_part = c.k_part;
  a.columns = c.columns;
  return hip_status(p->x_dtype == ORBIT_BF16 ? launch<__bf16>(a, c, p->y_dtype, stream) : launch<_Float16>(a, c, p->y_dtype, stream));
}
