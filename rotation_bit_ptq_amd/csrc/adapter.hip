// orbit_adapter_add: low-rank adapters of many requests beside a shared
// projection, out[m] = y[m] + s_a B_a (A_a x[m]), a = ids[m].
//
// Bound: memory (x, y and out once; the adapters in use once, then from L2).
// Two products: v = A x into the workspace, then out = y + s B v; v stays in
// float32.  16384 tokens of 8 adapters, rank 64, 4096 -> 4096: 118 us (3.5
// TB/s), 48 + 70; 1003 tokens of 48 adapters, rank 32 and less, 3072 ->
// 12288, float32 y: 66 us; 64 tokens of 64 adapters, rank 16: 8.2 to 9.0 us,
// twice the latency of a launch and of the chain id -> rank -> rows.
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
  int slices;  // of a tile's rows, see shrink_staged_kernel
  int columns, blocks;  // 256 columns a piece per workgroup; workgroups across N
};

constexpr int kWaves = 4;
// Adapters of a tile, past which its rows go one by one.  The whole call:
//   16 rows (1003 tokens, 3072 -> 12288, rank 32): six adapters a tile 58 us as
//     a tile and 79 by rows, eight 64 and 73, sixteen 75 by rows;
//   64 rows (4096 tokens, 4096 -> 4096, rank 64): nine 107 as a tile and 277 by
//     rows, 24 193 and 282, 48 304 and 290; 16384 tokens: 24 640 and 1231, 64
//     1312 and 1356; rank 16, 4096 tokens: 16 97 and 121, 32 139 and 123;
//     nearly the first product alone (1100 tokens, 4096 -> 64): rank 64, 24 87
//     and 148; rank 16, 16 42 and 47, 24 54 and 46.
constexpr int requests_at_most(int rows) { return rows == 64 ? 24 : 8; }
constexpr int kFewTokens = 256, kSomeTokens = 1024;  // see cut_of

// The adapter's rank, 0 where there is none.
__device__ __forceinline__ int rank_of(const AdapterArgs& a, int id) {
  if ((uint32_t)id >= a.adapters) return 0;
  const int r = a.ranks ? a.ranks[id] : a.R;
  return r < 0 ? 0 : r < a.R ? r : a.R;
}

// Eight products and their sum.  bf16: v_dot2_f32_bf16 (exact products);
// fp16: mixed-precision multiply-adds, which keep fp16's subnormal numbers.
__device__ __forceinline__ float dot8(const u32x4& x, const u32x4& w, float s, __bf16) {
  typedef __bf16 b2 __attribute__((ext_vector_type(2)));
  struct B4 {
    b2 e[4];
  };
  const B4 p = __builtin_bit_cast(B4, x), q = __builtin_bit_cast(B4, w);
#pragma unroll
  for (int j = 0; j < 4; ++j) s = __builtin_amdgcn_fdot2_f32_bf16(p.e[j], q.e[j], s, false);
  return s;
}
__device__ __forceinline__ float dot8(const u32x4& x, const u32x4& w, float s, _Float16) {
  const f16x8 p = __builtin_bit_cast(f16x8, x), q = __builtin_bit_cast(f16x8, w);
#pragma unroll
  for (int j = 0; j < 8; ++j) s = fmaf((float)p[j], (float)q[j], s);
  return s;
}

// Sums of four values over the wave at once: row i of 16 lanes ends up with
// the sum of s[i] (each exchange merges two values' halves).
__device__ __forceinline__ float sum_of_four(const float (&s)[4]) {
  auto merge32 = [](float x, float y) {
    const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(unsigned, x), __builtin_bit_cast(unsigned, y), false, false);
    return __builtin_bit_cast(float, (unsigned)r[0]) + __builtin_bit_cast(float, (unsigned)r[1]);
  };
  const float u = merge32(s[0], s[2]), w = merge32(s[1], s[3]);
  const auto r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(unsigned, u), __builtin_bit_cast(unsigned, w), false, false);
  float v = __builtin_bit_cast(float, (unsigned)r[0]) + __builtin_bit_cast(float, (unsigned)r[1]);
  v = dpp_add<kXor1>(v);
  v = dpp_add<kXor2>(v);
  v = dpp_add<kHalfMirror>(v);
  return dpp_add<kRowMirror>(v);
}

// v[m][r] = A[id][r] . x[m] over k0 <= k < k1 for RG rows and RW ranks (1, 4
// or 8) from r0, by one wave without matrix cores: the lanes take
// neighbouring vectors of K, so that every load is one contiguous KB.  A is
// read once for the rows that share an adapter.
template <class T, int RG, int RW>
__device__ __forceinline__ void row_products(const AdapterArgs& a, uint32_t m0, int r0, int k0, int k1, float* v) {
  const int lane = threadIdx.x & 63;
  int id[RG];
  const T* x[RG];
#pragma unroll
  for (int g = 0; g < RG; ++g) {
    const uint32_t m = min(m0 + g, a.M - 1);
    id[g] = m0 + g < a.M ? a.ids[m] : -1;
    x[g] = (const T*)a.x + (long long)m * a.xs + lane * 8;
  }
#pragma unroll
  for (int g = 0; g < RG; ++g) {
    bool seen = false;  // with an earlier row
#pragma unroll
    for (int h = 0; h < g; ++h) seen = seen || id[h] == id[g];
    const int rank = seen ? 0 : rank_of(a, id[g]);
    if (r0 >= rank) continue;
    const T* w[RW];
#pragma unroll
    for (int i = 0; i < RW; ++i)
      w[i] = (const T*)a.A + ((long long)id[g] * a.R + min(r0 + i, rank - 1)) * a.K + lane * 8;
    float s[RG][RW];
#pragma unroll
    for (int h = 0; h < RG; ++h)
#pragma unroll
      for (int i = 0; i < RW; ++i) s[h][i] = 0.0f;
    int k = k0;
    auto step = [&]() {
      u32x4 xv[RG], wv[RW];
#pragma unroll
      for (int h = 0; h < RG; ++h) xv[h] = *(const u32x4*)(x[h] + k);
#pragma unroll
      for (int i = 0; i < RW; ++i) wv[i] = *(const u32x4*)(w[i] + k);
#pragma unroll
      for (int h = 0; h < RG; ++h)
#pragma unroll
        for (int i = 0; i < RW; ++i) s[h][i] = dot8(xv[h], wv[i], s[h][i], T());
    };
    constexpr int kAtOnce = RG * RW == 1 ? 8 : 2;
    for (; k + 512 * kAtOnce <= k1;) {
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u, k += 512) step();
    }
    for (; k + 512 <= k1; k += 512) step();
    if (k + lane * 8 < k1) step();
#pragma unroll
    for (int h = g; h < RG; ++h) {
      float* const to = v + (long long)(m0 + h) * a.R + r0;
      const bool own = id[h] == id[g];
      if constexpr (RW >= 4) {
#pragma unroll
        for (int i = 0; i < RW; i += 4) {
          const float four[4] = {s[h][i], s[h][i + 1], s[h][i + 2], s[h][i + 3]};
          const float t = sum_of_four(four);
          if (own && (lane & 15) == 0 && r0 + i + (lane >> 4) < rank) to[i + (lane >> 4)] = t;
        }
      } else {
        const float t = wave_sum(s[h][0]);
        if (own && lane == 0) *to = t;
      }
    }
  }
}

// One row and four ranks per workgroup, one rank per wave.
template <class T>
__global__ __launch_bounds__(256) void shrink_rows_kernel(AdapterArgs a) {
  const int r0 = (int)blockIdx.y * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  row_products<T, 1, 1>(a, blockIdx.x, r0, 0, a.K, a.v);
}

// out[m][n] = y[m][n] + s B[id][n] . v[m]: a wave per row and 64 columns.  B's
// block is read in the order of memory, all of it in flight at once; a lane's
// eight ranks are summed over the lanes of a row of B.
template <class T, class YT, int KB>
__global__ __launch_bounds__(256) void expand_rows_kernel(AdapterArgs a) {
  typedef typename Vec8Of<T>::V V8;
  constexpr int kLanes = 4 * KB, kAcross = 64 / kLanes;  // lanes on a row of B, rows at once
  __shared__ float sums[kWaves][64];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const long long m = blockIdx.x;
  const int n0 = (int)blockIdx.y * 256 + wave * 64, n = n0 + lane;
  if (n0 >= a.N) return;
  const float y = (float)((const YT*)a.y)[m * a.ys + min(n, a.N - 1)];
  const int id = a.ids[m];
  float d = 0.0f;
  if ((uint32_t)id < a.adapters) {
    const int brow = lane / kLanes, bcol = lane % kLanes, r0 = bcol * 8 < a.R ? bcol * 8 : 0;
    const T* const b = (const T*)a.B + (long long)id * a.N * a.R + r0;
    u32x4 w[kLanes];
#pragma unroll
    for (int c = 0; c < kLanes; ++c) w[c] = *(const u32x4*)(b + (long long)min(n0 + c * kAcross + brow, a.N - 1) * a.R);
    const f32x4 v0 = *(const f32x4*)(a.v + m * a.R + r0), v1 = *(const f32x4*)(a.v + m * a.R + r0 + 4);
    const int used = rank_of(a, id) - bcol * 8;  // of this lane's eight ranks; what v holds past them is anything
    float own = 0.0f;
#pragma unroll
    for (int c = 0; c < kLanes; ++c) {
      const V8 q = __builtin_bit_cast(V8, w[c]);
      float s = 0.0f;
#pragma unroll
      for (int k = 0; k < 8; ++k) s = k < used ? fmaf((float)q[k], k < 4 ? v0[k & 3] : v1[k & 3], s) : s;
      s = dpp_add<kXor1>(s);
      s = dpp_add<kXor2>(s);
      if (KB >= 2) s = dpp_add<kHalfMirror>(s);
      if (KB >= 4) s = dpp_add<kRowMirror>(s);
      if (bcol == c) own = s;  // the sum is in all lanes of the row: lane c keeps the c-th
    }
    sums[wave][bcol * kAcross + brow] = own;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    d = sums[wave][lane] * (a.scale ? a.scale[id] : 1.0f);
  }
  // no adapter, or one of rank 0: y as it is, whatever the scale
  if (n < a.N) ((YT*)a.out)[m * a.os + n] = (YT)(rank_of(a, id) > 0 ? y + d : y);
}

// One row's request: its adapter (-1: none, or one of rank 0), rank, scale.
struct Request {
  int id, rank;
  float scale;
};

// Lane l's adapter: that of row m0 + l of a tile of TM <= 64 rows, -1: none.
template <int TM>
__device__ __forceinline__ int id_of(const AdapterArgs& a, uint32_t m0, int lane) {
  const int id = a.ids[min(m0 + lane, a.M - 1)];
  return lane < TM && m0 + lane < a.M && (uint32_t)id < a.adapters ? id : -1;
}
// And its request.  Rank and scale are loaded whatever the row, so that they
// wait for the id alone.
__device__ __forceinline__ Request request_of(const AdapterArgs& a, int id) {
  Request q = {id, a.R, 1.0f};
  if (a.adapters == 0) return q;
  if (a.ranks) q.rank = min(max(a.ranks[max(id, 0)], 0), a.R);
  if (a.scale) q.scale = a.scale[max(id, 0)];
  if (q.rank == 0) q.id = -1;
  if (q.id < 0) q.rank = 0, q.scale = 1.0f;
  return q;
}

// Whether a tile of TM rows, one per lane, has more adapters than it takes.
template <int TM>
__device__ __forceinline__ bool many_requests(int id) {
  unsigned long long rest = __ballot(id >= 0);
  for (int n = 0; rest != 0; ++n) {
    if (n == requests_at_most(TM)) return true;
    rest &= ~__ballot(id == __builtin_amdgcn_readlane(id, __builtin_ctzll(rest)));
  }
  return false;
}

// The distinct adapters of a tile, one after the other.  Everything about
// them is in the lanes' registers: a load here would wait for the operands'
// loads that are in flight.
struct Requests {
  unsigned long long rest, rows;  // rows still to come; rows of `id`
  int id, rank;

  __device__ __forceinline__ void begin(const Request& mine) { rest = __ballot(mine.id >= 0); }
  __device__ __forceinline__ bool next(const Request& mine) {
    if (rest == 0) return false;
    const int first = __builtin_ctzll(rest);
    id = __builtin_amdgcn_readlane(mine.id, first);
    rank = __builtin_amdgcn_readlane(mine.rank, first);
    rows = __ballot(mine.id == id);
    rest &= ~rows;
    return true;
  }
};

// Four rows and 16 ranks at a time.  Rows of one adapter: a wave takes four
// ranks of all, so A is read once for them.  Else a wave takes a row (1003
// tokens of 48 adapters, K 3072, rank 32 and less: 10 us; with all four rows
// per wave in turn 19).
template <class T>
__device__ __forceinline__ void four_rows(const AdapterArgs& a, uint32_t m0, int r0) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int id = a.ids[min(m0 + (threadIdx.x & 3), a.M - 1)];
  if (__ballot(id != __builtin_amdgcn_readfirstlane(id)) == 0) {
    row_products<T, 4, 4>(a, m0, r0 + wave * 4, 0, a.K, a.v);
  } else if (m0 + wave < a.M) {
    row_products<T, 1, 8>(a, m0 + wave, r0, 0, a.K, a.v);
    row_products<T, 1, 8>(a, m0 + wave, r0 + 8, 0, a.K, a.v);
  }
}

template <class T>
__global__ __launch_bounds__(256) void shrink_fours_kernel(AdapterArgs a) {
  four_rows<T>(a, blockIdx.x * 4, (int)blockIdx.y * 16);
}

// v = A x for many tokens, on the matrix cores: tiles of 64 rows, a part of K
// in chunks of 128.  blockIdx.y takes a part of K; the parts are summed, in a
// fixed order, by the second kernel, so no atomics.  The first a.slices of
// blockIdx.y share the rows of a tile of many requests instead (their whole
// sums go to the first part, zeros to the others) and mostly leave at once.
// A chunk of x and of the request's A go through LDS: sixteen lanes read 256
// contiguous bytes of a row (a matrix operand read from memory directly has
// its neighbouring lanes in 16 different rows, which costs the address unit
// four times the cycles), and the operands come back as 16-byte reads; the
// 16-byte places of a row are exchanged by its number (place ^ row mod 16),
// which spreads both over the banks.  The
// next chunk's loads are in flight, in registers, while one is multiplied.
// Wave w takes rows 16 w .. 16 w + 15 and all ranks, so sums stay in one
// wave.  In a tile of several requests (at the border of two prompts) a chunk
// of x is multiplied by each one's A before the next comes, and only its own
// rows keep the sums (zeros for the others' x would not do: an infinite
// weight would reach them).  So x is read once and such a workgroup, of which
// some compute units get several, ends soon after the others (16384 x 4096, rank 64, prompts of 1024 that end
// inside a tile: 47 us; as a second pass over x 56; none ends inside: 41).
template <class T, int RB>
__global__ __launch_bounds__(256, RB <= 4 ? 4 : 3) void shrink_staged_kernel(AdapterArgs a) {
  typedef typename Vec8Of<T>::V V8;
  constexpr int TM = 64, KC = 128;
  __shared__ __align__(16) T xs[TM][KC], ws[16 * RB][KC];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63, r16 = lane & 15, lg = lane >> 4;
  const int trow = threadIdx.x >> 4, tcol = (threadIdx.x & 15) * 8;  // this thread's place in 16 rows of a chunk
  const int tplace = ((threadIdx.x & 15) ^ trow) * 8;  // and in LDS
  const uint32_t m0 = blockIdx.x * TM;
  const int id = id_of<TM>(a, m0, lane);
  const bool many = many_requests<TM>(id);
  if ((int)blockIdx.y < a.slices) {
    if (!many) return;
    const uint32_t rows = TM / a.slices, from = m0 + blockIdx.y * rows, to = min(from + rows, a.M);
    for (uint32_t m = from; m < to; m += 4)
      for (int r0 = 0; r0 < a.R; r0 += 16) four_rows<T>(a, m, r0);
    for (int p = 1; p < a.parts; ++p)
      for (long long i = (long long)from * a.R + threadIdx.x; i < (long long)to * a.R; i += 256)
        a.v[(long long)p * a.M * a.R + i] = 0.0f;
    return;
  }
  if (many) return;
  const Request mine = request_of(a, id);
  const int part = (int)blockIdx.y - a.slices, first_k = part * a.k_part, k1 = min(a.K, first_k + a.k_part);
  float* const v = a.v + (long long)part * a.M * a.R;
  const T* xrow[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t m = m0 + i * 16 + trow;
    xrow[i] = (const T*)a.x + (long long)(m < a.M ? m : a.M - 1) * a.xs;
  }
  u32x4 xr[4];
  // past the end: what was read before
  auto load_x = [&](int k) {
    const int at = k + tcol < k1 ? k + tcol : first_k;
#pragma unroll
    for (int i = 0; i < 4; ++i) xr[i] = *(const u32x4*)(xrow[i] + at);
  };
  Requests ld, cp;
  ld.begin(mine);
  if (!ld.next(mine)) return;  // the same for the whole workgroup
  int lk = first_k;  // the chunk of A whose loads go out next, for request `ld`
  u32x4 wr[RB];
  auto load_w = [&]() {
    const T* const w = (const T*)a.A + (long long)ld.id * a.R * a.K + (lk + tcol < k1 ? lk + tcol : first_k);
#pragma unroll
    for (int i = 0; i < RB; ++i) wr[i] = *(const u32x4*)(w + (long long)min(i * 16 + trow, ld.rank - 1) * a.K);
    if (!ld.next(mine)) {
      ld.begin(mine);
      ld.next(mine);
      lk += KC;
    }
  };
  load_x(first_k);
  load_w();
  f32x4 acc[RB];
#pragma unroll
  for (int i = 0; i < RB; ++i) acc[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  for (int ck = first_k; ck < k1; ck += KC) {
    const bool in = ck + tcol < k1;
    const u32x4 zero = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < 4; ++i) *(u32x4*)&xs[i * 16 + trow][tplace] = in ? xr[i] : zero;
    cp.begin(mine);
    bool more = cp.next(mine), first = true;
    do {
#pragma unroll
      for (int i = 0; i < RB; ++i) *(u32x4*)&ws[i * 16 + trow][tplace] = in ? wr[i] : zero;
      __syncthreads();
      load_w();
      if (first) load_x(ck + KC);
      first = false;
      f32x4 sum[RB];
#pragma unroll
      for (int i = 0; i < RB; ++i) sum[i] = acc[i];
#pragma unroll
      for (int k = 0; k < KC; k += 32) {
        const int place = ((k / 8 + lg) ^ r16) * 8;
        const V8 x = *(const V8*)&xs[wave * 16 + r16][place];
#pragma unroll
        for (int i = 0; i < RB; ++i) sum[i] = mma(x, *(const V8*)&ws[i * 16 + r16][place], sum[i]);
      }
      const uint32_t own = (uint32_t)(cp.rows >> (wave * 16 + lg * 4));
#pragma unroll
      for (int i = 0; i < RB; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = (own >> j) & 1u ? sum[i][j] : acc[i][j];
      more = cp.next(mine);
      __syncthreads();
    } while (more);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t m = m0 + wave * 16 + lg * 4 + j;
    if (m >= a.M) continue;
#pragma unroll
    for (int i = 0; i < RB; ++i)
      if (i * 16 + r16 < a.R) v[(long long)m * a.R + i * 16 + r16] = acc[i][j];
  }
}

// Which tile of rows and which block of columns a workgroup of the second
// kernel takes.  Workgroups go round the eight XCDs, each with an L2 of its
// own: with eight blocks of columns or more, an XCD keeps to every eighth
// block for all tiles, so that the adapters' blocks of B stay in its L2.
struct Place {
  uint32_t tile;
  int block;
};
__device__ __forceinline__ Place place_of(const AdapterArgs& a, uint32_t tiles) {
  const uint32_t i = blockIdx.x;
  Place p;
  if (a.blocks >= 8) {
    p.tile = (i >> 3) % tiles;
    p.block = (int)((i >> 3) / tiles * 8 + (i & 7));
  } else {
    p.tile = i % tiles;
    p.block = (int)(i / tiles);
  }
  return p;
}

// Eight of a row's v from r0: the parts of K summed, the adapter's scale
// applied, zeros past its rank.  Loaded whether used or not (rows without an
// adapter hold anything), so that the loads need not wait for the request.
__device__ __forceinline__ void load_v(const AdapterArgs& a, uint32_t m, int r0, int rank, float scale, float (&f)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] = 0.0f;
  const float* const v = a.v + (long long)min(m, a.M - 1) * a.R + (r0 < a.R ? r0 : 0);
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
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] = r0 + j < rank ? f[j] * scale : 0.0f;
}

// A vector of VW elements of y and out.
template <class YT, int VW>
struct alignas(VW * sizeof(YT)) Vector {
  YT e[VW];
};

// The same for tiles of more than requests_at_most() requests (single tokens):
// the tile's rows, 16 at a time, and 256 J columns, without matrix cores.
// A row's block of B is read in the order of memory, KB * 4 KB at a time; a
// lane's eight ranks are summed over the lanes of a row of B.
template <class T, class YT, int TM, int KB, int VW>
__global__ __launch_bounds__(256) void expand_singles_kernel(AdapterArgs a) {
  typedef typename Vec8Of<T>::V V8;
  constexpr int RP = 32 * KB, kLanes = RP / 8, kAcross = 64 / kLanes;  // lanes on a row of B, rows at once
  __shared__ __align__(16) float vf[16][RP + 4];
  __shared__ __align__(16) float turns[kWaves][16][68];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const Place place = place_of(a, (a.M + TM - 1) / TM);
  if (place.block >= a.blocks) return;
  const uint32_t m0 = place.tile * TM;
  const int id = id_of<TM>(a, m0, lane);
  if (!many_requests<TM>(id)) return;  // expand_tiles_kernel's
  const Request mine = request_of(a, id);
  float(*const turn)[68] = turns[wave];
  const int brow = lane / kLanes, bcol = lane % kLanes, brank = bcol * 8;
  const int prow = lane / (64 / VW), pcol = (lane % (64 / VW)) * VW;
  constexpr int kAtOnce = KB == 1 ? 4 : 2;  // rows whose loads are in flight together
  for (int sub = 0; sub < TM && m0 + sub < a.M; sub += 16) {
    for (int i = threadIdx.x; i < 16 * kLanes; i += 256) {
      const int row = i / kLanes, r0 = (i - row * kLanes) * 8;
      float f[8];
      load_v(a, m0 + sub + row, r0, __shfl(mine.rank, sub + row), __shfl(mine.scale, sub + row), f);
      *(f32x4*)&vf[row][r0] = f32x4{f[0], f[1], f[2], f[3]};
      *(f32x4*)&vf[row][r0 + 4] = f32x4{f[4], f[5], f[6], f[7]};
    }
    __syncthreads();
    for (int j = 0; j < a.columns; ++j) {
      const int n0 = (place.block * a.columns + j) * 256 + wave * 64;
      if (n0 >= a.N) break;
      u32x4 w[kAtOnce][4 * KB];
      auto load_b = [&](int u, int row) {
        const int id = max(__builtin_amdgcn_readlane(mine.id, sub + row), 0);  // none: of rank 0, any will do
        const int rank = __builtin_amdgcn_readlane(mine.rank, sub + row);
        const T* const at = (const T*)a.B + (long long)id * a.N * a.R + (brank < rank ? brank : 0);
#pragma unroll
        for (int c = 0; c < 4 * KB; ++c) w[u][c] = *(const u32x4*)(at + (long long)min(n0 + c * kAcross + brow, a.N - 1) * a.R);
      };
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) load_b(u, u);
      Vector<YT, VW> y[16 / VW];  // N is a multiple of VW; past the end the last one
#pragma unroll
      for (int i = 0; i < 16 / VW; ++i)
        y[i] = *(const Vector<YT, VW>*)((const YT*)a.y + (long long)min(m0 + sub + i * VW + prow, a.M - 1) * a.ys + min(n0 + pcol, a.N - VW));
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int u = i % kAtOnce;
        const int used = __builtin_amdgcn_readlane(mine.rank, sub + i) - brank;  // of this lane's eight ranks
        const f32x4 v0 = *(const f32x4*)&vf[i][brank], v1 = *(const f32x4*)&vf[i][brank + 4];
        float own = 0.0f;
#pragma unroll
        for (int c = 0; c < 4 * KB; ++c) {
          const V8 b = __builtin_bit_cast(V8, w[u][c]);
          float s = 0.0f;
#pragma unroll
          for (int q = 0; q < 8; ++q) s = fmaf(q < used ? (float)b[q] : 0.0f, q < 4 ? v0[q & 3] : v1[q & 3], s);
          s = dpp_add<kXor1>(s);
          s = dpp_add<kXor2>(s);
          if (KB >= 2) s = dpp_add<kHalfMirror>(s);
          if (KB >= 4) s = dpp_add<kRowMirror>(s);
          if (bcol == c) own = s;  // the sum is in all lanes of the row: lane c keeps the c-th
        }
        turn[i][bcol * kAcross + brow] = own;
        if (i + kAtOnce < 16) load_b(u, i + kAtOnce);
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int i = 0; i < 16 / VW; ++i) {
        const uint32_t m = m0 + sub + i * VW + prow;
        if (m >= a.M || n0 + pcol >= a.N) continue;
        Vector<YT, VW> o;
#pragma unroll
        for (int c = 0; c < VW; ++c) o.e[c] = (YT)((float)y[i].e[c] + turn[i * VW + prow][pcol + c]);
        *(Vector<YT, VW>*)((YT*)a.out + (long long)m * a.os + n0 + pcol) = o;
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
    }
    __syncthreads();
  }
}

// out = y + s B v for tiles of 16 MB rows and 256 J columns, on the matrix
// cores with the product transposed (rows of B are the A operand), so that a
// lane's four results are neighbouring columns.  v enters as kTerms 16-bit
// numbers, a product each: fp16 (scaled by a power of two per row, which keeps
// float32's range) as two, 22 bits; bf16 as three, all 24 bits, where y is
// float32, and as two, 16 bits, where out is rounded to 8 or 11 bits anyway.
// Split terms have no product with an infinite weight (one may be zero or of
// the other sign), nor have the zeros past an adapter's rank, so products that
// came out NaN are summed again in float32, outside the matrix cores.
// (bf16 to float32, the third term: 16384 tokens, 4096 -> 4096, rank 64, 194 ->
// 196 us; 8192 tokens, 2048 -> 4096, rank 128, 120 -> 124.)
// The products of a tile's requests are kept in float32, each in its own
// rows, and leave through the wave's LDS rows, 16 at a time, in the order in
// which y is read and out written: neighbouring lanes on neighbouring
// vectors of VW columns (in the products' own order neighbouring lanes would
// be in 16 different rows, which takes the address unit four times longer).
// (Two workgroups per compute unit where 256 registers hold all of it: the sum
// in float32 would take a few more for 16-bit y in vectors of four.)
template <class T, class YT, int MB, int KB, int VW, int P>
__global__ __launch_bounds__(256, sizeof(YT) == 2 && KB <= 2 ? 2 : 1) void expand_tiles_kernel(AdapterArgs a) {
  typedef typename Vec8Of<T>::V V8;
  constexpr int TM = 16 * MB, RP = 32 * KB;
  typedef Vector<YT, VW> Part;
  constexpr int kRow = RP + 8;  // 16 bytes further per row: the operand reads spread over the banks
  constexpr int kPasses = 16 / VW;  // of VW rows each over 16 rows, 64 / VW lanes on a row
  constexpr int kTerms = __is_same(T, __bf16) && sizeof(YT) == 4 ? 3 : 2;
  __shared__ __align__(16) T vterms[kTerms][TM][kRow];
  __shared__ float up[TM];
  // B's block of a request and the products' way out share the wave's rows
  constexpr bool kStaged = KB <= 2;
  constexpr int kTurn = 16 * 68 * 4, kStage = kStaged ? 64 * kRow * 2 : 0;
  __shared__ __align__(16) char wave_rows[kWaves][kTurn > kStage ? kTurn : kStage];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63, r16 = lane & 15, lg = lane >> 4;
  float(*const turn)[68] = (float(*)[68])wave_rows[wave];
  T(*const stage)[kRow] = (T(*)[kRow])wave_rows[wave];
  constexpr int kLanes = RP / 8, kAcross = 64 / kLanes;  // lanes on a row of B, rows at once
  const int brow = lane / kLanes, brank = (lane % kLanes) * 8;
  const int prow = lane / (64 / VW), pcol = (lane % (64 / VW)) * VW;
  const Place place = place_of(a, (a.M + TM - 1) / TM);
  if (place.block >= a.blocks) return;
  const uint32_t m0 = place.tile * TM;
  const int id = id_of<TM>(a, m0, lane);
  if (many_requests<TM>(id)) return;  // expand_singles_kernel's
  const Request mine = request_of(a, id);

  // v of the tile: the parts of K summed, the adapter's scale applied, split
  constexpr int kPer = RP / 8;  // threads on a row, within a wave
  for (int i = threadIdx.x; i < TM * kPer; i += 256) {
    const int row = i / kPer, r0 = (i - row * kPer) * 8;
    const uint32_t m = m0 + row;
    float f[8];
    load_v(a, m, r0, __shfl(mine.rank, row), __shfl(mine.scale, row), f);
    int e = 0;
    if (!__is_same(T, __bf16)) {
      float m8 = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) m8 = fmaxf(m8, fabsf(f[j]));
#pragma unroll
      for (int d = 1; d < kPer; d *= 2) m8 = fmaxf(m8, __shfl_xor(m8, d));
      e = m8 > 0.0f && m8 < __builtin_inff() ? min(__builtin_amdgcn_frexp_expf(m8), 127) : 0;  // 2^127 is the last power
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = ldexpf(f[j], -e);
#pragma unroll
    for (int t = 0; t < kTerms; ++t) {
      Vec8<T> term;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        term.e[j] = (T)f[j];
        const float h = (float)term.e[j];
        f[j] = fabsf(h) < __builtin_inff() ? f[j] - h : 0.0f;
      }
      *(Vec8<T>*)&vterms[t][row][r0] = term;
    }
    if (r0 == 0) up[row] = ldexpf(1.0f, e);
  }
  __syncthreads();

  auto order = [] {  // between writes and reads of the wave's rows by other lanes
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  };
  for (int j = 0; j < a.columns; ++j) {
    const int n0 = (place.block * a.columns + j) * 256 + wave * 64;
    if (n0 >= a.N) return;
    // past the last row or column (N is a multiple of VW) the last one is
    // read again, so that no load is conditional and none waits for another
    auto load_y = [&](int mb, Part (&y)[kPasses]) {
#pragma unroll
      for (int i = 0; i < kPasses; ++i) {
        const uint32_t m = min(m0 + mb * 16 + i * VW + prow, a.M - 1);
        y[i] = *(const Part*)((const YT*)a.y + (long long)m * a.ys + min(n0 + pcol, a.N - VW));
      }
    };
    // the products of 16 rows lie in `turn`, some of them NaN
    auto sum_again = [&](int mb) {
      order();
#pragma unroll 1
      for (int row = 0; row < 16; ++row) {
        const int id = __builtin_amdgcn_readlane(mine.id, mb * 16 + row), rank = __builtin_amdgcn_readlane(mine.rank, mb * 16 + row);
        if (id < 0 || turn[row][lane] == turn[row][lane]) continue;
        const T* const b = (const T*)a.B + ((long long)id * a.N + min(n0 + lane, a.N - 1)) * a.R;
        float s = 0.0f;
#pragma unroll 1
        for (int r = 0; r < rank; ++r) {
          float v = 0.0f;
#pragma unroll
          for (int t = 0; t < kTerms; ++t) v += (float)vterms[t][mb * 16 + row][r];
          s = fmaf((float)b[r], v * up[mb * 16 + row], s);
        }
        turn[row][lane] = s;
      }
    };
    auto finish = [&](int mb, const Part (&y)[kPasses]) {  // the products of 16 rows lie in `turn`
      order();
#pragma unroll
      for (int i = 0; i < kPasses; ++i) {
        const uint32_t m = m0 + mb * 16 + i * VW + prow;
        float d[VW];
        if constexpr (VW >= 4) {
#pragma unroll
          for (int c = 0; c < VW; c += 4) *(f32x4*)(d + c) = *(const f32x4*)&turn[i * VW + prow][pcol + c];
        } else {
          d[0] = turn[i * VW + prow][pcol];
        }
        Part o;
#pragma unroll
        for (int c = 0; c < VW; ++c) o.e[c] = (YT)((float)y[i].e[c] + d[c]);
        if (m < a.M && n0 + pcol < a.N) *(Part*)((YT*)a.out + (long long)m * a.os + n0 + pcol) = o;
      }
      order();
    };
    Part yv[MB][kPasses];
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) load_y(mb, yv[mb]);
    u32x4 bf[P][4][KB];
    Requests ld, cp;
    ld.begin(mine);
    cp.begin(mine);
    bool more = ld.next(mine), left = cp.next(mine);
    auto load = [&](int p) {
      if (!more) return;
      // past the rank v is zero: any vector of the adapter's will do
      const T* const w = (const T*)a.B + (long long)ld.id * a.N * a.R;
#pragma unroll
      for (int nb = 0; nb < 4; ++nb)
#pragma unroll
        for (int kk = 0; kk < KB; ++kk) {
          const int n = kStaged ? n0 + (nb * KB + kk) * kAcross + brow : n0 + nb * 16 + r16;
          const int r = kStaged ? brank : kk * 32 + lg * 8;
          bf[p][nb][kk] = *(const u32x4*)(w + (long long)min(n, a.N - 1) * a.R + (r < ld.rank ? r : 0));
        }
      more = ld.next(mine);
    };
    f32x4 f[MB][4];  // this lane's row r16 of a block, columns 16 nb + 4 lg + 0 .. 3
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
      for (int nb = 0; nb < 4; ++nb) f[mb][nb] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    auto add = [&](int p) {
      if (!left) return;
      if (cp.rank & 7) {  // a vector holds values past the adapter's rank
#pragma unroll
        for (int kk = 0; kk < KB; ++kk) {
          const int r = kStaged ? brank : kk * 32 + lg * 8;
          const int used = cp.rank - (r < cp.rank ? r : 0);  // values of this lane's vector in use
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const uint32_t keep = used >= 2 * w + 2 ? 0xffffffffu : used == 2 * w + 1 ? 0xffffu : 0u;
#pragma unroll
            for (int nb = 0; nb < 4; ++nb) bf[p][nb][kk][w] &= keep;
          }
        }
      }
      if constexpr (kStaged) {
        // through LDS from the order of memory to the operands'; LDS serves
        // one wave's accesses in order
        order();
#pragma unroll
        for (int i = 0; i < 4 * KB; ++i) *(u32x4*)&stage[i * kAcross + brow][brank] = bf[p][i / KB][i % KB];
        order();
#pragma unroll
        for (int nb = 0; nb < 4; ++nb)
#pragma unroll
          for (int kk = 0; kk < KB; ++kk) bf[p][nb][kk] = *(const u32x4*)&stage[nb * 16 + r16][kk * 32 + lg * 8];
      }
#pragma unroll
      for (int mb = 0; mb < MB; ++mb) {
        const uint32_t rows = (uint32_t)(cp.rows >> (mb * 16)) & 0xffffu;
        if (MB > 1 && rows == 0) continue;
        f32x4 acc[4];
#pragma unroll
        for (int nb = 0; nb < 4; ++nb) acc[nb] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int kk = 0; kk < KB; ++kk) {
          V8 v[kTerms];
#pragma unroll
          for (int t = 0; t < kTerms; ++t) v[t] = *(const V8*)&vterms[t][mb * 16 + r16][kk * 32 + lg * 8];
#pragma unroll
          for (int nb = 0; nb < 4; ++nb)
#pragma unroll
            for (int t = 0; t < kTerms; ++t) acc[nb] = mma(__builtin_bit_cast(V8, bf[p][nb][kk]), v[t], acc[nb]);
        }
        const bool own = (rows >> r16) & 1u;
        const float s = up[mb * 16 + r16];
#pragma unroll
        for (int nb = 0; nb < 4; ++nb)
#pragma unroll
          for (int i = 0; i < 4; ++i) f[mb][nb][i] = own ? acc[nb][i] * s : f[mb][nb][i];
      }
      left = cp.next(mine);
    };
    while (left) {  // P requests at a time
#pragma unroll
      for (int p = 0; p < P; ++p) load(p);
#pragma unroll
      for (int p = 0; p < P; ++p) add(p);
    }
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) {
      order();
#pragma unroll
      for (int nb = 0; nb < 4; ++nb) *(f32x4*)&turn[r16][nb * 16 + lg * 4] = f[mb][nb];
      const f32x4 all = (f[mb][0] + f[mb][1]) + (f[mb][2] + f[mb][3]);
      const float one = (all[0] + all[1]) + (all[2] + all[3]);
      if (__any(one != one)) sum_again(mb);  // a NaN, or infinities of both signs
      finish(mb, yv[mb]);
    }
  }
}

// How a call is cut (times in us, K = N = 4096, rank 64, first + second product):
//   up to kFewTokens: a wave per (token, rank) and per (token, 64 columns).
//     128 tokens: 13, in tiles 14 for one adapter and 26 for eight in turn;
//     256 tokens: 21, in tiles 14 and 28 (rank 16: 12, in tiles 13 and 20);
//   up to kSomeTokens: a workgroup per (4 tokens, 16 ranks), expand in tiles;
//   more: both in tiles, K in parts that fill the compute units.  The first
//     product of 1024 tokens: 16 for one adapter and 31 for eight in turn by
//     fours, of 1025 in tiles 10 and 52.
// Expand's tiles have 64 rows where that leaves four workgroups per compute
// unit (B's block is then read a quarter as often), else 16.
struct Cut {
  int mb;  // expand's tiles: 16 mb rows (0: rows one by one)
  int parts, k_part, columns;
};

Cut cut_of(int64_t M, int64_t K, int64_t N) {
  Cut c = {0, 1, (int)K, 1};
  if (M > kSomeTokens) {
    const int64_t tiles = (M + 63) / 64;
    int64_t parts = (4 * kUnits + tiles - 1) / tiles;
    if (parts > (K + 511) / 512) parts = (K + 511) / 512;
    c.k_part = (int)(((K + parts - 1) / parts + 127) / 128 * 128);
    c.parts = (int)((K + c.k_part - 1) / c.k_part);
  }
  if (M > kFewTokens) {
    const int64_t across = (N + 255) / 256;
    c.mb = ((M + 63) / 64) * across >= 4 * kUnits ? 4 : 1;
    const int64_t work = ((M + 16 * c.mb - 1) / (16 * c.mb)) * across;
    c.columns = work >= 16 * kUnits ? 4 : work >= 8 * kUnits ? 2 : 1;
  }
  return c;
}

template <class T>
hipError_t launch_shrink(const AdapterArgs& a, hipStream_t stream) {
  const dim3 block(256);
  if (a.M <= kFewTokens) {
    shrink_rows_kernel<T><<<dim3(a.M, (a.R + 3) / 4), block, 0, stream>>>(a);
  } else if (a.M <= kSomeTokens) {
    shrink_fours_kernel<T><<<dim3((a.M + 3) / 4, (a.R + 15) / 16), block, 0, stream>>>(a);
  } else {
    const dim3 grid((a.M + 63) / 64, a.slices + a.parts);
    const int rb = (a.R + 15) / 16;
    if (rb == 1) shrink_staged_kernel<T, 1><<<grid, block, 0, stream>>>(a);
    else if (rb == 2) shrink_staged_kernel<T, 2><<<grid, block, 0, stream>>>(a);
    else if (rb <= 4) shrink_staged_kernel<T, 4><<<grid, block, 0, stream>>>(a);
    else shrink_staged_kernel<T, 8><<<grid, block, 0, stream>>>(a);
  }
  return hipGetLastError();
}

template <class T, class YT, int VW, int KB>
hipError_t launch_expand_kb(AdapterArgs a, int mb, hipStream_t stream) {
  const auto grid = [&](int rows) {
    const uint64_t across = a.blocks >= 8 ? (a.blocks + 7) / 8 * 8 : a.blocks;
    return (a.M + rows - 1) / rows * across;
  };
  if (grid(16) >= (1ull << 24)) return hipErrorInvalidConfiguration;  // 2^32 threads
  constexpr int kInFlight = KB == 1 ? 4 : KB == 2 ? 2 : 1;  // requests whose blocks of B are loaded together
  if (mb == 1) expand_tiles_kernel<T, YT, 1, KB, VW, kInFlight><<<dim3(grid(16)), dim3(256), 0, stream>>>(a);
  else expand_tiles_kernel<T, YT, 4, KB, VW, 1><<<dim3(grid(64)), dim3(256), 0, stream>>>(a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (mb == 1) {  // few tiles: as many workgroups as there are blocks of columns
    a.columns = 1;
    a.blocks = (a.N + 255) / 256;
    expand_singles_kernel<T, YT, 16, KB, VW><<<dim3(grid(16)), dim3(256), 0, stream>>>(a);
  } else {
    expand_singles_kernel<T, YT, 64, KB, VW><<<dim3(grid(64)), dim3(256), 0, stream>>>(a);
  }
  return hipGetLastError();
}

template <class T, class YT, int VW>
hipError_t launch_expand(const AdapterArgs& a, int mb, hipStream_t stream) {
  const int kb = (a.R + 31) / 32;
  if (kb == 1) return launch_expand_kb<T, YT, VW, 1>(a, mb, stream);
  if (kb == 2) return launch_expand_kb<T, YT, VW, 2>(a, mb, stream);
  return launch_expand_kb<T, YT, VW, 4>(a, mb, stream);
}

template <class T, class YT>
hipError_t launch_y(AdapterArgs& a, const Cut& c, hipStream_t stream) {
  if (c.mb == 0) {
    const dim3 grid(a.M, (a.N + 255) / 256);
    if (a.R <= 32) expand_rows_kernel<T, YT, 1><<<grid, dim3(256), 0, stream>>>(a);
    else if (a.R <= 64) expand_rows_kernel<T, YT, 2><<<grid, dim3(256), 0, stream>>>(a);
    else expand_rows_kernel<T, YT, 4><<<grid, dim3(256), 0, stream>>>(a);
    return hipGetLastError();
  }
  // y's and out's rows in vectors of eight, four or single elements
  const auto whole = [&](int w) {
    return a.N % w == 0 && a.ys % w == 0 && a.os % w == 0 && aligned_to(a.y, w * (int)sizeof(YT) > 16 ? 16 : w * (int)sizeof(YT)) &&
           aligned_to(a.out, w * (int)sizeof(YT) > 16 ? 16 : w * (int)sizeof(YT));
  };
  constexpr int kWide = 16 / sizeof(YT);  // elements of 16 bytes
  if (whole(kWide)) return launch_expand<T, YT, kWide>(a, c.mb, stream);
  if (kWide > 4 && whole(4)) return launch_expand<T, YT, 4>(a, c.mb, stream);
  return launch_expand<T, YT, 1>(a, c.mb, stream);
}

template <class T>
hipError_t launch(AdapterArgs& a, const Cut& c, int y_dtype, hipStream_t stream) {
  const hipError_t e = launch_shrink<T>(a, stream);
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
  return M * rank * 4 * cut_of(M, K, 1).parts;
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
  if (!vector_rows(p->x, p->M > 1 ? p->x_stride : 0) || !aligned_to(p->y, yb) || !aligned_to(p->out, yb)) return ORBIT_E_ARG;
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
  a.xs = p->M > 1 ? p->x_stride : 0;  // one row's stride says nothing
  a.ys = p->M > 1 ? p->y_stride : 0;
  a.os = p->M > 1 ? p->out_stride : 0;
  a.M = (uint32_t)p->M;
  a.adapters = (uint32_t)p->adapters;
  a.K = (int)p->K;
  a.N = (int)p->N;
  a.R = (int)p->rank;
  const Cut c = cut_of(p->M, p->K, p->N);
  a.parts = c.parts;
  a.slices = p->M > 4096 ? 4 : 16;  // a thousand short workgroups at most, or 16 rows to each
  a.k_part = c.k_part;
  a.columns = c.columns;
  a.blocks = (a.N + 256 * c.columns - 1) / (256 * c.columns);
  return hip_status(p->x_dtype == ORBIT_BF16 ? launch<__bf16>(a, c, p->y_dtype, stream) : launch<_Float16>(a, c, p->y_dtype, stream));
}
