// orbit_int8_qlinear: the product of 8-bit integers with a scale for each
// token and each channel,
//   y[m, n] = act(sx[m] sw[n] sum_k qx[m, k] qw[n, k] + bias[n]),
// on the int8 matrix cores; the sums are exact (int32), the scales, the bias
// and the activation float32, and y is rounded once.
//
// Two kernels.
// * tile_kernel, for products with enough tiles to fill the chip.  Bound: the
//   matrix cores, and what a compute unit takes in (launch_product).  16384 x
//   4096 -> 4096 243 to 262 us (2.1 to 2.3 POP/s; the library's int8 product of
//   8192^3 2.1), 4096 x 3072 -> 3072 39 to 41 us.
// * thin_kernel, for few tokens or few tiles.  Bound: the weights' bytes, or
//   what a compute unit takes in.  16 x 3072 -> 18432 11 us (5.1 TB/s).
// Everywhere the weights are the matrix instruction's A operand (rows) and
// the tokens its B operand (columns), so that a lane's results are
// neighbouring channels of one token.
//
// K is a multiple of 16.  What lies past a row's end inside a chunk is
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
// GELU in its erf form, y / 2 (1 + erf(y / sqrt 2)): erfc(x) = t P(t) exp(-x^2),
// t = 1 / (1 + 3 x / 8), x >= 0, P of degree 8 fitted here to exp(x^2) erfc(x)
// over 0 <= x <= 10 (relative error 1.4e-8); below zero 1 + erf is that small
// term itself, so that the tail keeps its digits (relative error 4e-7 down to y =
// -1, 1.1e-6 to -3, 2e-5 at -12, what float32 leaves of x^2; a P of degree 4 was
// within 1.5e-7 of 1, and 5e-5 off at -3, 4e-3 at -6).
__device__ __forceinline__ float activate(float y, int act) {
  if (act != ORBIT_ACT_GELU) return y;
  const float x = fabsf(y) * 0.70710678118654752f;
  const float t = __builtin_amdgcn_rcpf(fmaf(0.375f, x, 1.0f));
  float p = fmaf(0.06120922f, t, -0.28577687f);
  p = fmaf(p, t, 0.42928435f);
  p = fmaf(p, t, -0.22595349f);
  p = fmaf(p, t, 0.27140034f);
  p = fmaf(p, t, 0.12246978f);
  p = fmaf(p, t, 0.20507229f);
  p = fmaf(p, t, 0.2106828f);
  p = fmaf(p, t, 0.21161156f) * t;
  const float rest = p * __builtin_amdgcn_exp2f(-(x * x) * 1.4426950408889634f);
  return 0.5f * y * (y < 0.0f ? rest : 2.0f - rest);
}
template <class OT>
__device__ __forceinline__ void store8(OT* p, const float (&f)[8]) {
  Vec8<OT> v;
#pragma unroll
  for (int j = 0; j < 8; ++j) v.e[j] = (OT)f[j];
  *(Vec8<OT>*)p = v;
}

// Sums of `rows` tokens (from m0) and `cols` channels (from n0) that lie in
// LDS as int32 [rows][pitch], the tokens' scales behind them in column `cols`,
// finished and stored by `threads` threads.  Where rows are vectors (a.vec) a
// thread has eight channels of every so many-th row, whose scales and bias it
// reads before the product (by 256 x 192 they took 24000 of 80000 cycles when
// each row's were read in its turn).
// Otherwise one channel at a time (2048 x 2048 -> 8193 60 us; 96 when scale
// and bias were read for each result).
struct Finish {
  float sw[8], b[8];
  int r0, c, at_once;
  bool in;
  long long n;
  __device__ __forceinline__ Finish(const ProductArgs& a, int cols, long long n0, int t, int threads) {
    const int per = cols / 8;  // vectors of a row
    at_once = threads / per;   // rows
    r0 = t / per;
    c = (t - r0 * per) * 8;
    n = n0 + c;
    in = r0 < at_once && n < a.N;  // vec: N is a multiple of 8
    if (!a.vec || !in) return;
    const float* const w = a.sw + n;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      sw[j] = w[j];
      b[j] = 0.0f;
    }
    if (!a.bias) return;
    auto read = [&](auto* bias) {
#pragma unroll
      for (int j = 0; j < 8; ++j) b[j] = (float)bias[n + j];
    };
    if (a.bias_dtype == ORBIT_BF16) read((const __bf16*)a.bias);
    else if (a.bias_dtype == ORBIT_F16) read((const _Float16*)a.bias);
    else read((const float*)a.bias);
  }
  template <class OT>
  __device__ __forceinline__ void store(const ProductArgs& a, const int* sums, int pitch, int rows, int cols, long long m0, long long n0,
                                        int t, int threads) const {
    auto scale = [&](int r) { return __builtin_bit_cast(float, sums[r * pitch + cols]); };
    if (a.vec) {
      if (!in) return;
      const int end = (int)min((long long)rows, a.M - m0);
#pragma unroll 2
      for (int r = r0; r < end; r += at_once) {
        const float sx = scale(r);
        const i32x4 x = *(const i32x4*)(sums + r * pitch + c), y = *(const i32x4*)(sums + r * pitch + c + 4);
        float f[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = activate(fmaf((float)(j < 4 ? x[j & 3] : y[j & 3]), sx * sw[j], b[j]), a.act);
        store8((OT*)a.out + (m0 + r) * a.N + n, f);
      }
    } else {
      const int width = cols < threads ? cols : threads, step = threads / width, end = (int)min((long long)rows, a.M - m0);
      if (t >= step * width) return;
      for (int q = t % width; q < cols && n0 + q < a.N; q += width) {
        const float w = a.sw[n0 + q], bias = bias_of(a, n0 + q);
#pragma unroll 4
        for (int r = t / width; r < end; r += step)
          ((OT*)a.out)[(m0 + r) * a.N + n0 + q] = (OT)activate(fmaf((float)sums[r * pitch + q], scale(r) * w, bias), a.act);
      }
    }
  }
};

// The loads that go from memory straight to LDS are inline assembly with
// explicit waits: they have no register results, and the compiler would wait
// for every one of them before each LDS read.  gfx9 asks for a wait state
// between the write of m0 and the load, which is the block's own to keep.
__device__ __forceinline__ void load_lds(uint32_t to, uint32_t offset, const char* base) {  // 1 KB: lane l's 16 bytes to `to` + 16 l
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(to), "v"(offset), "s"(base) : "memory");
}
template <int N>
__device__ __forceinline__ void wait_loads() {  // until at most N loads of this wave are in flight, and no LDS read
  static_assert(N >= 0 && N < 64);
  __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | ((N >> 4) << 14));
}
__device__ __forceinline__ void meet() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}


// ---- few tokens ---------------------------------------------------------------
//
// A workgroup of eight waves takes 16 RB channels and up to 16 MB tokens
// (v_mfma_i32_16x16x64_i8); wave w the 128-byte chunks w, w + 8, ... of K,
// through an LDS ring of its own, so that no barrier stands between two
// chunks.  With rings of one stage two or three workgroups share a compute
// unit, one's loads beside another's sums (16 x 3072 -> 18432 with its tokens'
// codes made first: 16.2 us, with three stages and one workgroup 19.6).  The
// waves' sums are added in LDS (integers: the order does not matter).
// A chunk is blocks of 8 rows, one load instruction each (whole lines: blocks
// of 16 rows of 64 bytes were 5 to 10 % slower); 16-byte unit u of row r lies
// at 128 r + 16 (u ^ (r / 2) % 8), which puts the 16 rows that LDS serves at
// once in 16 different places of 256 bytes.
template <class OT, int MB, int RB, int S>
__global__ __launch_bounds__(512) void thin_kernel(ProductArgs a) {
  constexpr int kPitch = 16 * RB + 4, kChunk = (MB + RB) * 2048, kLoads = 2 * (MB + RB);
  extern __shared__ __align__(16) char smem[];
  int* const sums = (int*)smem;
  static_assert(16 * MB * kPitch * 4 <= 8 * S * kChunk, "the sums lie over the rings");
  const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int r16 = lane & 15, g = lane >> 4;
  const long long n0 = (long long)blockIdx.x * (16 * RB), m0 = (long long)blockIdx.y * (16 * MB);
  const char *const wbase = a.w + n0 * a.K, *const xbase = a.x + m0 * a.K;
  // this lane's sources: row lane / 4 of each block (past the end: the last
  // row again, whose results are dropped)
  const uint32_t unit = ((uint32_t)lane & 7u) ^ ((uint32_t)lane >> 4);
  uint32_t from[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int r = (i < 2 * RB ? i : i - 2 * RB) * 8 + (lane >> 3);
    from[i] = (uint32_t)min((long long)r, (i < 2 * RB ? a.N - n0 : a.M - m0) - 1) * (uint32_t)a.K + (unit ^ (i & 1 ? 4u : 0u)) * 16u;
  }
  const int chunks = (a.K + 127) / 128, mine = (chunks - wave + 7) / 8;  // 0 where K is short
  // bytes past the row's end: the row's last 16 again (multiplied as zero)
  auto back = [&](int b) { return (uint32_t)max(0, (chunks - 1) * 128 + (int)((unit ^ (b & 1 ? 4u : 0u)) * 16u) - (a.K - 16)); };
  const uint32_t ring = (uint32_t)wave * (S * kChunk);
  auto issue = [&](int i) {
    const int c = wave + 8 * i;
    const uint32_t at = (uint32_t)c * 128u, st = ring + (uint32_t)(i % S) * kChunk;
#pragma unroll
    for (int b = 0; b < kLoads; ++b) load_lds(st + b * 1024u, from[b] + at - (c == chunks - 1 ? back(b) : 0u), b < 2 * RB ? wbase : xbase);
  };
  const Finish finish(a, 16 * RB, n0, t, 512);
  const float sx = t < 16 * MB && m0 + t < a.M ? a.sx[m0 + t] : 0.0f;
  i32x4 acc[RB][MB];
#pragma unroll
  for (int i = 0; i < RB; ++i)
#pragma unroll
    for (int j = 0; j < MB; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < S; ++i)
    if (i < mine) issue(i);
  const uint32_t at = ring + (uint32_t)r16 * 128u, key = (uint32_t)r16 >> 1;
  for (int i = 0; i < mine; ++i) {
    if (mine - 1 - i >= S - 1) wait_loads<(S - 1) * kLoads>();
    else wait_loads<0>();  // the last few
    const char* const st = smem + at + (uint32_t)(i % S) * kChunk;
    i32x4 wv[2][RB], xv[2][MB];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t u = ((uint32_t)(4 * h + g) ^ key) << 4;
#pragma unroll
      for (int b = 0; b < RB; ++b) wv[h][b] = *(const i32x4*)(st + u + b * 2048);
#pragma unroll
      for (int b = 0; b < MB; ++b) xv[h][b] = *(const i32x4*)(st + u + (RB + b) * 2048);
    }
    const int c = wave + 8 * i;
    if (c * 128 + 128 > a.K) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const bool in = c * 128 + h * 64 + g * 16 < a.K;
#pragma unroll
        for (int b = 0; b < RB; ++b) wv[h][b] = in ? wv[h][b] : i32x4{0, 0, 0, 0};
      }
    }
    __builtin_amdgcn_s_waitcnt(0xc07f);  // this stage has been read
    asm volatile("" ::: "memory");
    if (i + S < mine) issue(i + S);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int b = 0; b < RB; ++b)
#pragma unroll
        for (int m = 0; m < MB; ++m) acc[b][m] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wv[h][b], xv[h][m], acc[b][m], 0, 0, 0);
  }
  __syncthreads();
  for (int i = t; i < 16 * MB * kPitch; i += 512) sums[i] = 0;
  __syncthreads();
  if (t < 16 * MB) sums[t * kPitch + 16 * RB] = __builtin_bit_cast(int, sx);
#pragma unroll
  for (int i = 0; i < RB; ++i)
#pragma unroll
    for (int j = 0; j < MB; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) atomicAdd(&sums[(16 * j + r16) * kPitch + 16 * i + g * 4 + q], acc[i][j][q]);
  __syncthreads();
  finish.template store<OT>(a, sums, kPitch, 16 * MB, 16 * RB, m0, n0, t, 512);
}

template <class OT, int MB, int RB, int S>
hipError_t launch_thin(ProductArgs a, hipStream_t stream) {
  constexpr int kLds = 8 * S * (MB + RB) * 2048;
  auto kern = thin_kernel<OT, MB, RB, S>;
  static LaunchCache cache;
  const hipError_t e = prepare_launch(cache, (const void*)kern, 512, kLds, nullptr);
  if (e != hipSuccess) return e;
  const dim3 grid((unsigned)((a.N + 16 * RB - 1) / (16 * RB)), (unsigned)((a.M + 16 * MB - 1) / (16 * MB)));
  kern<<<grid, dim3(512), kLds, stream>>>(a);
  return hipGetLastError();
}

// ---- many tiles ---------------------------------------------------------------
//
// A workgroup of WGM x WGN waves takes TM tokens x TN channels, a wave BM x BN
// blocks of 32 x 32 (v_mfma_i32_32x32x32_i8: lane l holds row or column l % 32
// and 16 bytes of k, the instruction's slots 16 (l / 32) ..).
// Chunks of 128 bytes of K of both operands pass through a ring of S LDS
// stages: while a chunk is multiplied, S - 1 are in flight.  Chunks of 64
// bytes in rings of twice the stages took 281 us for 260 (16384 x 4096 ->
// 4096).  A stage is laid out as the thin kernel's chunk.  A lane reads unit
// 2 s + l / 32 in step s (of four): both operands alike, so the order of k
// does not matter.
template <class OT, int WGM, int WGN, int BM, int BN, int S>
__global__ __launch_bounds__(64 * WGM * WGN) void tile_kernel(ProductArgs a) {
  constexpr int kWaves = WGM * WGN, TM = 32 * WGM * BM, TN = 32 * WGN * BN;
  constexpr int kStage = (TM + TN) * 128, kBlocks = (TM + TN) / 8;
  constexpr int kLoads = (kBlocks + kWaves - 1) / kWaves, kRest = kBlocks % kWaves;  // waves below kRest load one more
  constexpr int kPitch = 32 * BN + 4;
  static_assert(kWaves * 32 * kPitch * 4 <= S * kStage, "the results pass through the ring's memory");
  extern __shared__ __align__(16) char smem[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WGN, wn = wave - wm * WGN;

  // Each XCD (workgroups go round them) takes a row of neighbouring tiles, in
  // groups of 8 token tiles, so that what runs at once shares its operands in
  // the XCD's L2.
  const int tiles = a.tiles_m * a.tiles_n, each = (tiles + 7) / 8;
  const int tile = ((int)blockIdx.x & 7) * each + ((int)blockIdx.x >> 3);
  if (((int)blockIdx.x >> 3) >= each || tile >= tiles) return;
  const int group = tile / (8 * a.tiles_n), in_group = tile - group * 8 * a.tiles_n;
  const int height = min(8, a.tiles_m - group * 8);
  const int tn = in_group / height, tm = group * 8 + in_group - tn * height;
  const long long m0 = (long long)tm * TM, n0 = (long long)tn * TN;

  // this lane's sources (rows past the end: the last one again, whose results are dropped)
  const char* const xbase = a.x + m0 * a.K;
  const char* const wbase = a.w + n0 * a.K;
  const int last = (a.K + 127) / 128 - 1;
  // key of row r: (r / 2) % 8; a block's rows begin at a multiple of 8
  const uint32_t unit = ((uint32_t)lane & 7u) ^ ((uint32_t)lane >> 4);
  uint32_t from[kLoads];
  #pragma unroll
  for (int q = 0; q < kLoads; ++q) {
    const int blk = q * kWaves + wave, r = blk * 8 + (lane >> 3);
    const long long row = blk < TM / 8 ? min((long long)r, a.M - 1 - m0) : min((long long)r - TM, a.N - 1 - n0);
    from[q] = (uint32_t)row * (uint32_t)a.K + (unit ^ (blk & 1 ? 4u : 0u)) * 16u;
  }
  // bytes past the row's end in the last chunk: the row's last 16 again (multiplied as zero, below)
  auto back = [&](int blk) { return (uint32_t)max(0, last * 128 + (int)((unit ^ (blk & 1 ? 4u : 0u)) * 16u) - (a.K - 16)); };
  auto issue = [&](int c) {
    const uint32_t st = (uint32_t)(c % S) * kStage;
    const uint32_t at = (uint32_t)c * 128u;
#pragma unroll
    for (int q = 0; q < kLoads; ++q) {
      const int blk = q * kWaves + wave;
      if (kRest && q == kLoads - 1 && blk >= kBlocks) break;
      load_lds(st + (uint32_t)blk * 1024u, from[q] + at - (c == last ? back(blk) : 0u), blk < TM / 8 ? xbase : wbase);
    }
  };
  // chunk c has landed, for this wave's loads: `later` chunks may be in flight
  auto landed = [&](int later) {
    const bool more = kRest == 0 || wave < kRest;
    constexpr int kLess = kRest ? kLoads - 1 : kLoads;
    auto wait = [&](auto n) { more ? wait_loads<decltype(n)::value * kLoads>() : wait_loads<decltype(n)::value * kLess>(); };
    if (later >= S - 1) wait(std::integral_constant<int, S - 1>{});
    else if (later == S - 2) wait(std::integral_constant<int, S - 2>{});
    else if (later >= 1) wait(std::integral_constant<int, 1>{});
    else wait_loads<0>();
  };
  // where K ends inside the last chunk, its weights' other bytes become zeros
  auto arrived = [&](int c) {
    if (c == last && (a.K & 127)) {
      char* const st = smem + (c % S) * kStage + TM * 128;
      for (int i = threadIdx.x; i < TN * 8; i += 64 * kWaves) {
        const int r = i >> 3, u = (i & 7) ^ ((r >> 1) & 7);
        if (c * 128 + u * 16 >= a.K) *(i32x4*)(st + i * 16) = i32x4{0, 0, 0, 0};
      }
      __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0)
      meet();
    }
  };

  const int r32 = lane & 31, half = lane >> 5;
  const uint32_t key = ((uint32_t)r32 >> 1) & 7u;
  const uint32_t rx = (uint32_t)(wm * BM * 32 + r32) * 128u, rw = (uint32_t)(TM + wn * BN * 32 + r32) * 128u;
  i32x4 xv[2][BM], wv[2][BN];
  auto read = [&](int set, int c, int step) {
    const char* const st = smem + (c % S) * kStage + (((uint32_t)(2 * step + half) ^ key) << 4);
#pragma unroll
    for (int j = 0; j < BN; ++j) wv[set][j] = *(const i32x4*)(st + rw + j * 4096);
#pragma unroll
    for (int i = 0; i < BM; ++i) xv[set][i] = *(const i32x4*)(st + rx + i * 4096);
  };
  const Finish finish(a, 32 * BN, n0 + wn * BN * 32, lane, 64);
  float sx[BM];
#pragma unroll
  for (int i = 0; i < BM; ++i) sx[i] = a.sx[min(m0 + (wm * BM + i) * 32 + r32, a.M - 1)];
  i32x16 acc[BN][BM];
#pragma unroll
  for (int j = 0; j < BN; ++j)
#pragma unroll
    for (int i = 0; i < BM; ++i)
#pragma unroll
      for (int q = 0; q < 16; ++q) acc[j][i][q] = 0;
  auto mma = [&](int set) {
#pragma unroll
    for (int j = 0; j < BN; ++j)
#pragma unroll
      for (int i = 0; i < BM; ++i) acc[j][i] = __builtin_amdgcn_mfma_i32_32x32x32_i8(wv[set][j], xv[set][i], acc[j][i], 0, 0, 0);
  };
  // the next step's reads go out between this one's products
  auto interleave = [&] {
#pragma unroll
    for (int q = 0; q < BM * BN; ++q) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
  };

#pragma unroll
  for (int c = 0; c < S; ++c)
    if (c <= last) issue(c);
  landed(min(last, S - 1));
  meet();
  arrived(0);
  read(0, 0, 0);
  for (int c = 0; c <= last; ++c) {
#pragma unroll
    for (int step = 0; step < 3; ++step) {
      read((step + 1) & 1, c, step + 1);
      mma(step & 1);
      interleave();
    }
    // chunk c + 1 is there, and nobody reads chunk c any more
    landed(min(last - c - 1, S - 2));
    meet();
    if (c + S <= last) issue(c + S);
    arrived(c + 1);
    read(0, c + 1, 0);  // behind the last chunk: memory of the ring, not used
    mma(1);
    interleave();
  }
  __syncthreads();

  int* const mine = (int*)smem + wave * 32 * kPitch;
#pragma unroll
  for (int i = 0; i < BM; ++i) {
#pragma unroll
    for (int j = 0; j < BN; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *(i32x4*)(mine + r32 * kPitch + 32 * j + 8 * q + 4 * half) =
            i32x4{acc[j][i][4 * q], acc[j][i][4 * q + 1], acc[j][i][4 * q + 2], acc[j][i][4 * q + 3]};
    if (half == 0) mine[r32 * kPitch + 32 * BN] = __builtin_bit_cast(int, sx[i]);
    // the wave's own rows: LDS serves a wave in order
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    finish.template store<OT>(a, mine, kPitch, 32, 32 * BN, m0 + (wm * BM + i) * 32, n0 + wn * BN * 32, lane, 64);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
}

template <class OT, int WGM, int WGN, int BM, int BN, int S>
hipError_t launch_tiles(ProductArgs a, hipStream_t stream) {
  constexpr int TM = 32 * WGM * BM, TN = 32 * WGN * BN, kLds = S * (TM + TN) * 128;
  a.tiles_m = (int)((a.M + TM - 1) / TM);
  a.tiles_n = (int)((a.N + TN - 1) / TN);
  auto kern = tile_kernel<OT, WGM, WGN, BM, BN, S>;
  static LaunchCache cache;
  const hipError_t e = prepare_launch(cache, (const void*)kern, 64 * WGM * WGN, kLds, nullptr);
  if (e != hipSuccess) return e;
  const long long each = ((long long)a.tiles_m * a.tiles_n + 7) / 8;
  kern<<<dim3((unsigned)(8 * each)), dim3(64 * WGM * WGN), kLds, stream>>>(a);
  return hipGetLastError();
}

// The variant that the sizes give the least time by this estimate: a compute
// unit takes ceil(workgroups / units) workgroups, each as long as its
// (TM + TN) K operand bytes at 50 KB/us (what a unit was seen to take in, from
// one workgroup on the whole chip to several on each unit) or its 2 TM TN K
// operations at 9 per ps (the chip's settled 2.3 POP/s, shared), whichever is
// longer.  Measured, us (thin tiles of 16 x 32, 32 x 32, 64 x 32, 64 x 64; 128
// x 128, 256 x 192, 256 x 256): 16 x 3072 -> 18432 11.1, 12.6, 17.3, 18.6;
// 14.5, 25.9, 32.0.  64 x 4096 -> 4096 7.8, 6.2, 7.4, 16.3; 18.9, 34.9, 41.7.
// 256 x 4096 -> 4096 21.1, 16.5, 14.3, 10.2; 18.9, 35.9, 44.1.  333 x 2064 ->
// 8200 (-), 36.8; 13.2, 24.1, 29.7.  1024 x 4096 -> 4096 (-), 37.6; 22.7, 37.4,
// 46.1.  4096 x 3072 -> 3072 (-), 90.9; 51.4, 39.4, 41.7.  16384 x 4096 -> 4096
// (-), 534; 347, 277, 243.
template <class OT>
hipError_t launch_product(const ProductArgs& a, hipStream_t stream) {
  typedef hipError_t (*Launch)(ProductArgs, hipStream_t);
  static const struct {
    int tm, tn;
    Launch launch;
  } kVariants[] = {
      {16, 16, launch_thin<OT, 1, 1, 4>}, {16, 32, launch_thin<OT, 1, 2, 1>},  {32, 32, launch_thin<OT, 2, 2, 1>},
      {64, 32, launch_thin<OT, 4, 2, 1>}, {64, 64, launch_thin<OT, 4, 4, 1>},  {128, 128, launch_tiles<OT, 2, 4, 2, 1, 3>},
      {256, 192, launch_tiles<OT, 4, 2, 2, 3, 2>}, {256, 256, launch_tiles<OT, 2, 4, 4, 2, 2>}};
  Launch best = nullptr;
  double least = 0.0;
  for (const auto& v : kVariants) {
    const long long groups = ((a.M + v.tm - 1) / v.tm) * ((a.N + v.tn - 1) / v.tn);
    if ((a.M + v.tm - 1) / v.tm > 65535) continue;  // the grid's second dimension
    const double bytes = (v.tm + v.tn) / 50e3, ops = 2.0 * v.tm * v.tn / 9e6;
    const double us = (double)((groups + kUnits - 1) / kUnits) * (bytes > ops ? bytes : ops);
    if (!best || us < least) {
      best = v.launch;
      least = us;
    }
  }
  return best(a, stream);
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
    case ORBIT_BF16: e = launch_product<__bf16>(a, stream); break;
    case ORBIT_F16: e = launch_product<_Float16>(a, stream); break;
    default: e = launch_product<float>(a, stream);
  }
  return hip_status(e);
}
