// Attention of one new token per request over the paged cache
// (orbit_paged_attention):
//   o = sum_t p_t v_t / sum_t p_t,  p_t = exp(sm_scale q . k_t - m),
// the maximum m and the sums carried along the tokens (one pass over the
// cache).
//
// Bound: memory; per byte of a 16-bit cache there are 2 (q_heads / kv_heads)
// multiply-adds.  64 ragged requests of up to 8192 tokens, 32 / 8 heads of
// 128 in bf16: 180 us (5.2 TB/s); 16 of up to 65000 in int8, 24 / 4 heads:
// 124 us (3.8 TB/s, bound by the loads that three workgroups per compute unit
// keep in flight); one of 700 tokens: 10 us, two launches.
//
// Split.  A workgroup of four waves takes one key head of one request, up to
// 16 of the query heads that share it, and `chunk` tokens; wave w takes the
// tiles of 32 tokens w, w + 4, ... with sums of its own, so no barrier
// stands between two tiles.  The waves' sums meet once in LDS.  Contexts of
// more than one chunk leave partial sums in the workspace, which a second
// kernel joins in a fixed order.
//
// Products on the matrix cores (16x16x32), also for a single query head: the
// unused rows cost nothing that bounds the kernel.
//   S^T = K Q^T: A = 16 tokens x 32 coordinates, B = the queries, kept in
//   registers.  Keys are loaded like values, whole rows by neighbouring
//   lanes, and pass through LDS: read from memory in the operands' order
//   (neighbouring lanes in 16 rows) they cost the address unit four times
//   the cycles, and the second load of a line waits for the first's.  A lane
//   then holds head l % 16 and tokens 4 (l / 16) + i of each half tile.
//   O^T = V^T P^T: those lanes' probabilities are the B operand as they
//   stand if operand slot 8 g + j means token 4 g + j of the first half
//   (j < 4) or 4 g + j - 4 of the second.  A = V^T needs four tokens of one
//   coordinate side by side: values go through the wave's own LDS rows and
//   come back by the transposing read (ds_read_b64_tr_b16).
// Probabilities are multiplied as hi + lo pairs of 16-bit numbers (two
// products): 16 bits of each in bf16, for an output that keeps 8; 22 in fp16,
// for one that keeps 11 (8 with bf16 queries on an int8 cache).  bf16 has
// float32's range.  fp16 does not, and a context's many small weights may be
// all there is of an output (where the largest belongs to a token whose value
// is zero), so fp16 operands hold 2^15 p (kLift): their steps begin at 2^-39
// of the largest weight, a loss of 2^-19 of it over a million tokens (without
// the factor they began at 2^-24, and such outputs were 3 % off where the
// largest score led by 14; the time is the same, 124.6 us for the int8 case).
// The denominator is a float32 sum of unsplit weights.
// Such a pair has no product with an infinite value: lo may be zero or below.
// A wave that ends with a NaN therefore looks through its tokens once more,
// outside the loop: the infinite values decide (the test for a NaN takes 0.6 of
// the 180 us; pairs that are never zero or below would take a maximum each, in
// the loop, and add a little of every hidden weight).  Factors on sums (rescaling,
// joining) do not go below float32's smallest normal number, so that an
// infinite sum stays infinite.
//
// INT8 cache: codes become fp16 integers exactly (a byte permute and one
// packed subtraction).  A key's scale multiplies its score.  A value's scale
// goes into its probability, with the running maximum taken of z_t +
// log2(scale_t), so that the products stay in [0, 1] whatever the scales'
// size (before the lift).  Queries are scaled by a power of two per head to
// fit fp16.
#pragma once

#include "kv_cache.h"

namespace orbit {
namespace block {

struct AttentionArgs {
  Cache c;
  const char* q;
  char* out;
  float* lse;
  const int32_t *table, *lengths;
  float* part;  // [batch, q_heads, chunks, head_dim] then [batch, q_heads, chunks, 2]
  long long qbs, qhs, table_stride;
  long long part_ml;  // floats before the second part
  int q_heads, group, head_blocks;
  int chunk, chunks;
  int cap, window;
  float scale_log2e;
};

// Tokens of a request: [lo, hi), and where its tiles begin (a multiple of 32).
struct Span {
  int lo, hi, first;
};
__device__ __forceinline__ Span span_of(int len, int cap, int window) {
  Span s;
  s.hi = len < 0 ? 0 : len < cap ? len : cap;
  s.lo = window > 0 && s.hi > window ? s.hi - window : 0;
  s.first = s.lo & ~31;
  return s;
}

template <int F>
struct Mma;
template <>
struct Mma<ORBIT_KV_BF16> {
  typedef __bf16 T;
  typedef bf16x8 V8;
  static __device__ __forceinline__ f32x4 run(V8 a, V8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
};
template <>
struct Mma<ORBIT_KV_F16> {
  typedef _Float16 T;
  typedef f16x8 V8;
  static __device__ __forceinline__ f32x4 run(V8 a, V8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
  }
};
template <>
struct Mma<ORBIT_KV_INT8> : Mma<ORBIT_KV_F16> {};

// Four signed bytes to four fp16 integers: 0x6400 + (byte + 128) is the fp16
// number 1024 + byte + 128.
__device__ __forceinline__ u32x2 codes_to_f16(uint32_t w) {
  typedef _Float16 h2 __attribute__((ext_vector_type(2)));
  const uint32_t x = w ^ 0x80808080u;
  const h2 off = {(_Float16)1152.0f, (_Float16)1152.0f};
  const h2 a = __builtin_bit_cast(h2, __builtin_amdgcn_perm(0x64646464u, x, 0x04010400u)) - off;
  const h2 b = __builtin_bit_cast(h2, __builtin_amdgcn_perm(0x64646464u, x, 0x04030402u)) - off;
  u32x2 r;
  r.x = __builtin_bit_cast(uint32_t, a);
  r.y = __builtin_bit_cast(uint32_t, b);
  return r;
}

typedef short s16x4 __attribute__((ext_vector_type(4)));

constexpr int kTile = 32;
constexpr int kWaves = 4;

// Workgroups per compute unit (waves per SIMD) that the kernel's registers
// allow; 0: the compiler's choice.  More spill: at 128 coordinates an int8
// cache took 165 us at two, 141 at three, 142 at four (spilling).
constexpr int residents(int format, int dp, bool paged16) {
  if (format == ORBIT_KV_INT8) return dp == 64 ? 4 : dp == 128 ? 3 : 2;
  return dp == 64 ? 4 : dp == 128 && paged16 ? 2 : 1;
}

// A wave's rows of a tile in LDS, of ROW bytes each, without padding: 16-byte
// unit u of row r lies in place u ^ key(r).  The writes (a row's units side by
// side), the operand reads (four units of 16 rows) and the transposing reads
// (two units of 16 rows) then all touch every bank equally often.
template <int ROW>
struct Stage {
  static constexpr int kBytes = kTile * ROW;
  static __device__ __forceinline__ constexpr int key(int row) {
    return ROW == 64 ? (row >> 2) & 3 : ROW == 128 ? (row >> 1) & 7 : row & 15;
  }
};

// log2 of the factor on the probabilities: 2^15 is half of fp16's range, and
// rounding of large scores (a step of 16 at 2^27) stays within the other half.
constexpr float lift_of(int format) { return format == ORBIT_KV_BF16 ? 0.0f : 15.0f; }

// Two probabilities as a hi + lo pair of 16-bit numbers.  fp16: hi is rounded
// toward zero and lo to nearest (one instruction for two each).
__device__ __forceinline__ void split2(float p0, float p1, bf16x8& hi, bf16x8& lo, int j) {
  hi[j] = (__bf16)p0;
  hi[j + 1] = (__bf16)p1;
  lo[j] = (__bf16)(p0 - (float)hi[j]);
  lo[j + 1] = (__bf16)(p1 - (float)hi[j + 1]);
}
__device__ __forceinline__ void split2(float p0, float p1, f16x8& hi, f16x8& lo, int j) {
  typedef _Float16 h2 __attribute__((ext_vector_type(2)));
  const h2 h = __builtin_bit_cast(h2, __builtin_amdgcn_cvt_pkrtz(p0, p1));
  typedef float f2 __attribute__((ext_vector_type(2)));
  const h2 l = __builtin_convertvector((f2{p0 - (float)h[0], p1 - (float)h[1]}), h2);
  hi[j] = h[0];
  hi[j + 1] = h[1];
  lo[j] = l[0];
  lo[j + 1] = l[1];
}

// A factor on sums: never zero, so that an infinite one stays infinite.
__device__ __forceinline__ float factor(float log2) { return fmaxf(__builtin_amdgcn_exp2f(log2), 1.17549435e-38f); }

// Q: the queries' format (BF16 or F16); F: the cache's; DP: head_dim rounded
// up to 64, 128 or 256; PAGED16: pages of 16 tokens or more, so that half a
// tile lies in one page and its address is the wave's (scalar registers)
// plus a lane's constant; smaller pages take an address per row.
template <int Q, int F, int DP, bool PAGED16>
__global__ __launch_bounds__(256, residents(F, DP, PAGED16)) void attend_kernel(AttentionArgs a) {
  constexpr bool kCoded = F == ORBIT_KV_INT8;
  typedef Mma<F> M;
  typedef typename M::T T;
  typedef typename M::V8 V8;
  typedef typename Mma<Q>::T QT;
  constexpr int kSteps = DP / 32;                   // products per tile half
  constexpr int kReads = kCoded ? DP / 64 : kSteps;  // 16-byte operand reads of one key per lane
  constexpr int kRowLanes = kCoded ? DP / 16 : DP / 8;  // lanes on one value row
  constexpr int kRowsAtOnce = 64 / kRowLanes;
  constexpr int kVLoads = kTile / kRowsAtOnce;
  constexpr int kBlocks = DP / 16;
  constexpr int kElem = kCoded ? 1 : 2;
  constexpr float kLift = lift_of(F);

  typedef Stage<DP * kElem> Sk;  // keys as the cache holds them
  typedef Stage<DP * 2> Sv;      // values in 16 bits
  constexpr int kStageBytes = kWaves * (Sk::kBytes + Sv::kBytes);
  constexpr int kSumBytes = kWaves * 16 * DP * 4 + kWaves * 16 * 8;
  __shared__ __align__(1024) char lds[kStageBytes > kSumBytes ? kStageBytes : kSumBytes];

  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int r16 = lane & 15, lg = lane >> 4;
  const int head = blockIdx.x / a.head_blocks, hb = blockIdx.x - head * a.head_blocks;
  const int b = blockIdx.y;
  const int dim = a.c.head_dim;
  const Span span = span_of(a.lengths[b], a.cap, a.window);
  const int c0 = span.first + (int)blockIdx.z * a.chunk;
  const int heads_here = min(16, a.group - hb * 16);
  const int h0 = head * a.group + hb * 16;  // first query head
  if (c0 >= span.hi) {
    // the first chunk of a request with nothing to see writes its zeros
    if (blockIdx.z == 0) {
      for (int i = threadIdx.x; i < heads_here * dim; i += 256)
        ((QT*)a.out)[((long long)b * a.q_heads + h0) * dim + i] = (QT)0.0f;
      if (a.lse && (int)threadIdx.x < heads_here)
        a.lse[(long long)b * a.q_heads + h0 + threadIdx.x] = -__builtin_inff();
    }
    return;
  }
  const int c1 = min(span.hi, c0 + a.chunk);
  const int32_t* const table = a.table + b * a.table_stride;

  // Queries as the B operand: lane's head r16, coordinates as the keys' loads
  // bring them (INT8: 16 codes a load are two operands' slots).
  V8 qf[kSteps];
  float zscale = a.scale_log2e;
  {
    const QT* const qrow = (const QT*)a.q + b * a.qbs + (h0 + (r16 < heads_here ? r16 : 0)) * a.qhs;
    float f[kSteps][8];
    float m = 0.0f;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const int d = kCoded ? (s >> 1) * 64 + lg * 16 + (s & 1) * 8 : s * 32 + lg * 8;
      const bool in = r16 < heads_here && d < dim;
      Vec8<QT> v;
      if (in) v = *(const Vec8<QT>*)(qrow + d);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        f[s][j] = in ? (float)v.e[j] : 0.0f;
        if (kCoded) m = fmaxf(m, fabsf(f[s][j]));
      }
    }
    if (kCoded) {
      m = max_rows32(max_rows16(m));
      // 2^-e brings the largest into [1/2, 1); an infinite one stays infinite
      const int e = m > 0.0f && m < __builtin_inff() ? __builtin_amdgcn_frexp_expf(m) : 0;
      const float down = ldexpf(1.0f, -e / 2), down2 = ldexpf(1.0f, -e - (-e / 2));
      zscale = ldexpf(zscale, e);
#pragma unroll
      for (int s = 0; s < kSteps; ++s)
#pragma unroll
        for (int j = 0; j < 8; ++j) f[s][j] = f[s][j] * down * down2;
    }
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
#pragma unroll
      for (int j = 0; j < 8; ++j) qf[s][j] = (T)f[s][j];
  }

  // Loads are unconditional, so that none waits for another: tokens that are
  // not seen read page 0 (or the rest of their own page), coordinates past
  // head_dim the row's last vector again.  Scores of the former are masked and
  // their values cleared.  The latter are results that are not stored (values)
  // or meet zeros of the queries (keys: codes are finite, 16-bit ones are
  // cleared, as an infinite one times zero would be NaN).
  u32x4 kr[kVLoads], vr[kVLoads];
  u32x2 ksr[2], vsr[2];
  const int row_bytes = dim * kElem;
  const uint32_t page_bytes = (uint32_t)row_bytes << a.c.page_shift;  // of one head
  const int vcol = min((lane & (kRowLanes - 1)) * 16, row_bytes - 16);
  const int voff = (PAGED16 ? lane / kRowLanes * row_bytes : 0) + vcol;

  // The pages of a tile and which of its tokens are seen (bit t: token t).
  struct Pages {
    uint32_t page[PAGED16 ? 2 : 1];  // of each half; or of token (lane & 31)
    uint32_t live;
  };
  auto look_up = [&](int tile) {
    Pages p;
    p.live = 0;
    p.page[0] = 0;
    if constexpr (PAGED16) {
      p.page[1] = 0;
      if (tile < c1) {
        uint32_t live = 0xffffffffu;
        if (tile < span.lo) live <<= span.lo - tile;
        if (tile + 32 > c1) live &= (1u << (c1 - tile)) - 1u;
        p.page[0] = __builtin_amdgcn_readfirstlane((uint32_t)table[tile >> a.c.page_shift]);
        p.page[1] = tile + 16 < c1 ? __builtin_amdgcn_readfirstlane((uint32_t)table[(tile + 16) >> a.c.page_shift]) : 0u;
        if (p.page[0] >= a.c.pages) {
          live &= 0xffff0000u;
          p.page[0] = 0;
        }
        if (p.page[1] >= a.c.pages) {
          live &= 0xffffu;
          p.page[1] = 0;
        }
        p.live = live;
      }
    } else {
      const int t = tile + (lane & 31);
      uint32_t page = 0xffffffffu;
      if (t >= span.lo && t < c1) page = (uint32_t)table[t >> a.c.page_shift];
      p.live = (uint32_t)__ballot(page < a.c.pages);
      p.page[0] = page < a.c.pages ? page : 0u;
    }
    return p;
  };
  // The first byte of a head's part of a page, of its scales.
  auto head_of = [&](uint32_t page) { return ((uint64_t)page * a.c.kv_heads + head) * page_bytes; };
  auto load_rows = [&](u32x4 (&to)[kVLoads], const char* base, int tile, const Pages& p) {
#pragma unroll
    for (int i = 0; i < kVLoads; ++i) {
      if constexpr (PAGED16) {
        const int half = i * 2 / kVLoads;
        const uint32_t off = ((uint32_t)(tile + half * 16) & a.c.page_mask) + (i - half * (kVLoads / 2)) * kRowsAtOnce;
        to[i] = *(const u32x4*)(base + head_of(p.page[half]) + off * (uint32_t)row_bytes + voff);
      } else {
        const int t = i * kRowsAtOnce + lane / kRowLanes;
        const uint32_t page = (uint32_t)__shfl((int)p.page[0], t);
        to[i] = *(const u32x4*)(base + head_of(page) + ((uint32_t)(tile + t) & a.c.page_mask) * (uint32_t)row_bytes + voff);
      }
    }
  };
  auto load_keys = [&](int tile, const Pages& p) {
    load_rows(kr, a.c.k, tile, p);
    if constexpr (kCoded) {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        // four neighbouring tokens lie in one page (page_size >= 4), whose
        // number the first that is seen has
        const int t4 = half * 16 + lg * 4;
        uint32_t page;
        if constexpr (PAGED16) {
          page = p.page[half];
        } else {
          const uint32_t four = (p.live >> t4) & 15u;
          page = (uint32_t)__shfl((int)p.page[0], t4 + (four ? __builtin_ctz(four) : 0));
        }
        const uint64_t row = (((uint64_t)page * a.c.kv_heads + head) << a.c.page_shift) + ((uint32_t)(tile + t4) & a.c.page_mask);
        ksr[half] = *(const u32x2*)(a.c.ks + row);
        vsr[half] = *(const u32x2*)(a.c.vs + row);
      }
    }
  };
  auto load_values = [&](int tile, const Pages& p) { load_rows(vr, a.c.v, tile, p); };

  f32x4 o[kBlocks];
#pragma unroll
  for (int d = 0; d < kBlocks; ++d) o[d] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  float m_run = -__builtin_inff(), l_run = 0.0f;  // l: this lane's tokens alone
  char* const kstage = lds + wave * Sk::kBytes;
  char* const vstage = lds + kWaves * Sk::kBytes + wave * Sv::kBytes;
  // Where this lane writes its first vectors (others: constants further, the
  // keys' constant bits exchanged), and where it reads its first operands.
  const int lrow = lane / kRowLanes, lcol = lane & (kRowLanes - 1);
  const int kwrite = lrow * DP * kElem + ((lcol ^ Sk::key(lrow)) << 4);
  const int vwrite = lrow * DP * 2 + ((lcol * (kCoded ? 2 : 1) ^ Sv::key(lrow)) << 4);
  const int kread = r16 * DP * kElem + ((lg ^ Sk::key(r16)) << 4);  // row r16 + 16 has the same key
  const int trow = lg * 4 + (r16 >> 2);
  const int vread = trow * DP * 2 + ((((r16 & 3) >> 1) ^ Sv::key(trow)) << 4) + (r16 & 1) * 8;
  auto order = [] {  // between writes and reads of the wave's rows by other lanes (LDS serves a wave in order)
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  };

  int tile = c0 + wave * kTile;
  if (tile < c1) {
    constexpr int kStep = kWaves * kTile;
    Pages now = look_up(tile);
    load_keys(tile, now);
    load_values(tile, now);
    Pages next = look_up(tile + kStep);
    for (; tile < c1; tile += kStep) {
      const uint32_t live = now.live;
      // scores of the tile
      if (!kCoded && dim < DP) {
#pragma unroll
        for (int i = 0; i < kVLoads; ++i) kr[i] = lcol * 8 < dim ? kr[i] : u32x4{0u, 0u, 0u, 0u};
      }
#pragma unroll
      for (int i = 0; i < kVLoads; ++i)
        *(u32x4*)(kstage + i * kRowsAtOnce * DP * kElem + (kwrite ^ (Sk::key(i * kRowsAtOnce) << 4))) = kr[i];
      order();
      f32x4 s[2] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};
#pragma unroll
      for (int half = 0; half < 2; ++half)
#pragma unroll
        for (int i = 0; i < kReads; ++i) {
          const u32x4 k = *(const u32x4*)(kstage + half * 16 * DP * kElem + (kread ^ (i << 6)));
          if constexpr (kCoded) {
            union {
              u32x2 w[4];
              V8 v[2];
            } u;
#pragma unroll
            for (int c = 0; c < 4; ++c) u.w[c] = codes_to_f16(k[c]);
            s[half] = M::run(u.v[0], qf[2 * i], s[half]);
            s[half] = M::run(u.v[1], qf[2 * i + 1], s[half]);
          } else {
            s[half] = M::run(__builtin_bit_cast(V8, k), qf[i], s[half]);
          }
        }
      order();
      float z[8], vs[8];
#pragma unroll
      for (int half = 0; half < 2; ++half)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          z[half * 4 + i] = s[half][i] * zscale;
          if constexpr (kCoded) {
            typedef _Float16 h4 __attribute__((ext_vector_type(4)));
            z[half * 4 + i] *= (float)__builtin_bit_cast(h4, ksr[half])[i];
            vs[half * 4 + i] = (float)__builtin_bit_cast(h4, vsr[half])[i];
          }
        }
      if (live != 0xffffffffu) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const bool seen = (live >> ((j >> 2) * 16 + lg * 4 + (j & 3))) & 1u;
          z[j] = seen ? z[j] : -__builtin_inff();
          if constexpr (kCoded) vs[j] = seen ? vs[j] : 0.0f;
        }
      }
      // past the end page 0 is read, and never used
      now = next;
      load_keys(tile + kStep, now);
      next = look_up(tile + 2 * kStep);

      // running maximum (of z + log2(scale) where values carry one) and sums
      float mt = -__builtin_inff();
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if constexpr (kCoded) mt = fmaxf(mt, z[j] + __builtin_amdgcn_logf(fmaxf(vs[j], 5.9604645e-8f)));
        else mt = fmaxf(mt, z[j]);
      }
      mt = max_rows32(max_rows16(mt));
      if (__any(mt > m_run)) {
        const float m_new = fmaxf(m_run, mt);
        const float alpha = factor(m_run - (m_new == -__builtin_inff() ? 0.0f : m_new));
        m_run = m_new;
        l_run *= alpha;
#pragma unroll
        for (int d = 0; d < kBlocks; ++d) o[d] *= alpha;
      }
      const float m_use = m_run == -__builtin_inff() ? 0.0f : m_run - kLift;
      V8 hi, lo;
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        float p0 = __builtin_amdgcn_exp2f(z[j] - m_use), p1 = __builtin_amdgcn_exp2f(z[j + 1] - m_use);
        l_run += p0 + p1;
        if constexpr (kCoded) {
          p0 *= vs[j];
          p1 *= vs[j + 1];
        }
        split2(p0, p1, hi, lo, j);
      }

      // values to the wave's rows (LDS serves one wave's accesses in order)
      if (live != 0xffffffffu) {
#pragma unroll
        for (int i = 0; i < kVLoads; ++i)
          vr[i] = (live >> (i * kRowsAtOnce + lane / kRowLanes)) & 1u ? vr[i] : u32x4{0u, 0u, 0u, 0u};
      }
#pragma unroll
      for (int i = 0; i < kVLoads; ++i) {
        if constexpr (kCoded) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const u32x2 x = codes_to_f16(vr[i][2 * c]), y = codes_to_f16(vr[i][2 * c + 1]);
            *(u32x4*)(vstage + i * kRowsAtOnce * DP * 2 + (vwrite ^ ((Sv::key(i * kRowsAtOnce) ^ c) << 4))) =
                u32x4{x.x, x.y, y.x, y.y};
          }
        } else {
          *(u32x4*)(vstage + i * kRowsAtOnce * DP * 2 + (vwrite ^ (Sv::key(i * kRowsAtOnce) << 4))) = vr[i];
        }
      }
      order();
      load_values(tile + kStep, now);
      {
        typedef __attribute__((address_space(3))) s16x4* lds_ptr;
#pragma unroll
        for (int d = 0; d < kBlocks; ++d) {
          union {
            s16x4 h[2];
            V8 v;
          } u;
          // units 2 d and 2 d + 1; rows 16 apart have the same key
          const char* const at = vstage + (vread ^ (d << 5));
          u.h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)at);
          u.h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(at + 16 * DP * 2));
          o[d] = M::run(u.v, hi, o[d]);
          o[d] = M::run(u.v, lo, o[d]);
        }
      }
      order();
    }
  }
  if constexpr (!kCoded) {
    f32x4 all = o[0];
#pragma unroll
    for (int d = 1; d < kBlocks; ++d) all += o[d];
    const float one = (all[0] + all[1]) + (all[2] + all[3]);
    if (__any(one != one)) {  // a NaN, or infinities of both signs
      uint64_t lost = 0;      // bit 4 d + i: sum i of block d is NaN
#pragma unroll
      for (int d = 0; d < kBlocks; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i) lost |= (uint64_t)(o[d][i] != o[d][i]) << (4 * d + i);
      // Such a sum again, of the infinite (and NaN) values alone: each by 1 if
      // its token has a weight, by 0 at a score of minus infinity, by NaN at
      // one that is infinite or NaN.
#pragma unroll
      for (int d = 0; d < kBlocks; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[d][i] = (lost >> (4 * d + i)) & 1u ? 0.0f : o[d][i];
#pragma unroll 1
      for (int from = c0 + wave * kTile; from < c1; from += kWaves * kTile)
#pragma unroll 1
        for (int t = max(from, span.lo); t < min(from + kTile, c1); ++t) {
          const uint32_t page = (uint32_t)table[t >> a.c.page_shift];
          if (page >= a.c.pages) continue;
          const long long at = cache_row(a.c, page, head, (uint32_t)t & a.c.page_mask) * dim;
          float z = 0.0f;
#pragma unroll
          for (int s = 0; s < kSteps; ++s) {
            if (s * 32 + lg * 8 >= dim) continue;
            const Vec8<T> k = *(const Vec8<T>*)((const T*)a.c.k + at + s * 32 + lg * 8);
#pragma unroll
            for (int j = 0; j < 8; ++j) z = fmaf((float)qf[s][j], (float)k.e[j], z);
          }
          z = add_rows32(add_rows16(z)) * zscale;
          const float w = z == -__builtin_inff() ? 0.0f : z < __builtin_inff() ? 1.0f : __builtin_nanf("");
#pragma unroll
          for (int d = 0; d < kBlocks; ++d) {
            if (d * 16 + lg * 4 >= dim) continue;
            T v[4];
            __builtin_memcpy(v, (const T*)a.c.v + at + d * 16 + lg * 4, sizeof v);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float x = fabsf((float)v[i]) < __builtin_inff() ? 0.0f : (float)v[i];
              o[d][i] = (lost >> (4 * d + i)) & 1u ? fmaf(w, x, o[d][i]) : o[d][i];
            }
          }
        }
      // none of them: the NaN has another cause, and stays
#pragma unroll
      for (int d = 0; d < kBlocks; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[d][i] = (lost >> (4 * d + i)) & 1u && o[d][i] == 0.0f ? __builtin_nanf("") : o[d][i];
    }
  }
  l_run = add_rows32(add_rows16(l_run));

  // the four waves' sums meet; from here on the maximum stands for the lifted
  // one, that the sums are relative to
  m_run -= kLift;
  __syncthreads();
  float* const so = (float*)lds;                     // [wave][head][DP]
  float* const sm = (float*)(lds + kWaves * 16 * DP * 4);  // [wave][head], then the sums
  if (lg == 0) {
    sm[wave * 16 + r16] = m_run;
    sm[kWaves * 16 + wave * 16 + r16] = l_run;
  }
#pragma unroll
  for (int d = 0; d < kBlocks; ++d) *(f32x4*)(so + (wave * 16 + r16) * DP + d * 16 + lg * 4) = o[d];
  __syncthreads();
  const bool last = a.chunks == 1;
  for (int i = threadIdx.x; i < heads_here * (DP / 8); i += 256) {
    const int h = i / (DP / 8), d = (i - h * (DP / 8)) * 8;
    if (d >= dim) continue;
    float m = sm[h];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) m = fmaxf(m, sm[w * 16 + h]);
    const float m_use = m == -__builtin_inff() ? 0.0f : m;
    float l = 0.0f, f[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      const float e = factor(sm[w * 16 + h] - m_use);
      l = fmaf(e, sm[kWaves * 16 + w * 16 + h], l);
      const f32x4 x = *(const f32x4*)(so + (w * 16 + h) * DP + d), y = *(const f32x4*)(so + (w * 16 + h) * DP + d + 4);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        f[j] = fmaf(e, x[j], f[j]);
        f[4 + j] = fmaf(e, y[j], f[4 + j]);
      }
    }
    const long long bh = (long long)b * a.q_heads + h0 + h;
    if (last) {
      const float inv = l == 0.0f ? 0.0f : 1.0f / l;
      Vec8<QT> v;
#pragma unroll
      for (int j = 0; j < 8; ++j) v.e[j] = (QT)(l == 0.0f ? 0.0f : f[j] * inv);
      *(Vec8<QT>*)((QT*)a.out + bh * dim + d) = v;
      if (a.lse && d == 0) a.lse[bh] = (m + __builtin_amdgcn_logf(l)) * 0.69314718056f;
    } else {
      const long long at = bh * a.chunks + blockIdx.z;
      f32x4* const to = (f32x4*)(a.part + at * dim + d);
      to[0] = f32x4{f[0], f[1], f[2], f[3]};
      to[1] = f32x4{f[4], f[5], f[6], f[7]};
      if (d == 0) *(float2*)(a.part + a.part_ml + at * 2) = make_float2(m, l);
    }
  }
}

// Joins the chunks of one query head: a workgroup per (request, head), its
// groups of dim / 4 lanes taking every n-th chunk.
template <class QT>
__global__ __launch_bounds__(256) void join_kernel(AttentionArgs a) {
  __shared__ f32x4 so[256];
  __shared__ float sl[256];
  const int b = blockIdx.y, h = blockIdx.x;
  const Span span = span_of(a.lengths[b], a.cap, a.window);
  if (span.hi <= span.first) return;  // nothing to see: written already
  const int n = (span.hi - span.first + a.chunk - 1) / a.chunk;
  const long long bh = (long long)b * a.q_heads + h;
  const int dim = a.c.head_dim, lanes = dim >> 2;
  const int groups = 256 / lanes;
  const int g = threadIdx.x / lanes, t = threadIdx.x - g * lanes;
  const float2* const ml = (const float2*)(a.part + a.part_ml) + bh * a.chunks;
  float m = -__builtin_inff();
  for (int c = threadIdx.x & 63; c < n; c += 64) m = fmaxf(m, ml[c].x);
  m = dpp_max<kXor1>(m);
  m = dpp_max<kXor2>(m);
  m = dpp_max<kHalfMirror>(m);
  m = dpp_max<kRowMirror>(m);
  m = max_rows32(max_rows16(m));
  const float m_use = m == -__builtin_inff() ? 0.0f : m;
  f32x4 o = {0.0f, 0.0f, 0.0f, 0.0f};
  float l = 0.0f;
  if (g < groups) {
    const f32x4* const part = (const f32x4*)(a.part + bh * a.chunks * dim) + t;
#pragma unroll 4
    for (int c = g; c < n; c += groups) {
      const float2 x = ml[c];
      const float e = factor(x.x - m_use);
      const f32x4 v = part[(long long)c * lanes];
      l = fmaf(e, x.y, l);
#pragma unroll
      for (int j = 0; j < 4; ++j) o[j] = fmaf(e, v[j], o[j]);
    }
  }
  so[threadIdx.x] = o;
  sl[threadIdx.x] = l;
  __syncthreads();
  if (g != 0) return;
  const int used = groups < n ? groups : n;
  for (int i = 1; i < used; ++i) {
    o += so[i * lanes + t];
    l += sl[i * lanes + t];
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  struct alignas(8) {
    QT e[4];
  } v;
#pragma unroll
  for (int j = 0; j < 4; ++j) v.e[j] = (QT)(l == 0.0f ? 0.0f : o[j] * inv);
  *(decltype(v)*)((QT*)a.out + bh * dim + t * 4) = v;
  if (a.lse && t == 0) a.lse[bh] = (m + __builtin_amdgcn_logf(l)) * 0.69314718056f;
}

template <int Q, int F>
hipError_t launch_attend(const AttentionArgs& a, dim3 grid, hipStream_t stream) {
  const int dim = a.c.head_dim;
  if (a.c.page_shift >= 4) {
    if (dim <= 64) attend_kernel<Q, F, 64, true><<<grid, dim3(256), 0, stream>>>(a);
    else if (dim <= 128) attend_kernel<Q, F, 128, true><<<grid, dim3(256), 0, stream>>>(a);
    else attend_kernel<Q, F, 256, true><<<grid, dim3(256), 0, stream>>>(a);
  } else {
    if (dim <= 64) attend_kernel<Q, F, 64, false><<<grid, dim3(256), 0, stream>>>(a);
    else if (dim <= 128) attend_kernel<Q, F, 128, false><<<grid, dim3(256), 0, stream>>>(a);
    else attend_kernel<Q, F, 256, false><<<grid, dim3(256), 0, stream>>>(a);
  }
  return hipGetLastError();
}

hipError_t launch_attend_coded(const AttentionArgs& a, int q_dtype, dim3 grid, hipStream_t stream);

}  // namespace block
}  // namespace orbit
