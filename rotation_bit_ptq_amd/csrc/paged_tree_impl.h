// Attention of several new tokens per request over the paged cache
// (orbit_tree_attention): a tree of drafted tokens, a run (a prompt or a piece
// of one), or one token each behind a window with sinks:
//   o = sum_t p_t v_t / sum_t p_t,  p_t = exp(sm_scale q . k_t - m),
// over the tokens t that a new token sees, the maximum m and the sums carried
// along the tokens (one pass over the cache).
//
// Rows.  The new tokens of a request and the query heads of one key head are
// the rows r = token * group + head of one product with its keys.  A workgroup
// of eight waves takes 16 RB WR rows and a piece of the context: WR waves side
// by side on the rows (16 RB each), WT on the tokens.  Tiles of TILE tokens
// are loaded by all waves: into registers while the tile before is multiplied,
// then, converted to 16 bits where the cache holds codes, to LDS, from where
// every wave reads what it needs.  So a tile is read from memory once for all
// its rows, and a tile is in flight all the time.
//
// Products as in the single-token kernel (paged_attention_impl.h): S^T = K Q^T
// with the keys as A operand; O^T = V^T P^T with the probabilities in the
// lanes that computed them, as pairs of 16-bit numbers; V^T by transposing LDS
// reads.  A lane holds row l % 16 of its block and tokens 4 (l / 16) + i of
// each half of 32 tokens.
//
// What a row sees: prefix tokens in [lo, hi) and below `sinks`, and new tokens
// by the bits of its mask.  A wave whose rows all see all 32 tokens skips the
// masks.
//
// A product of a hidden token's weight, 0, with a value that is infinite or
// NaN is NaN, and so is an infinite value's with half of a pair that is zero.
// A wave whose sums are NaN therefore sums those coordinates once more, over
// the seen tokens alone and with unsplit weights, outside the loop.
#pragma once

#include "paged_attention_impl.h"

namespace orbit {
namespace block {

struct TreeArgs {
  Cache c;
  const char* q;
  char* out;
  float* lse;
  const int32_t *table, *lengths, *starts;
  const uint64_t* tree;
  float* part;  // [rows, pieces, head_dim], then [rows, pieces, 2], then the pieces in use [rows]; row = token * q_heads + head
  long long qts, qhs, table_stride;
  long long part_ml, part_n;  // floats before the second and the third
  int tokens, batch, q_heads, group;
  int words;      // of a token's mask; 0: a run
  int rows, wr;   // rows of a workgroup, waves on them
  int pieces, slots;
  int cap, window, sinks;
  float scale_log2e;
};

// Rows [begin, end) of a request and how they lie in its context.
struct Request {
  int b, begin, n;  // first row of q, new tokens
  int len, base;    // tokens in the context, and before the new ones (negative: more new tokens than context)
};
// Work slots: request b has those from floor(starts[b] group / rows) + b on,
// at least as many as it has row tiles, so that which request a slot belongs
// to is found without knowing the others' sizes.  Without starts each request
// has one new token.
__device__ __forceinline__ int start_of(const TreeArgs& a, int b) {
  if (!a.starts) return b;
  const int s = a.starts[b];
  return s < 0 ? 0 : s < a.tokens ? s : a.tokens;
}
__device__ __forceinline__ int first_slot(const TreeArgs& a, int b) {
  if (!a.starts) return b * ((a.group + a.rows - 1) / a.rows);
  return (int)((long long)start_of(a, b) * a.group / a.rows) + b;
}
// The last request whose first slot is not behind `slot`: the wave's lanes try
// 64 at a time.
__device__ __forceinline__ int request_at(const TreeArgs& a, int slot, int lane) {
  if (!a.starts) return slot / ((a.group + a.rows - 1) / a.rows);
  int lo = 0, span = a.batch;
  while (span > 1) {
    const int step = (span + 63) >> 6, at = lane * step;
    const int n = __popcll(__ballot(at < span && first_slot(a, lo + min(at, span - 1)) <= slot));
    const int skip = max(n - 1, 0) * step;
    lo += skip;
    span = min(step, span - skip);
  }
  return __builtin_amdgcn_readfirstlane(lo);
}
__device__ __forceinline__ Request request_of(const TreeArgs& a, int b) {
  Request r;
  r.b = b;
  r.begin = start_of(a, b);
  r.n = max(start_of(a, b + 1) - r.begin, 0);
  const int len = a.lengths[b];
  r.len = len < 0 ? 0 : len < a.cap ? len : a.cap;
  r.base = r.len - r.n;
  return r;
}

// The bits of tokens [from, to) among 32 from `tile` on.
__device__ __forceinline__ uint32_t range32(int from, int to, int tile) {
  const int x = min(max(from - tile, 0), 32), y = min(max(to - tile, 0), 32);
  const uint32_t below_y = y == 32 ? 0xffffffffu : (1u << y) - 1u, below_x = x == 32 ? 0xffffffffu : (1u << x) - 1u;
  return below_y & ~below_x;
}
// Bits j .. j + 31 of a mask of `words` words; j may be negative.
__device__ __forceinline__ uint32_t bits32(const uint64_t* mask, int words, int j) {
  const int w = j >> 6, sh = j & 63;
  const uint64_t lo = w >= 0 && w < words ? mask[w] : 0, hi = w + 1 >= 0 && w + 1 < words ? mask[w + 1] : 0;
  return (uint32_t)(sh ? (lo >> sh) | (hi << (64 - sh)) : lo);
}

constexpr int kTreeWaves = 8;
constexpr int tree_tile(int dp) { return dp == 256 ? 64 : 128; }
constexpr int tree_lds(int dp) { return 2 * tree_tile(dp) * dp * 2 + tree_tile(dp) * 12 + 16; }

// Q: the queries' format; F: the cache's; DP: head_dim rounded up to 64, 128
// or 256; RB: blocks of 16 rows per wave.
template <int Q, int F, int DP, int RB>
__global__ __launch_bounds__(64 * kTreeWaves, RB == 1 && DP == 64 ? 4 : 2) void tree_kernel(TreeArgs a) {
  constexpr bool kCoded = F == ORBIT_KV_INT8;
  typedef Mma<F> M;
  typedef typename M::T T;
  typedef typename M::V8 V8;
  typedef typename Mma<Q>::T QT;
  constexpr int kThreads = 64 * kTreeWaves, kTokens = tree_tile(DP), kSubs = kTokens / 32;
  constexpr int kSteps = DP / 32, kBlocks = DP / 16;
  constexpr int kElem = kCoded ? 1 : 2;
  constexpr int kRowLanes = DP * kElem / 16, kRowsAtOnce = kThreads / kRowLanes, kLoads = kTokens / kRowsAtOnce;
  static_assert(kLoads >= 1 && kTokens % kRowsAtOnce == 0, "whole rows per load");
  constexpr float kLift = lift_of(F);
  typedef Stage<DP * 2> St;
  constexpr int kStageBytes = kTokens * DP * 2;
  extern __shared__ __align__(1024) char lds[];
  char* const kstage = lds;
  char* const vstage = lds + kStageBytes;
  float* const kscale = (float*)(lds + 2 * kStageBytes);  // INT8: of each token
  float* const vscale = kscale + kTokens;
  uint32_t* const gone = (uint32_t*)(vscale + kTokens);  // tokens whose page is outside the cache: 1
  uint32_t* const any_gone = gone + kTokens;             // [2]: whether the tile has such tokens, by the tile's parity

  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r16 = lane & 15, lg = lane >> 4;
  const int dim = a.c.head_dim;
  // neighbouring workgroups take the key heads of one slot; the last slots
  // come first, as in a prompt they have the longest contexts
  const int order = (int)blockIdx.x / a.c.kv_heads, head = (int)blockIdx.x - order * a.c.kv_heads;
  const int slot = a.slots - 1 - order;
  const int b = request_at(a, slot, lane);
  if (b >= a.batch) return;
  const Request rq = request_of(a, b);
  const int row0 = (slot - first_slot(a, b)) * a.rows, all_rows = rq.n * a.group;
  if (row0 < 0 || row0 >= all_rows) return;
  const int rows_here = min(a.rows, all_rows - row0);

  // the tiles of TILE tokens that any of the rows sees part of: those of the
  // sinks, then those from the earliest window's first token on
  const int i_first = row0 / a.group, i_last = (row0 + rows_here - 1) / a.group;
  const int hi_all = a.words ? rq.len : max(rq.base + i_last + 1, 0);
  const int p_least = a.words ? rq.base - 1 : rq.base + i_first;
  const int lo_all = a.window ? max(p_least - a.window + 1, 0) : 0;
  const int end_tile = (hi_all + kTokens - 1) / kTokens;
  const int sink_tiles = a.window ? min((min(a.sinks, hi_all) + kTokens - 1) / kTokens, end_tile) : 0;
  const int first_tile = max(sink_tiles, lo_all / kTokens);
  const int tiles = sink_tiles + max(end_tile - first_tile, 0);
  const int per = max((tiles + a.pieces - 1) / a.pieces, 1), used = (tiles + per - 1) / per;
  const int k0 = (int)blockIdx.y * per, k1 = min(tiles, k0 + per);
  const bool last = used <= 1;  // nothing to join
  if (k0 >= k1 && blockIdx.y > 0) return;

  const int wt_all = kTreeWaves / a.wr < kSubs ? kTreeWaves / a.wr : kSubs;  // waves on the tokens
  const int wr = wave % a.wr, wt = wave / a.wr;
  const bool works = wt < wt_all && wr * 16 * RB < rows_here;

  // this lane's rows
  int lo[RB], hi[RB], token[RB], qhead[RB];
  int lo_max = 0, hi_min = 0x7fffffff;
#pragma unroll
  for (int rb = 0; rb < RB; ++rb) {
    const int r = row0 + (wr * RB + rb) * 16 + r16;
    const bool in = (wr * RB + rb) * 16 + r16 < rows_here;
    const int i = (in ? r : row0) / a.group;
    token[rb] = in ? rq.begin + i : -1;
    qhead[rb] = head * a.group + (in ? r : row0) - i * a.group;
    int p = rq.base + i;
    hi[rb] = p + 1;
    if (a.words) {
      hi[rb] = rq.base;
      if (a.window) {
        int seen = 0;
        const uint64_t* const mask = a.tree + (long long)(rq.begin + i) * a.words;
        for (int w = 0; w < a.words && w * 64 < rq.n; ++w) {
          const int left = rq.n - w * 64;
          seen += __popcll(left >= 64 ? mask[w] : mask[w] & ((1ull << left) - 1));
        }
        p = rq.base + seen - 1;
      }
    }
    lo[rb] = a.window ? max(p - a.window + 1, 0) : 0;
    if (in) {
      lo_max = max(lo_max, lo[rb]);
      hi_min = min(hi_min, hi[rb]);
    }
  }
#pragma unroll
  for (int s = 1; s < 16; s *= 2) {
    lo_max = max(lo_max, __shfl_xor(lo_max, s));
    hi_min = min(hi_min, __shfl_xor(hi_min, s));
  }
  lo_max = __builtin_amdgcn_readfirstlane(lo_max);
  hi_min = __builtin_amdgcn_readfirstlane(hi_min);

  // the bits of the tokens among 32 from t0 on that this lane's row rb sees
  auto seen32 = [&](int rb, int t0) {
    uint32_t m = range32(lo[rb], hi[rb], t0);
    if (a.window) m |= range32(0, min(a.sinks, hi[rb]), t0);
    if (a.words && t0 + 32 > rq.base && token[rb] >= 0)
      m |= bits32(a.tree + (long long)token[rb] * a.words, a.words, t0 - rq.base) & range32(max(rq.base, 0), rq.len, t0);
    return m;
  };

  // queries as the B operand
  V8 qf[RB][kSteps];
  float zscale[RB];
#pragma unroll
  for (int rb = 0; rb < RB; ++rb) {
    const QT* const qrow = (const QT*)a.q + (long long)max(token[rb], 0) * a.qts + qhead[rb] * a.qhs;
    float f[kSteps][8], m = 0.0f;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const int d = s * 32 + lg * 8;
      const bool in = token[rb] >= 0 && d < dim;
      Vec8<QT> v;
      if (in) v = *(const Vec8<QT>*)(qrow + d);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        f[s][j] = in ? (float)v.e[j] : 0.0f;
        if (kCoded) m = fmaxf(m, fabsf(f[s][j]));
      }
    }
    zscale[rb] = a.scale_log2e;
    if (kCoded) {  // into fp16's range by a power of two per row
      m = max_rows32(max_rows16(m));
      const int e = m > 0.0f && m < __builtin_inff() ? __builtin_amdgcn_frexp_expf(m) : 0;
      const float down = ldexpf(1.0f, -e / 2), down2 = ldexpf(1.0f, -e - (-e / 2));
      zscale[rb] = ldexpf(zscale[rb], e);
#pragma unroll
      for (int s = 0; s < kSteps; ++s)
#pragma unroll
        for (int j = 0; j < 8; ++j) f[s][j] = f[s][j] * down * down2;
    }
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
#pragma unroll
      for (int j = 0; j < 8; ++j) qf[rb][s][j] = (T)f[s][j];
  }

  // Loading.  This thread's rows of a tile are lrow + i * kRowsAtOnce, 16
  // bytes at unit lcol of each.  Tokens from hi_all on, and those whose page
  // lies outside the cache, are zeros.
  const int lrow = tid / kRowLanes, lcol = tid & (kRowLanes - 1);
  const int row_bytes = dim * kElem;
  const bool col_in = lcol * 16 < row_bytes;
  const int32_t* const table = a.table + b * a.table_stride;
  auto tile_at = [&](int k) { return (k < sink_tiles ? k : first_tile + k - sink_tiles) * kTokens; };
  u32x4 kr[kLoads], vr[kLoads];
  _Float16 ksr[kLoads], vsr[kLoads];
  uint32_t page[kLoads];  // of the next tile's rows; 0xffffffff: nothing to read
  auto look_up = [&](int k) {
    const int t0 = tile_at(k) + lrow;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int t = t0 + i * kRowsAtOnce;
      page[i] = k < k1 && t < hi_all ? (uint32_t)table[t >> a.c.page_shift] : 0xffffffffu;
    }
  };
  uint32_t absent;  // bit i: row i was not read
  auto load = [&](int k) {
    const int t0 = tile_at(k) + lrow;
    absent = 0;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int t = t0 + i * kRowsAtOnce;
      const bool there = page[i] < a.c.pages;
      absent |= (uint32_t)!there << i;
      const long long row = there ? cache_row(a.c, page[i], head, (uint32_t)t & a.c.page_mask) : 0;
      const long long at = row * row_bytes + (col_in ? lcol * 16 : 0);
      kr[i] = *(const u32x4*)(a.c.k + at);
      vr[i] = *(const u32x4*)(a.c.v + at);
      if constexpr (kCoded) {
        ksr[i] = a.c.ks[row];
        vsr[i] = a.c.vs[row];
      }
    }
  };
  auto store = [&](int k) {
    const int t0 = tile_at(k) + lrow;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int r = lrow + i * kRowsAtOnce;
      const bool keep = !((absent >> i) & 1u) && col_in;
      const u32x4 zero = {0u, 0u, 0u, 0u};
      const u32x4 k4 = keep ? kr[i] : zero, v4 = keep ? vr[i] : zero;
      const int key = St::key(r & 15);
      if constexpr (kCoded) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const u32x2 x = codes_to_f16(k4[2 * c]), y = codes_to_f16(k4[2 * c + 1]);
          const u32x2 z = codes_to_f16(v4[2 * c]), w = codes_to_f16(v4[2 * c + 1]);
          const int at = r * DP * 2 + (((lcol * 2 + c) ^ key) << 4);
          *(u32x4*)(kstage + at) = u32x4{x.x, x.y, y.x, y.y};
          *(u32x4*)(vstage + at) = u32x4{z.x, z.y, w.x, w.y};
        }
      } else {
        const int at = r * DP * 2 + ((lcol ^ key) << 4);
        *(u32x4*)(kstage + at) = k4;
        *(u32x4*)(vstage + at) = v4;
      }
      if (lcol == 0) {
        const bool out = (absent >> i) & 1u;
        if constexpr (kCoded) {
          kscale[r] = out ? 0.0f : (float)ksr[i];
          vscale[r] = out ? 0.0f : (float)vsr[i];
        }
        gone[r] = out;
        if (out && t0 + i * kRowsAtOnce < hi_all) any_gone[k & 1] = 1;
      }
    }
  };

  f32x4 o[RB][kBlocks];
  float m_run[RB], l_run[RB];  // l: this lane's tokens alone
#pragma unroll
  for (int rb = 0; rb < RB; ++rb) {
    m_run[rb] = -__builtin_inff();
    l_run[rb] = 0.0f;
#pragma unroll
    for (int d = 0; d < kBlocks; ++d) o[rb][d] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  }
  const int kread = r16 * DP * 2 + ((lg ^ St::key(r16)) << 4);
  const int trow = lg * 4 + (r16 >> 2);
  const int vread = trow * DP * 2 + ((((r16 & 3) >> 1) ^ St::key(trow)) << 4) + (r16 & 1) * 8;

  if (tid < 2) any_gone[tid] = 0;
  if (k0 < k1) {
    look_up(k0);
    load(k0);
    look_up(k0 + 1);
  }
  for (int k = k0; k < k1; ++k) {
    __syncthreads();  // the tile before has been read
    store(k);
    __syncthreads();
    if (tid == 0) any_gone[(k + 1) & 1] = 0;
    if (k + 1 < k1) {
      load(k + 1);
      look_up(k + 2);
    }
    if (!works) continue;
    const int t0 = tile_at(k);
    const bool holes = any_gone[k & 1] != 0;
#pragma unroll 1
    for (int sub = wt; sub < kSubs; sub += wt_all) {
      const int ts = t0 + sub * 32;
      if (ts >= hi_all) break;
      const char* const ks = kstage + sub * 32 * DP * 2;
      const char* const vs = vstage + sub * 32 * DP * 2;
      f32x4 s[RB][2];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
#pragma unroll
        for (int rb = 0; rb < RB; ++rb) s[rb][half] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
          const V8 kv = __builtin_bit_cast(V8, *(const u32x4*)(ks + half * 16 * DP * 2 + (kread ^ (i << 6))));
#pragma unroll
          for (int rb = 0; rb < RB; ++rb) s[rb][half] = M::run(kv, qf[rb][i], s[rb][half]);
        }
      }
      float kt[8], vt[8];
      if constexpr (kCoded) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          *(f32x4*)(kt + half * 4) = *(const f32x4*)(kscale + sub * 32 + half * 16 + lg * 4);
          *(f32x4*)(vt + half * 4) = *(const f32x4*)(vscale + sub * 32 + half * 16 + lg * 4);
        }
      }
      const bool masked = holes || !((ts >= lo_max || ts + 32 <= a.sinks) && ts + 32 <= hi_min);
      uint32_t there = 0xffffffffu;
      if (holes) there = (uint32_t)__ballot(gone[sub * 32 + (lane & 31)] == 0);
      V8 ph[RB], pl[RB];
#pragma unroll
      for (int rb = 0; rb < RB; ++rb) {
        float z[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          z[j] = s[rb][j >> 2][j & 3] * zscale[rb];
          if constexpr (kCoded) z[j] *= kt[j];
        }
        uint32_t seen = 0xffffffffu;
        if (masked) {
          seen = seen32(rb, ts) & there;
#pragma unroll
          for (int j = 0; j < 8; ++j) z[j] = (seen >> ((j >> 2) * 16 + lg * 4 + (j & 3))) & 1u ? z[j] : -__builtin_inff();
        }
        float mt = -__builtin_inff();
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if constexpr (kCoded) mt = fmaxf(mt, z[j] + __builtin_amdgcn_logf(fmaxf(vt[j], 5.9604645e-8f)));
          else mt = fmaxf(mt, z[j]);
        }
        mt = max_rows32(max_rows16(mt));
        if (__any(mt > m_run[rb])) {
          const float m_new = fmaxf(m_run[rb], mt);
          const float alpha = factor(m_run[rb] - (m_new == -__builtin_inff() ? 0.0f : m_new));
          m_run[rb] = m_new;
          l_run[rb] *= alpha;
#pragma unroll
          for (int d = 0; d < kBlocks; ++d) o[rb][d] *= alpha;
        }
        const float m_use = m_run[rb] == -__builtin_inff() ? 0.0f : m_run[rb] - kLift;
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          float p0 = __builtin_amdgcn_exp2f(z[j] - m_use), p1 = __builtin_amdgcn_exp2f(z[j + 1] - m_use);
          l_run[rb] += p0 + p1;
          if constexpr (kCoded) {  // a hidden token's scale may be infinite or NaN
            p0 = !masked || (seen >> ((j >> 2) * 16 + lg * 4 + (j & 3))) & 1u ? p0 * vt[j] : 0.0f;
            p1 = !masked || (seen >> ((j >> 2) * 16 + lg * 4 + (j & 3) + 1)) & 1u ? p1 * vt[j + 1] : 0.0f;
          }
          split2(p0, p1, ph[rb], pl[rb], j);
        }
      }
      typedef __attribute__((address_space(3))) s16x4* lds_ptr;
#pragma unroll
      for (int d = 0; d < kBlocks; ++d) {
        union {
          s16x4 h[2];
          V8 v;
        } u;
        const char* const at = vs + (vread ^ (d << 5));
        u.h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)at);
        u.h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(at + 16 * DP * 2));
#pragma unroll
        for (int rb = 0; rb < RB; ++rb) {
          o[rb][d] = M::run(u.v, ph[rb], o[rb][d]);
          o[rb][d] = M::run(u.v, pl[rb], o[rb][d]);
        }
      }
    }
  }

  if constexpr (!kCoded) {
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
      f32x4 all = o[rb][0];
#pragma unroll
      for (int d = 1; d < kBlocks; ++d) all += o[rb][d];
      const float one = (all[0] + all[1]) + (all[2] + all[3]);
      if (works && __any(one != one)) {  // a NaN, or infinities of both signs
        uint64_t lost = 0;               // bit 4 d + i: sum i of block d is NaN
#pragma unroll
        for (int d = 0; d < kBlocks; ++d)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            lost |= (uint64_t)(o[rb][d][i] != o[rb][d][i]) << (4 * d + i);
            o[rb][d][i] = o[rb][d][i] != o[rb][d][i] ? 0.0f : o[rb][d][i];
          }
        const float m_use = m_run[rb] == -__builtin_inff() ? 0.0f : m_run[rb];
#pragma unroll 1
        for (int k = k0; k < k1; ++k)
#pragma unroll 1
          for (int sub = wt; sub < kSubs; sub += wt_all)
#pragma unroll 1
            for (int x = 0; x < 32; ++x) {
              const int t = tile_at(k) + sub * 32 + x;
              if (t >= hi_all) break;
              const uint32_t pg = (uint32_t)table[t >> a.c.page_shift];
              if (pg >= a.c.pages) continue;
              const long long at = cache_row(a.c, pg, head, (uint32_t)t & a.c.page_mask) * dim;
              float z = 0.0f;
#pragma unroll
              for (int s = 0; s < kSteps; ++s) {
                if (s * 32 + lg * 8 >= dim) continue;
                const Vec8<T> kv = *(const Vec8<T>*)((const T*)a.c.k + at + s * 32 + lg * 8);
#pragma unroll
                for (int j = 0; j < 8; ++j) z = fmaf((float)qf[rb][s][j], (float)kv.e[j], z);
              }
              z = add_rows32(add_rows16(z)) * zscale[rb];
              const bool seen = (seen32(rb, t & ~31) >> (t & 31)) & 1u;
              if (!seen || z == -__builtin_inff()) continue;
              const float p = __builtin_amdgcn_exp2f(z - m_use + kLift), w = p < 1.17549435e-38f ? 1.17549435e-38f : p;
#pragma unroll
              for (int d = 0; d < kBlocks; ++d) {
                if (d * 16 + lg * 4 >= dim) continue;
                T v[4];
                __builtin_memcpy(v, (const T*)a.c.v + at + d * 16 + lg * 4, sizeof v);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const float f = (float)v[i];
                  o[rb][d][i] = (lost >> (4 * d + i)) & 1u ? fmaf(fabsf(f) < __builtin_inff() ? p : w, f, o[rb][d][i]) : o[rb][d][i];
                }
              }
            }
      }
    }
  }

  // The sums of the waves on the same rows meet in LDS, one block of rows
  // after the other; from here on the maximum stands for the lifted one.
  float* const so = (float*)lds;  // [wave with wt > 0][16][DP], then its maxima and sums
  float* const sm = so + (wt_all - 1) * a.wr * 16 * DP;
  const int mine = (wt - 1) * a.wr + wr;
#pragma unroll
  for (int rb = 0; rb < RB; ++rb) {
    l_run[rb] = add_rows32(add_rows16(l_run[rb]));
    m_run[rb] -= kLift;
    if (wt_all > 1) {
      __syncthreads();
      if (wt > 0 && wt < wt_all) {
#pragma unroll
        for (int d = 0; d < kBlocks; ++d) *(f32x4*)(so + (mine * 16 + r16) * DP + d * 16 + lg * 4) = o[rb][d];
        if (lg == 0) {
          sm[(mine * 16 + r16) * 2] = m_run[rb];
          sm[(mine * 16 + r16) * 2 + 1] = l_run[rb];
        }
      }
      __syncthreads();
      if (wt == 0) {
        float m = m_run[rb];
        for (int w = 1; w < wt_all; ++w) m = fmaxf(m, sm[(((w - 1) * a.wr + wr) * 16 + r16) * 2]);
        const float m_use = m == -__builtin_inff() ? 0.0f : m;
        const float e0 = factor(m_run[rb] - m_use);
        float l = l_run[rb] * e0;
#pragma unroll
        for (int d = 0; d < kBlocks; ++d) o[rb][d] *= e0;
        for (int w = 1; w < wt_all; ++w) {
          const int from = ((w - 1) * a.wr + wr) * 16 + r16;
          const float e = factor(sm[from * 2] - m_use);
          l = fmaf(e, sm[from * 2 + 1], l);
#pragma unroll
          for (int d = 0; d < kBlocks; ++d) {
            const f32x4 x = *(const f32x4*)(so + from * DP + d * 16 + lg * 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) o[rb][d][i] = fmaf(e, x[i], o[rb][d][i]);
          }
        }
        m_run[rb] = m;
        l_run[rb] = l;
      }
    }
    if (wt != 0 || token[rb] < 0) continue;
    const long long row = (long long)token[rb] * a.q_heads + qhead[rb];
    const float l = l_run[rb];
    if (last) {
      const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
      for (int d = 0; d < kBlocks; ++d) {
        if (d * 16 + lg * 4 >= dim) continue;
        struct alignas(8) {
          QT e[4];
        } v;
#pragma unroll
        for (int i = 0; i < 4; ++i) v.e[i] = (QT)(l == 0.0f ? 0.0f : o[rb][d][i] * inv);
        *(decltype(v)*)((QT*)a.out + row * dim + d * 16 + lg * 4) = v;
      }
      if (lg == 0) {
        if (a.lse) a.lse[row] = (m_run[rb] + __builtin_amdgcn_logf(l)) * 0.69314718056f;
        if (a.pieces > 1) ((int*)(a.part + a.part_n))[row] = 0;
      }
    } else {
      const long long at = row * a.pieces + blockIdx.y;
#pragma unroll
      for (int d = 0; d < kBlocks; ++d)
        if (d * 16 + lg * 4 < dim) *(f32x4*)(a.part + at * dim + d * 16 + lg * 4) = o[rb][d];
      if (lg == 0) {
        *(float2*)(a.part + a.part_ml + at * 2) = make_float2(m_run[rb], l);
        if (blockIdx.y == 0) ((int*)(a.part + a.part_n))[row] = used;
      }
    }
  }
}

// Joins the pieces of one row: a workgroup of 64 threads for up to four rows
// (dim / 4 lanes each) in a fixed order.
template <class QT>
__global__ __launch_bounds__(64) void tree_join_kernel(TreeArgs a) {
  const int dim = a.c.head_dim, lanes = dim >> 2;
  const int at_once = 64 / lanes, g = threadIdx.x / lanes, t = threadIdx.x - g * lanes;
  const long long row = (long long)blockIdx.x * at_once + g;
  // rows that no request has (behind the last one's) hold no count
  if (g >= at_once || row >= (long long)a.tokens * a.q_heads) return;
  const int tok = (int)(row / a.q_heads);
  if (tok < start_of(a, 0) || tok >= start_of(a, a.batch)) return;
  const int n = ((const int*)(a.part + a.part_n))[row];
  if (n <= 1 || n > a.pieces) return;
  const float2* const ml = (const float2*)(a.part + a.part_ml) + row * a.pieces;
  float m = -__builtin_inff();
  for (int c = 0; c < n; ++c) m = fmaxf(m, ml[c].x);
  const float m_use = m == -__builtin_inff() ? 0.0f : m;
  f32x4 o = {0.0f, 0.0f, 0.0f, 0.0f};
  float l = 0.0f;
  const f32x4* const part = (const f32x4*)(a.part + row * a.pieces * dim) + t;
#pragma unroll 4
  for (int c = 0; c < n; ++c) {
    const float e = factor(ml[c].x - m_use);
    const f32x4 v = part[(long long)c * lanes];
    l = fmaf(e, ml[c].y, l);
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = fmaf(e, v[j], o[j]);
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  struct alignas(8) {
    QT e[4];
  } v;
#pragma unroll
  for (int j = 0; j < 4; ++j) v.e[j] = (QT)(l == 0.0f ? 0.0f : o[j] * inv);
  *(decltype(v)*)((QT*)a.out + row * dim + t * 4) = v;
  if (a.lse && t == 0) a.lse[row] = (m + __builtin_amdgcn_logf(l)) * 0.69314718056f;
}

// The unit files instantiate these (one file per pair of formats).
template <int Q, int F>
hipError_t launch_tree(const TreeArgs& a, int rb, dim3 grid, hipStream_t stream) {
  const int dim = a.c.head_dim;
  auto go = [&](auto dp, auto blocks) {
    constexpr int DP = decltype(dp)::value;
    auto kern = tree_kernel<Q, F, DP, decltype(blocks)::value>;
    static LaunchCache cache;
    const hipError_t e = prepare_launch(cache, (const void*)kern, 64 * kTreeWaves, tree_lds(DP), nullptr);
    if (e != hipSuccess) return e;
    kern<<<grid, dim3(64 * kTreeWaves), tree_lds(DP), stream>>>(a);
    return hipGetLastError();
  };
  typedef std::integral_constant<int, 1> One;
  typedef std::integral_constant<int, 2> Two;
  if (dim <= 64) return rb == 1 ? go(std::integral_constant<int, 64>{}, One{}) : go(std::integral_constant<int, 64>{}, Two{});
  if (dim <= 128) return rb == 1 ? go(std::integral_constant<int, 128>{}, One{}) : go(std::integral_constant<int, 128>{}, Two{});
  return go(std::integral_constant<int, 256>{}, One{});
}

hipError_t launch_tree_bf16(const TreeArgs& a, int rb, dim3 grid, hipStream_t stream);
hipError_t launch_tree_f16(const TreeArgs& a, int rb, dim3 grid, hipStream_t stream);
hipError_t launch_tree_int8(const TreeArgs& a, int q_dtype, int rb, dim3 grid, hipStream_t stream);

}  // namespace block
}  // namespace orbit
