// Attention of several new tokens per request over the paged cache
// (orbit_tree_attention): a tree of drafted tokens, a run (a prompt or a piece
// of one), or one token each behind a window with sinks:
//   o = sum_t p_t v_t / sum_t p_t,  p_t = exp(sm_scale q . k_t - m),
// over the tokens t that a new token sees, the maximum m and the sums carried
// along the tokens (one pass over the cache).
//
// Rows.  The new tokens of a request and the query heads of one key head are
// the rows r = token * group + head of one product with its keys.  A workgroup
// of eight waves takes up to 8 R rows (R = 16 or 32 to a wave) and a piece of
// the context: as many waves side by side on the rows as these need, the
// others on the tokens.  Tiles of 64 tokens (32 at head dimensions above 128)
// go from memory straight to an LDS ring of four stages, eight (four) rows by
// each wave, and every wave reads what it needs: a tile is read from memory
// once for all its rows, two or three are in flight while one is multiplied,
// and one barrier stands between two.  Codes of an int8 cache go through a
// ring that is the wave's own and become fp16 on their way to tiles in LDS,
// once for all rows.
//
// Products.  S^T = K Q^T with the keys as A operand; O^T = V^T P^T with the
// probabilities in the lanes that computed them; V^T by transposing LDS reads.
// R = 16, where a request has at most 32 rows on average: 16x16x32 products,
// probabilities as pairs of 16-bit numbers as in the single-token kernel
// (paged_attention_impl.h).  Those are bound by memory.  R = 32: 32x32x16
// products, half the instructions around a score; from 128 rows on the
// instructions bound them.  Probabilities are pairs for requests of at most 32
// rows there too, and one 16-bit number for larger ones, as pairs double their
// products (4096 new of 8192 tokens 627 us, trees below 125): that rounding is
// relative (within 2^-8 of each in bfloat16), as its value's was.
//
// What bounds it, 4096 new of 8192 tokens, 32 + 8 heads of 128, 420 to 443 us
// (0.93 to 0.98 PFLOP/s): no one part.  32 x 32 scores cost a wave 16 products
// (512 cycles), 24 LDS reads and about 100 vector instructions (a product and
// an exponential each, half a conversion, a sum and half a maximum for each of
// a lane's 16 scores); a SIMD's matrix cores are busy 40 % of the time, its
// vector issue 43 %, and its two waves wait 32 % of theirs: nothing sets one's
// products against the other's weights but chance.
// 16 trees of up to 60 drafted tokens after up to 8192 take 94 us (2.8 TB/s),
// 8 of 16 after up to 65000 in an int8 cache 156 us (2.0 TB/s),
// 64 single tokens behind a window of 4096 with sinks 175 us (5.4 TB/s).
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
  int rows;       // of a workgroup, at most
  int pieces;     // of a row's context, at most
  int slots;      // where there are no pieces: of row tiles
  int target;     // workgroups that the pieces should make
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
  r.begin = __builtin_amdgcn_readfirstlane(start_of(a, b));
  r.n = max(__builtin_amdgcn_readfirstlane(start_of(a, b + 1)) - r.begin, 0);
  const int len = __builtin_amdgcn_readfirstlane(a.lengths[b]);
  r.len = len < 0 ? 0 : len < a.cap ? len : a.cap;
  r.base = r.len - r.n;
  return r;
}

// Over a wave's lanes, x of this lane and those before it: six steps between
// registers (by LDS they took most of the time in which a piece is found).
template <class V, class F>
__device__ __forceinline__ V scan_lanes(V x, F add) {  // of values >= 0
  auto step = [&](auto ctrl, auto rows) {
    x = add(x, __builtin_bit_cast(V, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), decltype(ctrl)::value,
                                                                 decltype(rows)::value, 15, false)));
  };
  step(std::integral_constant<int, 0x111>{}, std::integral_constant<int, 15>{});  // from 1, 2, 4, 8 lanes before in the row of 16
  step(std::integral_constant<int, 0x112>{}, std::integral_constant<int, 15>{});
  step(std::integral_constant<int, 0x114>{}, std::integral_constant<int, 15>{});
  step(std::integral_constant<int, 0x118>{}, std::integral_constant<int, 15>{});
  step(std::integral_constant<int, 0x142>{}, std::integral_constant<int, 10>{});  // rows 1 and 3: from the last of the row before
  step(std::integral_constant<int, 0x143>{}, std::integral_constant<int, 12>{});  // rows 2 and 3: from lane 31
  return x;
}
template <class V, class F>
__device__ __forceinline__ V over_lanes(V x, F add) {
  return __builtin_bit_cast(V, __builtin_amdgcn_readlane(__builtin_bit_cast(int, scan_lanes(x, add)), 63));
}

// What a workgroup takes, where contexts are cut in pieces: a row tile of a
// request, and a piece of `per` tiles of its context; rq.b < 0: nothing.  Every
// workgroup counts the requests' row tiles and tiles, from which the size of a
// piece (one for all, so that together they are about a.target workgroups)
// and whose item this is follow.  Whole pieces come first and the contexts'
// rests last, where they fill what the others leave.
struct Item {
  Request rq;
  int row_tile, piece, per;
};
__device__ __forceinline__ Item item_of(const TreeArgs& a, int item, int tile, int lane) {
  int begin, n, len, row_tiles, tiles;  // of this lane's request
  auto count = [&](int x) {
    begin = n = len = row_tiles = tiles = 0;
    if (x >= a.batch) return;
    begin = start_of(a, x);
    n = max(start_of(a, x + 1) - begin, 0);
    len = min(max(a.lengths[x], 0), a.cap);
    row_tiles = (n * a.group + a.rows - 1) / a.rows;
    tiles = (len + tile - 1) / tile;
    if (a.window) tiles = min(tiles, (a.window + n) / tile + a.sinks / tile + 3);  // at most, for any of its rows
  };
  auto add = [](auto x, auto y) { return x + y; };
  int most = 0, rows = 0;
  float all = 0.0f;
  for (int x = 0; x < a.batch; x += 64) {
    count(x + lane);
    most = max(most, over_lanes(row_tiles ? tiles : 0, [](int x, int y) { return max(x, y); }));
    rows += over_lanes(row_tiles, add);
    all += over_lanes((float)row_tiles * (float)tiles, add);
  }
  // as many whole pieces as leave a workgroup to each rest
  const float left = fmaxf((float)a.target - 0.5f * (float)rows * (float)a.c.kv_heads, 0.25f * (float)a.target);
  Item it;
  it.per = max(max((int)(all * (float)a.c.kv_heads / left) + 1, (most + a.pieces - 1) / a.pieces), 2);
  it.per = __builtin_amdgcn_readfirstlane(it.per);
  it.rq.b = -1;
  for (int rest = 0; rest < 2; ++rest) {
    for (int x = 0; x < a.batch; x += 64) {
      if (a.batch > 64) count(x + lane);
      const int whole = tiles / it.per;
      // a request with nothing to see has zeros to write
      const int mine = row_tiles * (!rest ? whole : tiles > whole * it.per || tiles == 0);
      const int upto = scan_lanes(mine, add);
      const int total = __builtin_amdgcn_readlane(upto, 63);
      if (item < total) {
        const int who = __builtin_ctzll(__ballot(upto > item));
        const int local = item - (__builtin_amdgcn_readlane(upto, who) - __builtin_amdgcn_readlane(mine, who));
        const int r = __builtin_amdgcn_readlane(row_tiles, who);
        it.piece = rest ? __builtin_amdgcn_readlane(whole, who) : local / r;
        it.row_tile = r - 1 - (rest ? local : local - it.piece * r);
        it.rq.b = x + who;
        it.rq.begin = __builtin_amdgcn_readlane(begin, who);
        it.rq.n = __builtin_amdgcn_readlane(n, who);
        it.rq.len = __builtin_amdgcn_readlane(len, who);
        it.rq.base = it.rq.len - it.rq.n;
        return it;
      }
      item -= total;
    }
  }
  return it;
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

// A tile's rows in LDS, of ROW bytes, without padding: 16-byte unit u of row r
// lies in place u ^ key(r).  LDS serves 256 bytes at a time, so that a key's
// upper bits tell apart the rows 0 - 3 (4 - 7) whose four units, and the rows
// 0 - 7 whose two units a transposing read takes at once, all of them 16 rows
// of one unit (the operands' reads), and the last one neighbouring rows of
// which the conversion writes every other unit.  Row r + 8's key is row r's ^ 1.
// (By key = r's low bits 60 % of the cycles in LDS were conflicts: 487 us for 4096 new of 8192 tokens, 460 so.)
template <int ROW>
struct TreeStage {
  static __device__ __forceinline__ constexpr int key(int r) {
    return ROW == 128 ? (r & 2) << 1 | (r & 4) >> 1 | ((r >> 3 ^ r >> 1) & 1)
                      : (r & 1) << 3 | (r & 2) << 1 | (r & 4) >> 1 | ((r >> 3 ^ r) & 1);
  }
};

constexpr int kTreeWaves = 8;
constexpr int kTreeWords = 8;  // stages of the words
constexpr int kTreeStages = 4;
constexpr int kJoinMost = 256;  // threads of a workgroup that joins
constexpr int tree_key_tiles(bool coded) { return coded ? 2 : kTreeStages; }
constexpr int tree_value_tiles(bool coded) { return coded ? 3 : kTreeStages; }  // values are read a step later
constexpr int tree_tile(int dp) { return dp == 256 ? 32 : 64; }
constexpr int tree_rows(int dp) { return tree_tile(dp) / kTreeWaves; }  // of a tile, by each wave
// LDS: the 16-bit tiles (keys, then values), an int8 cache's codes and scales
// in the waves' own rings, what is made of the scales (float32: the keys', the
// values' and their logarithms), for each stage a word (bits: rows whose page
// lies outside the cache) and another (bytes: a wave's scales that are infinite
// or NaN), whether a wave saw such a page, 32 rows of zeros, and rows' maxima
// and sums.
constexpr int tree_tiles_lds(int dp, bool coded) { return (tree_key_tiles(coded) + tree_value_tiles(coded)) * tree_tile(dp) * dp * 2; }
constexpr int tree_raw_stage(int dp) { return 2 * tree_rows(dp) * dp; }    // of a wave
constexpr int tree_scale_stage(int dp) { return 4 * tree_rows(dp); }
constexpr int tree_lds(int dp, bool coded) {
  return tree_tiles_lds(dp, coded) +
         (coded ? kTreeStages * (kTreeWaves * (tree_raw_stage(dp) + tree_scale_stage(dp)) + 12 * tree_tile(dp)) : 0) + kTreeWords * 16 +
         kTreeWaves * 4 + 511 + (dp <= 128 ? 32 * dp * 2 : 0) + kTreeWaves * 32 * 8;
}
alignas(16) static __device__ const uint32_t kTreeZeros[4] = {0, 0, 0, 0};  // what is read in the place of tokens that are not there

// 16 (4) bytes a lane from memory to LDS at `to`, in lane order.  Inline, with
// explicit waits: the compiler would wait for all of them before each LDS read.
// Between the write of m0 and the load stands the wait state that gfx9 asks
// for, which the compiler does not add inside an inline block.
__device__ __forceinline__ void tree_load16(uint32_t to, const char* from) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(to), "v"(from) : "memory");
}
__device__ __forceinline__ void load_lds16(uint32_t to, uint32_t offset, const char* base) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(to), "v"(offset), "s"(base) : "memory");
}
__device__ __forceinline__ void tree_load4(uint32_t to, const char* from) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" ::"s"(to), "v"(from) : "memory");
}
template <int N>
__device__ __forceinline__ void tree_wait() {  // until at most N of this wave's loads are in flight, and no LDS access
  static_assert(N >= 0 && N < 64);
  __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | ((N >> 4) << 14));
  asm volatile("" ::: "memory");
}

// One product: 16x16x32 or 32x32x16, by the accumulator.
typedef float f32x16 __attribute__((ext_vector_type(16)));
__device__ __forceinline__ f32x4 tree_mma(bf16x8 a, bf16x8 b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0); }
__device__ __forceinline__ f32x4 tree_mma(f16x8 a, f16x8 b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0); }
__device__ __forceinline__ f32x16 tree_mma(bf16x8 a, bf16x8 b, f32x16 c) { return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0); }
__device__ __forceinline__ f32x16 tree_mma(f16x8 a, f16x8 b, f32x16 c) { return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0); }

// Q: the queries' format; F: the cache's; DP: head_dim rounded up to 64, 128
// or 256; R: rows of a wave, 16 or 32; PAIR: weights of every request, and not of
// those with at most 32 rows alone, as two 16-bit numbers.
//
// The lanes.  G = 64 / R lanes hold a row; lane l is number g = l / R of row l
// % R and holds, of 32 tokens' scores, tokens 4 G q + 4 g + i (i < 4), and of a
// row's sums coordinates 4 G c + 4 g + i: what a 16x16x32 (R = 16, both halves
// of the tokens) or a 32x32x16 product (R = 32) leaves.  32 rows to a wave take
// half the instructions around a score that 16 do (two blocks of 16 rows in a
// wave: 555 us for 4096 new of 8192 tokens).
template <int Q, int F, int DP, int R, bool PAIR>
__global__ __launch_bounds__(64 * kTreeWaves, R == 16 && DP == 64 ? 4 : 2) void tree_kernel(TreeArgs a) {
  constexpr bool kCoded = F == ORBIT_KV_INT8, kWide = R == 32;
  typedef Mma<F> M;
  typedef typename M::T T;
  typedef typename M::V8 V8;
  typedef typename Mma<Q>::T QT;
  constexpr int G = 64 / R, kStride = 4 * G;   // lanes of a row; tokens or coordinates between a lane's fours
  constexpr int kQuads = 32 / kStride;         // fours of scores of a lane
  constexpr int kTokens = tree_tile(DP), kSubs = kTokens / 32, kRows = tree_rows(DP), S = kTreeStages;
  constexpr int kSteps = DP / (8 * G);         // coordinates of a product: 8 G
  constexpr int kBlocks = DP / R;              // of a row's coordinates
  constexpr int kElem = kCoded ? 1 : 2;
  constexpr int kRowLanes = DP * kElem / 16, kAtOnce = 64 / kRowLanes;  // lanes on a row, rows of a load
  constexpr int kLoads = (kRows + kAtOnce - 1) / kAtOnce;               // of each tensor and tile; INT8: and one of scales
  constexpr int kInFlight = 2 * kLoads + (kCoded ? 1 : 0);
  constexpr float kLift = lift_of(F);
  typedef TreeStage<DP * 2> St;
  constexpr int kKeyTiles = tree_key_tiles(kCoded), kValueTiles = tree_value_tiles(kCoded);
  constexpr int kTileBytes = kTokens * DP * 2, kValuesAt = kKeyTiles * kTileBytes, kRaw = tree_raw_stage(DP);
  constexpr int kScale = tree_scale_stage(DP);
  constexpr uint32_t kRawAt = tree_tiles_lds(DP, kCoded), kScaleAt = kRawAt + (kCoded ? S * kTreeWaves * kRaw : 0),
                     kMadeAt = kScaleAt + (kCoded ? S * kTreeWaves * kScale : 0), kGoneAt = kMadeAt + (kCoded ? S * kTokens * 12 : 0),
                     kOddAt = kGoneAt + kTreeWords * 8, kSawAt = kOddAt + kTreeWords * 8,
                     kZerosAt = (kSawAt + kTreeWaves * 4 + 511) / 512 * 512,
                     kSumsAt = kZerosAt + (DP <= 128 ? 32 * DP * 2 : 0);
  static_assert(tree_tiles_lds(DP, kCoded) + (kCoded ? S * kTreeWaves * kRaw : 0) >= kTreeWaves * R * DP * 4);  // sums, at the end
  extern __shared__ __align__(1024) char lds[];

  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int rl = lane & (R - 1), g = lane / R, r16 = lane & 15;
  const int dim = a.c.head_dim;
  // neighbouring workgroups take the key heads of one item
  const int item = (int)blockIdx.x / a.c.kv_heads, head = (int)blockIdx.x - item * a.c.kv_heads;
  Item it;
  if (a.pieces > 1) {
    it = item_of(a, item, kTokens, lane);
    if (it.rq.b < 0 || it.piece < 0) return;  // negative: starts that decrease
  } else {
    // the last slots first: in a prompt they have the longest contexts
    const int slot = a.slots - 1 - item, b = request_at(a, slot, lane);
    it.rq = request_of(a, b);
    it.row_tile = __builtin_amdgcn_readfirstlane(slot - first_slot(a, b));
    it.piece = 0;
    it.per = 1 << 30;
  }
  const Request rq = it.rq;
  const int row0 = it.row_tile * a.rows, all_rows = rq.n * a.group;
  if (row0 < 0 || row0 >= all_rows) return;
  const int rows_here = min(a.rows, all_rows - row0);

  // the tiles that any of the rows sees part of: those of the sinks, then
  // those from the earliest window's first token on
  const int i_first = row0 / a.group, i_last = (row0 + rows_here - 1) / a.group;
  const int hi_all = a.words ? rq.len : max(rq.base + i_last + 1, 0);
  const int p_least = a.words ? rq.base - 1 : rq.base + i_first;
  const int lo_all = a.window ? max(p_least - a.window + 1, 0) : 0;
  const int end_tile = (hi_all + kTokens - 1) / kTokens;
  const int sink_tiles = a.window ? min((min(a.sinks, hi_all) + kTokens - 1) / kTokens, end_tile) : 0;
  const int first_tile = max(sink_tiles, lo_all / kTokens);
  const int tiles = sink_tiles + max(end_tile - first_tile, 0);
  const int per = it.per, used = (tiles + per - 1) / per;
  const int k0 = min(it.piece * per, tiles), k1 = min(tiles, k0 + per);
  const bool last = used <= 1;  // nothing to join
  if (k0 >= k1 && it.piece > 0) return;

  // Waves on the rows, so many as these need, and on the tokens; where four
  // are on the tokens a step takes two tiles, otherwise one.
  int wrs = 1;
  while (wrs * R < rows_here) wrs *= 2;
  const int wt_all = min(kTreeWaves / wrs, 2 * kSubs), step = wt_all > kSubs ? 2 : 1;
  const int wr = wave & (wrs - 1), wt = wave / wrs;
  const bool works = wt < wt_all && wr * R < rows_here;

  // this lane's row: its token, its query head, the prefix tokens [lo, hi)
  const bool row_in = wr * R + rl < rows_here;
  const int row_at = row_in ? row0 + wr * R + rl : row0;
  const int row_i = row_at / a.group;
  const int token = rq.begin + row_i, qhead = head * a.group + row_at - row_i * a.group;
  int lo = 0, hi = a.words ? rq.base : rq.base + row_i + 1;
  if (a.window) {
    int p = rq.base + row_i;
    if (a.words) {
      int seen = 0;
      const uint64_t* const mask = a.tree + (long long)token * a.words;
      for (int w = 0; w < a.words && w * 64 < rq.n; ++w) {
        const int left = rq.n - w * 64;
        seen += __popcll(left >= 64 ? mask[w] : mask[w] & ((1ull << left) - 1));
      }
      p = rq.base + seen - 1;
    }
    lo = max(p - a.window + 1, 0);
  }
  // all of the wave's rows see the tokens [lo_max, hi_min)
  const int i0 = (row0 + wr * R) / a.group, i1 = (row0 + min(wr * R + R, rows_here) - 1) / a.group;
  int lo_max = a.window ? max(rq.base + i1 - a.window + 1, 0) : 0, hi_min = a.words ? rq.base : rq.base + i0 + 1;
  if (a.window && a.words) {
    lo_max = row_in ? lo : 0;
#pragma unroll
    for (int s = 1; s < R; s *= 2) lo_max = max(lo_max, __shfl_xor(lo_max, s));
  }
  lo_max = __builtin_amdgcn_readfirstlane(lo_max);
  hi_min = __builtin_amdgcn_readfirstlane(hi_min);

  // the bits of the tokens among 32 from t0 on that this lane's row sees
  auto seen32 = [&](int t0) {
    uint32_t m = range32(lo, hi, t0);
    if (a.window) m |= range32(0, min(a.sinks, hi), t0);
    if (a.words && t0 + 32 > rq.base && row_in)
      m |= bits32(a.tree + (long long)token * a.words, a.words, t0 - rq.base) & range32(max(rq.base, 0), rq.len, t0);
    return m;
  };
  auto bit_of = [&](int j) { return j / 4 * kStride + g * 4 + j % 4; };  // of score j among the 32 tokens
  // over the lanes of a row
  auto row_max = [&](float v) { return max_rows32(kWide ? v : max_rows16(v)); };
  auto row_add = [&](float v) { return add_rows32(kWide ? v : add_rows16(v)); };

  // Loading.  This wave's rows of a tile are kRows wave .. + kRows - 1, load i
  // takes those from i * kAtOnce on, a lane 16 bytes: rows on one page, all of
  // them seen by some row and without padding, at constant places from a
  // scalar address.  Otherwise each lane has an address of its own, and tokens
  // from hi_all on, those whose page lies outside the cache, and coordinates
  // past head_dim are read as zeros.
  const int row_bytes = dim * kElem;
  const int lrow = lane / kRowLanes, lplace = lane & (kRowLanes - 1);
  typedef const __attribute__((address_space(4))) int32_t* const_ptr;  // by scalar loads, which no vector load waits for
  const int32_t* const table = a.table + rq.b * a.table_stride;
  auto tile_at = [&](int k) { return (k < sink_tiles ? k : first_tile + k - sink_tiles) * kTokens; };
  const bool plain = (int)a.c.page_mask + 1 >= kRows && dim == DP;
  uint32_t lane_at[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int r = i * kAtOnce + lrow;
    // unit of the row that belongs in this lane's place (keys of rows 16 apart are the same)
    lane_at[i] = (uint32_t)(r * row_bytes + (kCoded ? lplace : lplace ^ St::key((wave * kRows + r) & 15)) * 16);
  }
  constexpr int kPairs = kRows / 2;
  const uint32_t scale_at = 4 * ((uint32_t)lane % kPairs);  // INT8: two tokens a lane, keys' scales, then values'
  uint32_t page = 0xffffffffu;  // of the next tile's first row
  auto look_up = [&](int k) {
    const int t = tile_at(k) + wave * kRows;
    page = k < k1 && t < hi_all ? (uint32_t)((const_ptr)(uintptr_t)table)[t >> a.c.page_shift] : 0xffffffffu;
  };
  auto issue = [&](int k) {
    const int t0 = tile_at(k) + wave * kRows, stage = (int)((uint32_t)k % S);
    const uint32_t to = kCoded ? kRawAt + (uint32_t)(stage * kTreeWaves + wave) * kRaw
                               : (uint32_t)stage * kTileBytes + (uint32_t)wave * kRows * DP * 2;
    constexpr uint32_t kValues = kCoded ? kRows * DP : kValuesAt;
    const uint32_t to_scales = kScaleAt + ((uint32_t)k % S * kTreeWaves + wave) * kScale;
    uint32_t gone = 0;  // of this wave's rows
    if (plain && page < a.c.pages && t0 + kRows <= hi_all) {
      const long long row = cache_row(a.c, page, head, (uint32_t)t0 & a.c.page_mask);
      const char *const kb = a.c.k + row * row_bytes, *const vb = a.c.v + row * row_bytes;
      if constexpr (kCoded) {
        if (lane < 2 * kPairs) tree_load4(to_scales, (const char*)((lane < kPairs ? a.c.ks : a.c.vs) + row) + scale_at);
      }
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        if (kRows < kAtOnce && lrow >= kRows) break;
        load_lds16(to + i * 1024, lane_at[i], kb);
        load_lds16(to + kValues + i * 1024, lane_at[i], vb);
      }
    } else {
      auto page_of = [&](int t) { return t < hi_all ? (uint32_t)table[t >> a.c.page_shift] : 0xffffffffu; };
      const char* from_k[kLoads];
      const char* from_v[kLoads];
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int r = i * kAtOnce + lrow, t = t0 + r;
        const uint32_t pg = page_of(t);
        const bool there = pg < a.c.pages;
        const int byte = (int)(lane_at[i] - (uint32_t)(r * row_bytes));
        const bool in = there && byte < row_bytes;
        const long long at = cache_row(a.c, there ? pg : 0, head, (uint32_t)t & a.c.page_mask) * row_bytes + byte;
        from_k[i] = in ? a.c.k + at : (const char*)kTreeZeros;
        from_v[i] = in ? a.c.v + at : (const char*)kTreeZeros;
        const uint64_t lost = __ballot(!there && t < hi_all && r < kRows);
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) gone |= (uint32_t)((lost >> (j * kRowLanes)) & 1u) << (i * kAtOnce + j);
      }
      if constexpr (kCoded) {  // the two tokens lie on one page, as pages are even
        const int t = t0 + 2 * (lane % kPairs);
        const uint32_t pg = page_of(t);
        const long long at = cache_row(a.c, pg < a.c.pages ? pg : 0, head, (uint32_t)t & a.c.page_mask);
        const char* const from_s = pg < a.c.pages ? (const char*)((lane < kPairs ? a.c.ks : a.c.vs) + at) : (const char*)kTreeZeros;
        if (lane < 2 * kPairs) tree_load4(to_scales, from_s);
      }
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        if (kRows < kAtOnce && lrow >= kRows) break;
        tree_load16(to + i * 1024, from_k[i]);
        tree_load16(to + kValues + i * 1024, from_v[i]);
      }
    }
    if (lane == 0) ((uint8_t*)(lds + kGoneAt))[(uint32_t)k % kTreeWords * 8 + wave] = (uint8_t)gone;
  };
  // INT8: this wave's rows of tile k become fp16, and their scales float32
  auto convert = [&](int k) {
    const char* const raw = lds + kRawAt + (uint32_t)(((uint32_t)k % S) * kTreeWaves + wave) * kRaw;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      if (kRows < kAtOnce && lrow >= kRows) break;
      const int r = wave * kRows + i * kAtOnce + lrow;
      const u32x4 k4 = *(const u32x4*)(raw + i * 1024 + lane * 16), v4 = *(const u32x4*)(raw + kRows * DP + i * 1024 + lane * 16);
      char* const to = lds + (uint32_t)k % kKeyTiles * kTileBytes + r * DP * 2;
      char* const to_v = lds + kValuesAt + (uint32_t)k % kValueTiles * kTileBytes + r * DP * 2;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int at = ((lplace * 2 + c) ^ St::key(r & 15)) << 4;
        const u32x2 x = codes_to_f16(k4[2 * c]), y = codes_to_f16(k4[2 * c + 1]);
        const u32x2 z = codes_to_f16(v4[2 * c]), w = codes_to_f16(v4[2 * c + 1]);
        *(u32x4*)(to + at) = u32x4{x.x, x.y, y.x, y.y};
        *(u32x4*)(to_v + at) = u32x4{z.x, z.y, w.x, w.y};
      }
    }
    bool odd = false;
    if (lane < kRows) {
      const char* const from = lds + kScaleAt + ((uint32_t)k % S * kTreeWaves + wave) * kScale + lane * 2;
      const float x = (float)*(const _Float16*)from, y = (float)*(const _Float16*)(from + 2 * kRows);
      float* const made = (float*)(lds + kMadeAt) + (uint32_t)k % S * (3 * kTokens) + wave * kRows + lane;
      made[0] = x;
      made[kTokens] = y;
      made[2 * kTokens] = __builtin_amdgcn_logf(fmaxf(y, 5.9604645e-8f));
      odd = y - y != 0.0f;
    }
    const bool some = __any(odd);
    if (lane == 0) ((uint8_t*)(lds + kOddAt))[(uint32_t)k % kTreeWords * 8 + wave] = some;
  };
  // this wave's loads have landed
  auto landed = [&](int later) {  // but for those of the `later` last tiles
    if (later >= 3) tree_wait<3 * kInFlight>();
    else if (later == 2) tree_wait<2 * kInFlight>();
    else if (later == 1) tree_wait<kInFlight>();
    else tree_wait<0>();
  };
  auto meet = [] {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };

  // Queries.  kWide: read by whole rows (7500 cycles of a prompt's workgroup
  // went into reading them as operands, 32 bytes of 32 rows at a time) and
  // brought into the operands' order in LDS, in stages that no load is on its
  // way to yet: behind the tiles in flight, or (INT8) where codes will be
  // converted to, from the first barrier on.
  Vec8<QT> q8[kSteps];
  constexpr int kRowUnits = DP / 8;  // 16-byte units of a row
  {
    const long long at = (long long)token * a.qts + qhead * a.qhs;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      int r = rl, d = (s * G + g) * 8;
      long long from = at;
      if constexpr (kWide) {
        r = s * (64 / kRowUnits) + lane / kRowUnits;
        d = lane % kRowUnits * 8;
        from = __shfl(at, r);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) q8[s].e[j] = (QT)0.0f;
      if (wr * R + r < rows_here && d < dim) q8[s] = *(const Vec8<QT>*)((const QT*)a.q + from + d);
    }
  }
  // the pages of the first tiles' rows, a lane each
  uint32_t first_pages = 0xffffffffu;
  if (lane < kTreeStages && k0 + lane < k1) {
    const int t = tile_at(k0 + lane) + wave * kRows;
    if (t < hi_all) first_pages = (uint32_t)table[t >> a.c.page_shift];
  }
  // whether any page that the piece's rows see lies outside the cache.  Pages
  // between the sinks and the window are not looked at: a server gives them up,
  // and a part of a tile that no row sees is masked anyway.
  bool bad = false;
  auto look = [&](int from, int to) {  // tokens
    if (from < to)
      for (int x = (from >> a.c.page_shift) + tid; x <= (to - 1) >> a.c.page_shift; x += 64 * kTreeWaves)
        bad |= (uint32_t)table[x] >= a.c.pages;
  };
  if (k0 < sink_tiles) {
    const int from = tile_at(k0), to = min(min(k1, sink_tiles) * kTokens, hi_all);
    look(from, min(to, a.sinks));
    look(max(from, lo_all), to);  // a window may reach into them
  }
  if (k1 > sink_tiles) look(max(tile_at(max(k0, sink_tiles)), lo_all), min(tile_at(k1 - 1) + kTokens, hi_all));
  // as the B operand
  V8 qf[kSteps];
  float zscale = fabsf(a.scale_log2e);
  {
    if constexpr (kWide) {
      char* const mine = lds + (kCoded ? wave * R * DP * 2 : wave / 4 * kValuesAt + (k0 + 2 + wave / 2 % 2) % S * kTileBytes + wave % 2 * R * DP * 2);
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        const int r = s * (64 / kRowUnits) + lane / kRowUnits;
        *(Vec8<QT>*)(mine + r * DP * 2 + ((lane % kRowUnits ^ St::key(r & 15)) << 4)) = q8[s];
      }
#pragma unroll
      for (int s = 0; s < kSteps; ++s) q8[s] = *(const Vec8<QT>*)(mine + rl * DP * 2 + (((s * G + g) ^ St::key(rl & 15)) << 4));
    }
    float f[kSteps][8], m = 0.0f;
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        // the scale's sign goes to the query, so that the largest product is the largest score
        f[s][j] = a.scale_log2e < 0.0f ? -(float)q8[s].e[j] : (float)q8[s].e[j];
        if (kCoded) m = fmaxf(m, fabsf(f[s][j]));
      }
    if (kCoded) {  // into fp16's range by a power of two per row
      m = row_max(m);
      const int e = m > 0.0f && m < __builtin_inff() ? __builtin_amdgcn_frexp_expf(m) : 0;
      const float down = ldexpf(1.0f, -e / 2), down2 = ldexpf(1.0f, -e - (-e / 2));
      zscale = ldexpf(zscale, e);
#pragma unroll
      for (int s = 0; s < kSteps; ++s)
#pragma unroll
        for (int j = 0; j < 8; ++j) f[s][j] = f[s][j] * down * down2;
    }
    zscale = fmaxf(zscale, 1.17549435e-38f);  // not 0: a hidden score is minus infinity
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
#pragma unroll
      for (int j = 0; j < 8; ++j) qf[s][j] = (T)f[s][j];
      asm volatile("" : "+v"(qf[s]));  // or the unrounded values are kept too, for the sums below
    }
  }

  // The sums: o[c], coordinates kStride c + 4 g + i; relative to m_run.
  typedef float f32xR __attribute__((ext_vector_type(kWide ? 16 : 4)));
  constexpr float kSlack = F == ORBIT_KV_BF16 ? 8.0f : 0.0f;
  f32xR o[kBlocks];
  float m_run = -__builtin_inff(), l_run = 0.0f;  // l: this lane's tokens alone
  constexpr int kOf = kWide ? 16 : 4;  // sums of a block in a lane
#pragma unroll
  for (int d = 0; d < kBlocks; ++d)
#pragma unroll
    for (int i = 0; i < kOf; ++i) o[d][i] = 0.0f;
  // where this lane reads its first operands
  int kread = rl * DP * 2 + ((g ^ St::key(rl & 15)) << 4);
  const int trow = g * 4 + (r16 >> 2), tunit = (kWide ? ((lane >> 4) & 1) * 2 : 0) + ((r16 & 3) >> 1);
  int vread = trow * DP * 2 + ((tunit ^ St::key(trow)) << 4) + (r16 & 1) * 8;

  // With 32 rows (kWide) the scores of 32 tokens are computed beside the
  // weights of the 32 before them, whose products come next, so that a wave's
  // matrix and vector instructions overlap; also over a step's end where it has
  // one tile: those values are read behind the next barrier, so the stage after
  // next is filled and not the next.
  constexpr int kScores = 4 * kQuads;  // of a lane
  float vt[kCoded ? kScores : 1];  // INT8: the values' scales
  int pend = 0;  // place of their values in LDS
  bool pend_odd = false;  // INT8: some of the values' scales are infinite or NaN
  uint32_t pend_seen = 0;

  // The operands' places: `lds` is at LDS's beginning, and its address would be added to each.
  typedef const __attribute__((address_space(3))) u32x4* lds_16;
  V8 ph[kScores / 8], pl[kScores / 8];
  // Scores of 32 tokens (SCORES), and weights of the pending ones (WEIGHTS), a
  // part of both at a time: the weights' instructions stand between the keys'
  // reads and their products.
  // CHECKED: values' scales of hidden tokens may be infinite or NaN.
  // Scores z of the 32 tokens whose keys lie `skip` behind the place that
  // `keys` says, weights of s.
  auto advance_as = [&](float (&z)[kScores], const float (&s)[kScores], int keys, auto skip, auto with_scores, auto with_weights, auto in_pairs, auto checked) {
    constexpr bool SCORES = decltype(with_scores)::value, WEIGHTS = decltype(with_weights)::value, CHECKED = decltype(checked)::value;
    constexpr int kPairs2 = kScores / 2;  // weights, two by two
    const float m_use = m_run == -__builtin_inff() ? 0.0f : m_run - kLift;
    f32xR acc[kWide ? 1 : 2];
    if constexpr (SCORES) {
#pragma unroll
      for (int h = 0; h < (kWide ? 1 : 2); ++h)
#pragma unroll
        for (int i = 0; i < kOf; ++i) acc[h][i] = 0.0f;
    }
    constexpr int kAheadK = kWide ? 3 : 1;  // keys are read so many parts ahead
    V8 kv[kAheadK + 1][kWide ? 1 : 2];
    auto read_keys = [&](int i) {
#pragma unroll
      for (int h = 0; h < (kWide ? 1 : 2); ++h)
        kv[i % (kAheadK + 1)][h] = __builtin_bit_cast(V8, *(lds_16)(uint32_t)((keys ^ (i * G << 4)) + h * 16 * DP * 2 + decltype(skip)::value));
    };
    if constexpr (SCORES) {
#pragma unroll
      for (int i = 0; i < kAheadK && i < kSteps; ++i) read_keys(i);
    }
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      if constexpr (SCORES) {
        if (i + kAheadK < kSteps) read_keys(i + kAheadK);
      }
      if constexpr (WEIGHTS) {
#pragma unroll
        for (int x = kPairs2 * i / kSteps; x < kPairs2 * (i + 1) / kSteps; ++x) {
          const int j = 2 * x;
          float p[2];
#pragma unroll
          for (int y = 0; y < 2; ++y) p[y] = __builtin_amdgcn_exp2f(fmaf(s[j + y], zscale, -m_use));
          l_run += p[0] + p[1];
          if constexpr (kCoded) {
#pragma unroll
            for (int y = 0; y < 2; ++y) p[y] = !CHECKED || (pend_seen >> bit_of(j + y)) & 1u ? p[y] * vt[j + y] : 0.0f;
          }
          if constexpr (decltype(in_pairs)::value) {
            split2(p[0], p[1], ph[j / 8], pl[j / 8], j % 8);
          } else {
            ph[j / 8][j % 8] = (T)p[0];
            ph[j / 8][j % 8 + 1] = (T)p[1];
          }
        }
      }
      if constexpr (SCORES) {
#pragma unroll
        for (int h = 0; h < (kWide ? 1 : 2); ++h) acc[h] = tree_mma(kv[i % (kAheadK + 1)][h], qf[i], acc[h]);
      }
      if constexpr (SCORES) __builtin_amdgcn_sched_barrier(0);
    }
    if constexpr (SCORES) {
#pragma unroll
      for (int j = 0; j < kScores; ++j) z[j] = acc[kWide ? 0 : j / 4][kWide ? j : j % 4];
    }
  };
  auto advance = [&](float (&z)[kScores], const float (&s)[kScores], int keys, auto skip, auto with_scores, auto with_weights, auto in_pairs) {
    if (kCoded && decltype(with_weights)::value && pend_odd) advance_as(z, s, keys, skip, with_scores, with_weights, in_pairs, std::true_type{});
    else advance_as(z, s, keys, skip, with_scores, with_weights, in_pairs, std::false_type{});
  };
  // The pending tokens' weights with their values, by blocks of R coordinates
  // (and 16 tokens: kWide); some products' operands are read ahead.
  auto products = [&](auto in_pairs) {
    typedef __attribute__((address_space(3))) s16x4* lds_ptr;
    constexpr int kAll = kBlocks * (kWide ? 2 : 1);
    // rows 8 (kWide) or 16 further: this far, with the units' places exchanged
    constexpr int kFar = kWide ? 8 : 16, kOther = kWide ? 1 : 0;
    constexpr int kAheadV = kWide ? 4 : 2;
    union Block {
      s16x4 h[2];
      V8 v;
    } u[kAheadV + 1];
    const int values = vread + pend;
    auto read = [&](int n) {
      const int d = kWide ? n >> 1 : n, m = kWide ? n & 1 : 0;
      const int at = values ^ (d * (R / 8) << 4);
      u[n % (kAheadV + 1)].h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(uint32_t)(at + m * 16 * DP * 2));
      u[n % (kAheadV + 1)].h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(uint32_t)((at ^ (kOther << 4)) + (m * 16 + kFar) * DP * 2));
    };
#pragma unroll
    for (int n = 0; n < kAheadV && n < kAll; ++n) read(n);
#pragma unroll
    for (int n = 0; n < kAll; ++n) {
      if (n + kAheadV < kAll) read(n + kAheadV);
      const int d = kWide ? n >> 1 : n, m = kWide ? n & 1 : 0;
      o[d] = tree_mma(u[n % (kAheadV + 1)].v, ph[m], o[d]);
      if constexpr (decltype(in_pairs)::value) o[d] = tree_mma(u[n % (kAheadV + 1)].v, pl[m], o[d]);
      if (kWide || n % 2) __builtin_amdgcn_sched_barrier(0);
    }
  };

  // Tiles in flight beside a step's: codes' places are free once converted;
  // others' when the next barrier says so (kWide: the next but one).
  const int ahead = kCoded ? S : step == 2 || kWide ? 2 : S - 1;
#pragma unroll 1
  for (int x = k0; x < min(k0 + ahead, k1); ++x) {
    page = __builtin_amdgcn_readlane(first_pages, x - k0);
    issue(x);
  }
  look_up(k0 + ahead);
  if constexpr (kWide) {
    for (int x = tid; x < 32 * DP * 2 / 16; x += 64 * kTreeWaves) *(u32x4*)(lds + kZerosAt + x * 16) = u32x4{0u, 0u, 0u, 0u};
  }
  if (lane == 0) ((uint32_t*)(lds + kSawAt))[wave] = 0;
  if (__any(bad)) ((uint32_t*)(lds + kSawAt))[wave] = 1;
  tree_wait<62>();
  meet();
  const u32x4 bad0 = *(const u32x4*)(lds + kSawAt), bad1 = *(const u32x4*)(lds + kSawAt + 16);
  const bool holes = __builtin_amdgcn_readfirstlane(bad0.x | bad0.y | bad0.z | bad0.w | bad1.x | bad1.y | bad1.z | bad1.w) != 0;
  auto fresh = [&] { asm volatile("" : "+v"(kread), "+v"(vread)); };  // the places made of them are not kept in registers
  // A step's tiles, there and ready to be read by all waves.
  auto begin_step = [&](int k, auto step, int here) {
    landed(min(k1, k + ahead) - k - here);
    if constexpr (kCoded) {
      // two tiles take a place that the step before had: it must have been read
      if (step == 2) meet();
      convert(k);
      if (here == 2) convert(k + 1);
      tree_wait<62>();
    }
    meet();  // the tiles are there, and those of the step before (kWide: the one before that) have been read
#pragma unroll 1
    for (int x = k + ahead; x < min(k + ahead + step, k1); ++x) {  // into their stages
      issue(x);
      look_up(x + 1);
    }
    fresh();
  };
  // Scores z of the 32 tokens from ts on (part `sub` of tile `at`) are
  // scaled, masked, the maximum carried on.
  auto take = [&](float (&z)[kScores], int at, int sub, int ts) {
    float lv[kCoded ? kScores : 1];
    if constexpr (kCoded) {
      const float* const made = (const float*)(lds + kMadeAt) + (uint32_t)at % S * (3 * kTokens) + sub * 32 + g * 4;
#pragma unroll
      for (int q = 0; q < kQuads; ++q) {
        const f32x4 x = *(const f32x4*)(made + q * kStride), y = *(const f32x4*)(made + kTokens + q * kStride),
                    l = *(const f32x4*)(made + 2 * kTokens + q * kStride);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          z[q * 4 + i] *= x[i];
          vt[q * 4 + i] = y[i];
          lv[q * 4 + i] = l[i];
        }
      }
      const uint32_t* const odd = (const uint32_t*)(lds + kOddAt + (uint32_t)at % kTreeWords * 8);
      pend_odd = __builtin_amdgcn_readfirstlane(kRows == 4 ? odd[0] | odd[1] : odd[sub]) != 0;
      pend_seen = 0xffffffffu;
    }
    if (holes || !((ts >= lo_max || ts + 32 <= a.sinks) && ts + 32 <= hi_min)) {
      uint32_t seen = seen32(ts);
      if (holes) {  // a wave's rows are a byte, or half of one
        uint64_t rows = *(const uint64_t*)(lds + kGoneAt + (uint32_t)at % kTreeWords * 8);
        if (kRows == 4) {
          const uint64_t gone = rows;
          rows = 0;
#pragma unroll
          for (int w = 0; w < 8; ++w) rows |= ((gone >> (8 * w)) & 15u) << (4 * w);
        }
        seen &= ~(uint32_t)(rows >> (sub * 32));
      }
      pend_seen = seen;
#pragma unroll
      for (int j = 0; j < kScores; ++j) z[j] = (seen >> bit_of(j)) & 1u ? z[j] : -__builtin_inff();
    }
    float mt = -__builtin_inff();
#pragma unroll
    for (int j = 0; j < kScores; ++j) {
      if constexpr (kCoded) mt = fmaxf(mt, fmaf(z[j], zscale, lv[j]));
      else mt = fmaxf(mt, z[j]);
    }
    if constexpr (!kCoded) mt *= zscale;
    mt = row_max(mt);
    // with float32's range for the weights (bfloat16) a larger score by less
    // than 2^8 may stay: the sums are relative to m_run either way
    if (__any(mt > m_run + kSlack)) {
      const float m_new = fmaxf(m_run, mt);
      const float alpha = factor(m_run - (m_new == -__builtin_inff() ? 0.0f : m_new));
      m_run = m_new;
      l_run *= alpha;
#pragma unroll
      for (int d = 0; d < kBlocks; ++d) o[d] *= alpha;
    }
  };
  auto keys_of = [&](int at) { return kread + (int)((uint32_t)at % kKeyTiles) * kTileBytes; };
  auto values_of = [&](int at, int sub) { return kValuesAt + (int)((uint32_t)at % kValueTiles) * kTileBytes + sub * 32 * DP * 2; };
  typedef std::integral_constant<int, 0> First;
  typedef std::integral_constant<int, 32 * DP * 2> Second;
  float s[kScores];
  if (kWide && step == 1) {
    // nothing is pending: zeros
#pragma unroll
    for (int j = 0; j < kScores; ++j) {
      s[j] = -__builtin_inff();
      if constexpr (kCoded) vt[j] = 0.0f;
    }
    pend = kZerosAt;
    auto next = [&](float (&z)[kScores], const float (&was)[kScores], int k, int keys, auto skip, int sub) {
      advance(z, was, keys, skip, std::true_type{}, std::true_type{}, std::false_type{});
      products(std::false_type{});
      pend = values_of(k, sub);
      take(z, k, sub, tile_at(k) + sub * 32);
    };
#pragma unroll 1
    for (int k = k0; k < k1; ++k) {
      begin_step(k, std::integral_constant<int, 1>{}, 1);
      // a wave has both halves of the tile or one; scores in two sets of registers
      if (works && tile_at(k) + wt * 32 < hi_all) {
        const int keys = keys_of(k) + wt * 32 * DP * 2;
        float z[kScores];
        next(z, s, k, keys, First{}, wt);
        if (wt_all == 1 && tile_at(k) + 32 < hi_all) {
          next(s, z, k, keys, Second{}, 1);
        } else {
#pragma unroll
          for (int j = 0; j < kScores; ++j) s[j] = z[j];
        }
      }
    }
    if (works) {
      float none[kScores];
      advance(none, s, 0, First{}, std::false_type{}, std::true_type{}, std::false_type{});
      products(std::false_type{});
    }
  } else {
    auto steps = [&](auto in_pairs) {
#pragma unroll 1
      for (int k = k0; k < k1; k += step) {
        const int here = min(step, k1 - k);  // tiles of this step
        begin_step(k, step, here);
        const int n1 = works ? here * kSubs : 0;
#pragma unroll 1
        for (int n = wt; n < n1; n += wt_all) {
          const int at = k + n / kSubs, sub = n % kSubs, ts = tile_at(at) + sub * 32;
          if (ts >= hi_all) break;
          advance(s, s, keys_of(at) + sub * 32 * DP * 2, First{}, std::true_type{}, std::false_type{}, in_pairs);
          take(s, at, sub, ts);
          pend = values_of(at, sub);
          advance(s, s, 0, First{}, std::false_type{}, std::true_type{}, in_pairs);
          products(in_pairs);
        }
      }
    };
    // a request of few rows keeps pairs beside larger ones, too: what it is batched with does not cost it digits
    if (PAIR || all_rows <= 32) steps(std::true_type{});
    else steps(std::false_type{});
  }

  if constexpr (!kCoded) {
    float one = 0.0f;
#pragma unroll
    for (int d = 0; d < kBlocks; ++d)
#pragma unroll
      for (int i = 0; i < kOf; ++i) one += o[d][i];
    if (works && __any(one != one)) {  // a NaN, or infinities of both signs
      uint64_t lost = 0;               // bit kOf d + i: that sum is NaN
#pragma unroll
      for (int d = 0; d < kBlocks; ++d)
#pragma unroll
        for (int i = 0; i < kOf; ++i) {
          lost |= (uint64_t)(o[d][i] != o[d][i]) << (kOf * d + i);
          o[d][i] = o[d][i] != o[d][i] ? 0.0f : o[d][i];
        }
      const float m_use = m_run == -__builtin_inff() ? 0.0f : m_run;
#pragma unroll 1
      for (int k = k0; k < k1; k += step)
#pragma unroll 1
        for (int n = wt; n < min(step, k1 - k) * kSubs; n += wt_all)
#pragma unroll 1
          for (int x = 0; x < 32; ++x) {
            const int t = tile_at(k + n / kSubs) + n % kSubs * 32 + x;
            if (t >= hi_all) break;
            const uint32_t pg = (uint32_t)table[t >> a.c.page_shift];
            if (pg >= a.c.pages) continue;
            const long long at = cache_row(a.c, pg, head, (uint32_t)t & a.c.page_mask) * dim;
            float z = 0.0f;
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
              const int e = (s * G + g) * 8;
              if (e >= dim) continue;
              const Vec8<T> kv = *(const Vec8<T>*)((const T*)a.c.k + at + e);
#pragma unroll
              for (int j = 0; j < 8; ++j) z = fmaf((float)qf[s][j], (float)kv.e[j], z);
            }
            z = row_add(z) * zscale;
            const bool seen = (seen32(t & ~31) >> (t & 31)) & 1u;
            if (!seen || z == -__builtin_inff()) continue;
            const float p = __builtin_amdgcn_exp2f(z - m_use + kLift), w = p < 1.17549435e-38f ? 1.17549435e-38f : p;
#pragma unroll
            for (int c = 0; c < DP / kStride; ++c) {
              const int e = c * kStride + g * 4;
              if (e >= dim) continue;
              T v[4];
              __builtin_memcpy(v, (const T*)a.c.v + at + e, sizeof v);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float f = (float)v[i];
                const int d = c * 4 / kOf, y = c * 4 % kOf + i;
                o[d][y] = (lost >> (kOf * d + y)) & 1u ? fmaf(fabsf(f) < __builtin_inff() ? p : w, f, o[d][y]) : o[d][y];
              }
            }
          }
    }
  }

  // Waves on the same rows bring their sums to one maximum and the sums of all
  // waves meet in LDS, where a row's 16-byte unit u is in place u ^ key(row);
  // rows leave it whole, those of a wave's rows shared among the waves that
  // hold a part of them.  From here on the maximum stands for the lifted one.
  float2* const sm = (float2*)(lds + kSumsAt);  // [wave][R]: maxima and sums
  l_run = row_add(l_run);
  m_run -= kLift;
  if (g == 0) sm[wave * R + rl] = make_float2(m_run, l_run);
  __syncthreads();  // and the tiles have been read
  if (works) {
    float m = m_run;
    for (int w = 0; w < wt_all; ++w) m = fmaxf(m, sm[(w * wrs + wr) * R + rl].x);
    const float e = factor(m_run - (m == -__builtin_inff() ? 0.0f : m));
    float* const mine = (float*)lds + (wave * R + rl) * DP;
#pragma unroll
    for (int c = 0; c < DP / kStride; ++c) {
      const int d = c * 4 / kOf, y = c * 4 % kOf;
      f32x4 v;
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = o[d][y + i] * e;
      *(f32x4*)(mine + ((c * G + g) ^ St::key(rl & 15)) * 4) = v;
    }
  }
  __syncthreads();
  if (!works) return;
  float m = -__builtin_inff(), l = 0.0f;  // of this lane's row
  for (int w = 0; w < wt_all; ++w) m = fmaxf(m, sm[(w * wrs + wr) * R + rl].x);
  for (int w = 0; w < wt_all; ++w) {
    const float2 x = sm[(w * wrs + wr) * R + rl];
    l = fmaf(factor(x.x - (m == -__builtin_inff() ? 0.0f : m)), x.y, l);
  }
  const long long row_of = (long long)token * a.q_heads + qhead;
  if (wt == 0 && g == 0 && row_in) {
    if (!last) *(float2*)(a.part + a.part_ml + (row_of * a.pieces + it.piece) * 2) = make_float2(m, l);
    else if (a.lse) a.lse[row_of] = (m + __builtin_amdgcn_logf(l)) * 0.69314718056f;
    if (a.pieces > 1 && it.piece == 0) ((int*)(a.part + a.part_n))[row_of] = last ? 0 : used;
  }
  const float inv = !last ? 1.0f : l == 0.0f ? 0.0f : 1.0f / l;
  constexpr int kFours = DP / 4, kTogether = 64 / kFours;  // lanes of a row, rows at a time
  auto put = [&](int r0, auto one) {
    const int r = r0 + lane / kFours, u = lane % kFours;
    const long long row = __shfl(row_of, r);
    const float scale = __shfl(inv, r);
    const float* const from = (const float*)lds + (wr * R + r) * DP + (u ^ St::key(r & 15)) * 4;
    f32x4 v = *(const f32x4*)from;
    if constexpr (!decltype(one)::value)
      for (int w = 1; w < wt_all; ++w) v += *(const f32x4*)(from + w * wrs * R * DP);
    if (wr * R + r < rows_here && u * 4 < dim) {
      if (last) {
        struct alignas(8) {
          QT e[4];
        } y;
#pragma unroll
        for (int i = 0; i < 4; ++i) y.e[i] = (QT)(scale == 0.0f ? 0.0f : v[i] * scale);
        *(decltype(y)*)((QT*)a.out + row * dim + u * 4) = y;
      } else {
        *(f32x4*)(a.part + (row * a.pieces + it.piece) * dim + u * 4) = v;
      }
    }
  };
  if (wt_all == 1) {
#pragma unroll 4
    for (int n = 0; n < R / kTogether; ++n) put(n * kTogether, std::true_type{});
  } else {
#pragma unroll 1
    for (int r0 = wt * kTogether; r0 < R; r0 += wt_all * kTogether) put(r0, std::false_type{});
  }
}

// Joins the pieces of a row.  A workgroup to each (SHARED): groups of dim / 4
// lanes take every so many-th piece, and the first group adds their sums, in a
// fixed order.  Or a group to each, where there are so many rows that groups
// fill the chip.  A group's first piece is read before it is known whether
// there is one.
template <class QT, bool SHARED>
__global__ __launch_bounds__(kJoinMost) void tree_join_kernel(TreeArgs a) {
  __shared__ __align__(16) float so[SHARED ? kJoinMost * 4 : 4], sm[SHARED ? kJoinMost * 2 : 2];
  const int dim = a.c.head_dim, lanes = dim >> 2;
  const int groups = (int)blockDim.x / lanes, at = (int)threadIdx.x / lanes, t = (int)threadIdx.x - at * lanes;
  const int parts = SHARED ? groups : 1, g = SHARED ? at : 0;
  const long long rows = (long long)a.tokens * a.q_heads;
  const long long row = SHARED ? (long long)blockIdx.x : min((long long)blockIdx.x * groups + min(at, groups - 1), rows - 1);
  const float2* const ml = (const float2*)(a.part + a.part_ml) + row * a.pieces;
  const f32x4* const part = (const f32x4*)(a.part + row * a.pieces * dim) + t;
  const int n = ((const int*)(a.part + a.part_n))[row];
  const int from = min(g, a.pieces - 1);
  float2 w = ml[from];
  f32x4 v = part[(long long)from * lanes];
  if (!SHARED && (at >= groups || (long long)blockIdx.x * groups + at >= rows)) return;
  const int tok = (int)(row / a.q_heads);
  // rows that no request has (behind the last one's) hold no count
  if (tok < start_of(a, 0) || tok >= start_of(a, a.batch)) return;
  if (n <= 1 || n > a.pieces) return;
  float m = -__builtin_inff(), l = 0.0f;
  f32x4 o = {0.0f, 0.0f, 0.0f, 0.0f};
  if (g < parts && g < n) {
    m = w.x;
#pragma unroll 4
    for (int c = g + parts; c < n; c += parts) m = fmaxf(m, ml[c].x);
    const float m_use = m == -__builtin_inff() ? 0.0f : m;
    auto add = [&] {
      const float e = factor(w.x - m_use);
      l = fmaf(e, w.y, l);
#pragma unroll
      for (int j = 0; j < 4; ++j) o[j] = fmaf(e, v[j], o[j]);
    };
    add();
#pragma unroll 4
    for (int c = g + parts; c < n; c += parts) {
      w = ml[c];
      v = part[(long long)c * lanes];
      add();
    }
    if constexpr (SHARED) {
      *(f32x4*)(so + (g * lanes + t) * 4) = o;
      if (t == 0) {
        sm[2 * g] = m;
        sm[2 * g + 1] = l;
      }
    }
  }
  if constexpr (SHARED) {
    __syncthreads();
    if (g != 0) return;
    const int used = min(n, parts);
    for (int c = 1; c < used; ++c) m = fmaxf(m, sm[2 * c]);
    const float m_use = m == -__builtin_inff() ? 0.0f : m;
    l = 0.0f;
    o = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
    for (int c = 0; c < used; ++c) {
      const float e = factor(sm[2 * c] - m_use);
      const f32x4 x = *(const f32x4*)(so + (c * lanes + t) * 4);
      l = fmaf(e, sm[2 * c + 1], l);
#pragma unroll
      for (int j = 0; j < 4; ++j) o[j] = fmaf(e, x[j], o[j]);
    }
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  struct alignas(8) {
    QT e[4];
  } y;
#pragma unroll
  for (int j = 0; j < 4; ++j) y.e[j] = (QT)(l == 0.0f ? 0.0f : o[j] * inv);
  *(decltype(y)*)((QT*)a.out + row * dim + t * 4) = y;
  if (a.lse && t == 0) a.lse[row] = (m + __builtin_amdgcn_logf(l)) * 0.69314718056f;
}

// The unit files instantiate these (one file per pair of formats).
template <int Q, int F>
hipError_t launch_tree(const TreeArgs& a, bool few, dim3 grid, hipStream_t stream) {
  const int dim = a.c.head_dim;
  auto go = [&](auto dp, auto rows, auto pair) {
    constexpr int DP = decltype(dp)::value, kLds = tree_lds(DP, F == ORBIT_KV_INT8);
    auto kern = tree_kernel<Q, F, DP, decltype(rows)::value, decltype(pair)::value>;
    static LaunchCache cache;
    const hipError_t e = prepare_launch(cache, (const void*)kern, 64 * kTreeWaves, kLds, nullptr);
    if (e != hipSuccess) return e;
    kern<<<grid, dim3(64 * kTreeWaves), kLds, stream>>>(a);
    return hipGetLastError();
  };
  typedef std::integral_constant<int, 16> Narrow;
  typedef std::integral_constant<int, 32> Wide;
  if (dim <= 64) {
    const std::integral_constant<int, 64> dp;
    return few ? go(dp, Narrow{}, std::true_type{}) : go(dp, Wide{}, std::false_type{});
  }
  if (dim <= 128) {
    const std::integral_constant<int, 128> dp;
    return few ? go(dp, Narrow{}, std::true_type{}) : go(dp, Wide{}, std::false_type{});
  }
  const std::integral_constant<int, 256> dp;
  return few ? go(dp, Narrow{}, std::true_type{}) : go(dp, Narrow{}, std::false_type{});
}

hipError_t launch_tree_bf16(const TreeArgs& a, bool few, dim3 grid, hipStream_t stream);
hipError_t launch_tree_f16(const TreeArgs& a, bool few, dim3 grid, hipStream_t stream);
hipError_t launch_tree_int8(const TreeArgs& a, int q_dtype, bool few, dim3 grid, hipStream_t stream);

}  // namespace block
}  // namespace orbit
