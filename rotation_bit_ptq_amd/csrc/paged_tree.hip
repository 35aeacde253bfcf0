// orbit_tree_attention: argument checks, the split, and the fp16 cache (see
// paged_tree_impl.h for the kernels).
#include "paged_tree_impl.h"

#include <cmath>

using namespace orbit;
using namespace orbit::block;

namespace orbit {
namespace block {
hipError_t launch_tree_f16(const TreeArgs& a, bool few, dim3 grid, hipStream_t stream) {
  return launch_tree<ORBIT_KV_F16, ORBIT_KV_F16>(a, few, grid, stream);
}
}  // namespace block
}  // namespace orbit

namespace {

bool sizes_ok(int64_t tokens, int64_t batch, int64_t q_heads, int64_t kv_heads, int64_t head_dim, int64_t page_size, int64_t width,
              int64_t window, int64_t sinks) {
  if (tokens < 0 || tokens >= ORBIT_MAX_ROWS || batch < 0 || batch > 65535) return false;
  if (kv_heads < 1 || kv_heads > 1024 || q_heads < 1 || q_heads > 65536 || q_heads % kv_heads) return false;
  if (tokens * (q_heads / kv_heads) >= (1LL << 30)) return false;
  if (head_dim < 8 || head_dim > 256 || head_dim % 8 || page_size < 1 || page_size > 1024) return false;
  if (width < 0 || width > (1LL << 30) / page_size) return false;
  return window >= 0 && window <= (1LL << 30) && sinks >= 0 && sinks <= (1LL << 30);
}

struct Split {
  bool few;          // 16 rows per wave, and weights in pairs
  int rows, target;  // of a workgroup; workgroups
  int64_t slots, pieces, groups;  // groups: workgroups of a key head
};

// Rows per workgroup: 16 to a wave where a request has at most 32 on average,
// and at head dimensions above 128, whose sums take the registers; otherwise
// 32 (up to 128 or 256).  Pieces: so many that the workgroups fill the units
// twice over (four times where two are resident in a unit; 16 trees of 60
// tokens after up to 8192 took 153, 109, 114, 126 us with one to four times as
// many workgroups as units), but two tiles at least (item_of).  How many a
// request may have goes by the batch's sizes, not by its own length, so that
// the workspace is known beforehand: 64 trees of 4 tokens, one after 65000 and
// 63 after 500, take 228 us, that one alone 55; beside 599 of 500, where no
// context is cut, 1124 (600 of 500: 338).
Split split_of(int64_t tokens, int64_t batch, int64_t q_heads, int64_t kv_heads, int64_t head_dim, int64_t cap, int64_t window,
               int64_t sinks, bool single) {
  Split s = {};
  const int dp = head_dim <= 64 ? 64 : head_dim <= 128 ? 128 : 256;
  const int64_t group = q_heads / kv_heads, n = batch > 0 ? (tokens + batch - 1) / batch : 0;
  s.few = n * group <= 32;
  s.rows = kTreeWaves * 16 * (s.few || dp == 256 ? 1 : 2);
  s.slots = single ? batch * ((group + s.rows - 1) / s.rows) : tokens * group / s.rows + batch;
  s.target = kUnits * (s.few && dp == 64 ? 4 : 2);
  int64_t span = cap;
  if (window > 0 && window + sinks + n < span) span = window + sinks + n;
  const int64_t most = (span + 127) / 128;
  // a batch's longest request is taken to be up to four times its average
  int64_t least = (batch + 3) / 4;
  if (tokens * group / s.rows > least) least = tokens * group / s.rows;
  if (least < 1) least = 1;
  s.pieces = (s.target + least * kv_heads - 1) / (least * kv_heads);
  if (s.pieces > most) s.pieces = most;
  // every workgroup counts the requests: not too many
  if (s.pieces < 1 || batch > 512) s.pieces = 1;
  s.groups = s.slots + (s.pieces > 1 ? s.target / kv_heads + 2 : 0);
  return s;
}

int64_t bytes_of(const Split& s, int64_t tokens, int64_t q_heads, int64_t head_dim) {
  return s.pieces == 1 ? 0 : tokens * q_heads * (s.pieces * (head_dim + 2) + 1) * 4;
}

}  // namespace

extern "C" int64_t orbit_tree_attention_workspace(int64_t tokens, int64_t batch, int64_t q_heads, int64_t kv_heads, int64_t head_dim,
                                                  int64_t page_size, int64_t table_width, int64_t window, int64_t sinks,
                                                  int32_t single) {
  if (!sizes_ok(tokens, batch, q_heads, kv_heads, head_dim, page_size, table_width, window, sinks)) return -1;
  if (tokens == 0 || batch == 0) return 0;
  return bytes_of(split_of(tokens, batch, q_heads, kv_heads, head_dim, table_width * page_size, window, sinks, single != 0), tokens,
                  q_heads, head_dim);
}

extern "C" orbit_status orbit_tree_attention(const orbit_tree_attention_args* p, hipStream_t stream) {
  if (!p) return ORBIT_E_ARG;
  const orbit_status st = check_cache(p->cache);
  if (st != ORBIT_OK) return st;
  const orbit_kv_cache& c = p->cache;
  if (!sizes_ok(p->tokens, p->batch, p->q_heads, c.kv_heads, c.head_dim, c.page_size, p->table_width, p->window, p->sinks))
    return ORBIT_E_SHAPE;
  if (p->q_dtype != ORBIT_BF16 && p->q_dtype != ORBIT_F16) return ORBIT_E_DTYPE;
  if (c.format == ORBIT_KV_BF16 && p->q_dtype != ORBIT_BF16) return ORBIT_E_DTYPE;
  if (c.format == ORBIT_KV_F16 && p->q_dtype != ORBIT_F16) return ORBIT_E_DTYPE;
  if (!std::isfinite(p->sm_scale)) return ORBIT_E_ARG;
  if (p->q_token_stride < 0 || p->q_head_stride < 0 || p->table_stride < 0) return ORBIT_E_SHAPE;
  if (p->tree && (p->tree_words < 1 || p->tree_words > 1024)) return ORBIT_E_SHAPE;
  const bool single = !p->starts;
  if (single && (p->tree || p->tokens != p->batch)) return ORBIT_E_SHAPE;  // one new token each
  if (p->tokens == 0 || p->batch == 0) return ORBIT_OK;
  if (!p->q || !p->out || !p->lengths || !aligned_to(p->out, 16) || !aligned_to(p->lengths, 4)) return ORBIT_E_ARG;
  if (!aligned_to(p->starts, 4) || !aligned_to(p->tree, 8)) return ORBIT_E_ARG;
  // the stride of one token or head says nothing
  const int64_t qts = p->tokens > 1 ? p->q_token_stride : 0, qhs = p->q_heads > 1 ? p->q_head_stride : 0;
  if (!vector_rows(p->q, qts) || qhs % 8) return ORBIT_E_ARG;
  if (p->table_width > 0 && (!p->block_table || !aligned_to(p->block_table, 4))) return ORBIT_E_ARG;
  if (p->lse && !aligned_to(p->lse, 4)) return ORBIT_E_ARG;
  const Split s = split_of(p->tokens, p->batch, p->q_heads, c.kv_heads, c.head_dim, p->table_width * c.page_size, p->window, p->sinks,
                           single);
  const int64_t need = bytes_of(s, p->tokens, p->q_heads, c.head_dim);
  if (need > 0 && (!p->workspace || !aligned_to(p->workspace, 16) || p->workspace_bytes < need)) return ORBIT_E_ARG;
  if (s.groups * c.kv_heads >= (1LL << 31)) return ORBIT_E_SHAPE;
  TreeArgs a = {};
  a.c = cache_of(c);
  a.q = (const char*)p->q;
  a.out = (char*)p->out;
  a.lse = p->lse;
  a.table = p->block_table;
  a.lengths = p->lengths;
  a.starts = p->starts;
  a.tree = (const uint64_t*)p->tree;
  a.part = (float*)p->workspace;
  a.qts = qts;
  a.qhs = qhs;
  a.table_stride = p->table_stride;
  a.part_ml = p->tokens * p->q_heads * s.pieces * (int64_t)c.head_dim;
  a.part_n = a.part_ml + p->tokens * p->q_heads * s.pieces * 2;
  a.tokens = (int)p->tokens;
  a.batch = (int)p->batch;
  a.q_heads = (int)p->q_heads;
  a.group = (int)(p->q_heads / c.kv_heads);
  a.words = p->tree ? (int)p->tree_words : 0;
  a.rows = s.rows;
  a.target = s.target;
  a.pieces = (int)s.pieces;
  a.slots = (int)s.slots;
  a.cap = c.pages > 0 ? (int)(p->table_width * c.page_size) : 0;  // no page: nothing to see
  a.window = (int)p->window;
  a.sinks = (int)p->sinks;
  a.scale_log2e = p->sm_scale * 1.44269504089f;
  const dim3 grid((unsigned)(s.groups * c.kv_heads));
  hipError_t e;
  switch (c.format) {
    case ORBIT_KV_BF16: e = launch_tree_bf16(a, s.few, grid, stream); break;
    case ORBIT_KV_F16: e = launch_tree_f16(a, s.few, grid, stream); break;
    default: e = launch_tree_int8(a, p->q_dtype, s.few, grid, stream);
  }
  if (e == hipSuccess && s.pieces > 1) {
    const int64_t rows = p->tokens * p->q_heads;
    auto join = [&](auto type) {
      typedef decltype(type) QT;
      if (rows <= 16 * kUnits) {
        tree_join_kernel<QT, true><<<dim3((unsigned)rows), dim3(kJoinMost), 0, stream>>>(a);
      } else {
        const int groups = kJoinMost / (c.head_dim / 4);
        tree_join_kernel<QT, false><<<dim3((unsigned)((rows + groups - 1) / groups)), dim3(kJoinMost), 0, stream>>>(a);
      }
    };
    if (p->q_dtype == ORBIT_BF16) join(__bf16());
    else join(_Float16());
    e = hipGetLastError();
  }
  return hip_status(e);
}
