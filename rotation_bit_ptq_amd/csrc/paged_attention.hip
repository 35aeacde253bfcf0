// orbit_paged_attention: argument checks, the split, and the 16-bit caches
// (see paged_attention_impl.h for the kernels).
#include "paged_attention_impl.h"

#include <cmath>

using namespace orbit;
using namespace orbit::block;

namespace {

bool sizes_ok(int64_t batch, int64_t q_heads, int64_t kv_heads, int64_t head_dim, int64_t page_size, int64_t width,
              int64_t window) {
  if (batch < 0 || batch > 65535 || kv_heads < 1 || kv_heads > 1024 || q_heads < 1 || q_heads > 65536) return false;
  if (q_heads % kv_heads || head_dim < 8 || head_dim > 256 || head_dim % 8) return false;
  if (page_size < 1 || page_size > 1024 || width < 0 || width > (1LL << 30) / page_size) return false;
  return window >= 0 && window <= (1LL << 30);
}

struct Split {
  int chunk, chunks;
};

// Tokens per workgroup: whole rounds of its four waves' tiles, so many that
// the pieces of full contexts make 16 workgroups per compute unit at 512
// bytes a token (128 coordinates in 16 bits), in proportion fewer where a
// token is smaller, as a piece's start and end cost the same.  Two or three
// are resident; the others fill in for the empty pieces of requests shorter
// than the table and level the workgroups' speeds.  64 ragged requests of up
// to 8192 tokens in 16 bits: 193 us at 8, 184 at 16, 188 at 24; 16 of up to
// 65000 in int8: 147 at 6, 128 at 8, 141 at 16.
// The pieces divide the table, whatever the lengths: a table much wider than
// the contexts leaves fewer workgroups with work (requests of 2000 tokens,
// 32 / 8 heads of 128 in 16 bits, tables of 2000, 16384 and 131072 tokens: 16
// of them 37, 31 and 42 us, four 15, 15 and 20).
Split split_of(int64_t batch, int64_t q_heads, int64_t kv_heads, int64_t head_dim, int format, int64_t cap, int64_t window) {
  const int64_t round = kTile * kWaves;
  int64_t span = cap;
  if (window > 0 && window + 31 < span) span = window + 31;
  if (span < 1) span = 1;
  const int64_t rows = batch * kv_heads * ((q_heads / kv_heads + 15) / 16);
  int64_t per_unit = 16 * head_dim * (format == ORBIT_KV_INT8 ? 1 : 2) / 256;
  per_unit = per_unit < 4 ? 4 : per_unit > 16 ? 16 : per_unit;
  int64_t pieces = rows > 0 ? (kUnits * per_unit + rows - 1) / rows : 1;
  const int64_t most = (span + round - 1) / round;
  if (pieces > most) pieces = most;
  const int64_t chunk = ((span + pieces - 1) / pieces + round - 1) / round * round;
  return Split{(int)chunk, (int)((span + chunk - 1) / chunk)};
}

int64_t bytes_of(const Split& s, int64_t batch, int64_t q_heads, int64_t head_dim) {
  return s.chunks == 1 ? 0 : batch * q_heads * s.chunks * (head_dim + 2) * 4;
}

}  // namespace

extern "C" int64_t orbit_paged_attention_workspace(int64_t batch, int64_t q_heads, int64_t kv_heads, int64_t head_dim,
                                                   int64_t page_size, int64_t table_width, int64_t window, int32_t format) {
  if (!sizes_ok(batch, q_heads, kv_heads, head_dim, page_size, table_width, window)) return -1;
  if (format != ORBIT_KV_BF16 && format != ORBIT_KV_F16 && format != ORBIT_KV_INT8) return -1;
  return bytes_of(split_of(batch, q_heads, kv_heads, head_dim, format, table_width * page_size, window), batch, q_heads,
                  head_dim);
}

extern "C" orbit_status orbit_paged_attention(const orbit_paged_attention_args* p, hipStream_t stream) {
  if (!p) return ORBIT_E_ARG;
  const orbit_status st = check_cache(p->cache);
  if (st != ORBIT_OK) return st;
  const orbit_kv_cache& c = p->cache;
  if (!sizes_ok(p->batch, p->q_heads, c.kv_heads, c.head_dim, c.page_size, p->table_width, p->window))
    return ORBIT_E_SHAPE;
  if (p->q_dtype != ORBIT_BF16 && p->q_dtype != ORBIT_F16) return ORBIT_E_DTYPE;
  if (c.format == ORBIT_KV_BF16 && p->q_dtype != ORBIT_BF16) return ORBIT_E_DTYPE;
  if (c.format == ORBIT_KV_F16 && p->q_dtype != ORBIT_F16) return ORBIT_E_DTYPE;
  if (!std::isfinite(p->sm_scale)) return ORBIT_E_ARG;
  if (p->q_batch_stride < 0 || p->q_head_stride < 0 || p->table_stride < 0) return ORBIT_E_SHAPE;
  if (p->batch == 0) return ORBIT_OK;
  if (!p->q || !p->out || !p->lengths || !aligned_to(p->out, 16) || !aligned_to(p->lengths, 4)) return ORBIT_E_ARG;
  // the stride of one request or head says nothing
  const int64_t qbs = p->batch > 1 ? p->q_batch_stride : 0, qhs = p->q_heads > 1 ? p->q_head_stride : 0;
  if (!vector_rows(p->q, qbs) || qhs % 8) return ORBIT_E_ARG;
  if (p->table_width > 0 && (!p->block_table || !aligned_to(p->block_table, 4))) return ORBIT_E_ARG;
  if (p->lse && !aligned_to(p->lse, 4)) return ORBIT_E_ARG;
  const Split s = split_of(p->batch, p->q_heads, c.kv_heads, c.head_dim, c.format, p->table_width * c.page_size, p->window);
  const int64_t need = bytes_of(s, p->batch, p->q_heads, c.head_dim);
  if (need > 0 && (!p->workspace || !aligned_to(p->workspace, 16) || p->workspace_bytes < need)) return ORBIT_E_ARG;
  AttentionArgs a = {};
  a.c = cache_of(c);
  a.q = (const char*)p->q;
  a.out = (char*)p->out;
  a.lse = p->lse;
  a.table = p->block_table;
  a.lengths = p->lengths;
  a.part = (float*)p->workspace;
  a.qbs = qbs;
  a.qhs = qhs;
  a.table_stride = p->table_stride;
  a.part_ml = p->batch * p->q_heads * s.chunks * (int64_t)c.head_dim;
  a.q_heads = (int)p->q_heads;
  a.group = (int)(p->q_heads / c.kv_heads);
  a.head_blocks = (a.group + 15) / 16;
  a.chunk = s.chunk;
  a.chunks = s.chunks;
  a.cap = c.pages > 0 ? (int)(p->table_width * c.page_size) : 0;  // no page: nothing to see
  a.window = (int)p->window;
  a.scale_log2e = p->sm_scale * 1.44269504089f;
  const dim3 grid((unsigned)(c.kv_heads * a.head_blocks), (unsigned)p->batch, (unsigned)s.chunks);
  hipError_t e;
  switch (c.format) {
    case ORBIT_KV_BF16: e = launch_attend<ORBIT_KV_BF16, ORBIT_KV_BF16>(a, grid, stream); break;
    case ORBIT_KV_F16: e = launch_attend<ORBIT_KV_F16, ORBIT_KV_F16>(a, grid, stream); break;
    default: e = launch_attend_coded(a, p->q_dtype, grid, stream);
  }
  if (e == hipSuccess && s.chunks > 1) {
    const dim3 g((unsigned)p->q_heads, (unsigned)p->batch);
    if (p->q_dtype == ORBIT_BF16) join_kernel<__bf16><<<g, dim3(256), 0, stream>>>(a);
    else join_kernel<_Float16><<<g, dim3(256), 0, stream>>>(a);
    e = hipGetLastError();
  }
  return hip_status(e);
}
