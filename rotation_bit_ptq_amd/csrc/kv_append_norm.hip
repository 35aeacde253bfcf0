// orbit_kv_append_normed and orbit_qk_norm: queries and keys normed for each
// head, the position rotation (and the Hadamard rotation) in the same pass,
// into the paged cache or as rows.
//
// Bound: memory, or latency for few tokens; the kernel is the append's with
// the norm between the loads and the rotation (kv_append_impl.h): a head lies
// in one group of lanes, so its sums take three to five exchanges, and nothing
// is read twice but the partners of the rotation's pairs (from L1).
#include "kv_append_impl.h"

#include <cmath>

using namespace orbit;
using namespace orbit::block;
using namespace orbit::block::append;

namespace {

// The norm's arguments; heads of `dim`.
orbit_status fill_norm(const orbit_head_norm& n, AppendArgs& a) {
  if (n.norm != ORBIT_NORM_RMS && n.norm != ORBIT_NORM_LAYER) return ORBIT_E_ARG;
  if (!(n.eps >= 0.0f) || !std::isfinite(n.eps)) return ORBIT_E_ARG;
  a.norm = n.norm;
  a.eps = n.eps;
  if (!n.q_weight && !n.k_weight) return ORBIT_OK;
  if (!is_dtype(n.w_dtype)) return ORBIT_E_DTYPE;
  if (n.q_weight_stride < 0 || n.k_weight_stride < 0) return ORBIT_E_SHAPE;
  const int64_t eb = dtype_bytes(n.w_dtype);
  if (!aligned_to(n.q_weight, eb) || !aligned_to(n.k_weight, eb)) return ORBIT_E_ARG;
  a.q_weight = (const char*)n.q_weight;
  a.k_weight = (const char*)n.k_weight;
  a.q_weight_stride = n.q_weight_stride;
  a.k_weight_stride = n.k_weight_stride;
  a.w_dtype = n.w_dtype;
  a.w_vec = vector_rows(n.q_weight, n.q_weight_stride) && vector_rows(n.k_weight, n.k_weight_stride);
  return ORBIT_OK;
}

}  // namespace

extern "C" orbit_status orbit_kv_append_normed(const orbit_kv_append_args* p, const orbit_head_norm* norm, hipStream_t stream) {
  if (!p || !norm) return ORBIT_E_ARG;
  AppendArgs a = {};
  orbit_status st = fill(*p, a);
  if (st != ORBIT_OK) return st;
  if ((st = fill_norm(*norm, a)) != ORBIT_OK || p->tokens == 0) return st;
  a.qots = (long long)a.q_heads * a.c.head_dim;
  a.qohs = a.c.head_dim;
  hipError_t e;
  switch (p->in_dtype) {
    case ORBIT_BF16: e = append_by_format<__bf16, true>(a, p->cache.format, stream); break;
    case ORBIT_F16: e = append_by_format<_Float16, true>(a, p->cache.format, stream); break;
    default: e = append_by_format<float, true>(a, p->cache.format, stream);
  }
  return hip_status(e);
}

extern "C" orbit_status orbit_qk_norm(const orbit_qk_norm_args* p, hipStream_t stream) {
  if (!p) return ORBIT_E_ARG;
  if (p->tokens < 0 || p->tokens >= ORBIT_MAX_ROWS) return ORBIT_E_SHAPE;
  if (!is_dtype(p->dtype)) return ORBIT_E_DTYPE;
  const int64_t dim = p->head_dim;
  if (dim < 8 || dim > 256 || dim % 8) return ORBIT_E_SHAPE;
  if (p->q_heads < 1 || p->q_heads > 65536 || p->k_heads < 0 || p->k_heads > 65536) return ORBIT_E_SHAPE;
  const bool table = p->cos_sin != nullptr, keys = p->k_heads > 0;
  if (table && (p->rot_dim < 0 || p->rot_dim > dim || p->rot_dim % 2 || p->table_len < 1)) return ORBIT_E_SHAPE;
  if (p->hadamard && (dim & (dim - 1))) return ORBIT_E_SHAPE;
  for (int64_t s : {p->q_token_stride, p->q_head_stride, p->k_token_stride, p->k_head_stride, p->q_out_token_stride, p->q_out_head_stride,
                    p->k_out_token_stride, p->k_out_head_stride})
    if (s < 0) return ORBIT_E_SHAPE;
  AppendArgs a = {};
  const orbit_status st = fill_norm(p->norm, a);
  if (st != ORBIT_OK || p->tokens == 0) return st;
  const int64_t eb = dtype_bytes(p->dtype);
  if (!p->q || !p->q_out || !aligned_to(p->q, eb) || !aligned_to(p->q_out, eb)) return ORBIT_E_ARG;
  if (keys && (!p->k || !p->k_out || !aligned_to(p->k, eb) || !aligned_to(p->k_out, eb))) return ORBIT_E_ARG;
  if (table && (!p->positions || !aligned_to(p->positions, 8) || !aligned_to(p->cos_sin, 4))) return ORBIT_E_ARG;
  a.c.kv_heads = (int)p->k_heads;
  a.c.head_dim = (int)dim;
  a.q = (const char*)p->q;
  a.k = (const char*)p->k;
  a.q_out = (char*)p->q_out;
  a.k_out = (char*)(keys ? p->k_out : p->q_out);  // null would mean a cache
  a.positions = p->positions;
  a.cos_sin = table && p->rot_dim > 0 ? p->cos_sin : nullptr;
  a.qts = p->q_token_stride;
  a.qhs = p->q_head_stride;
  a.kts = p->k_token_stride;
  a.khs = p->k_head_stride;
  a.qots = p->q_out_token_stride;
  a.qohs = p->q_out_head_stride;
  a.kots = p->k_out_token_stride;
  a.kohs = p->k_out_head_stride;
  a.table_len = p->table_len;
  a.tokens = (uint32_t)p->tokens;
  a.q_heads = (int)p->q_heads;
  a.tasks = (int)(p->q_heads + p->k_heads);
  a.rot = a.cos_sin ? p->rot_dim : 0;
  a.half = a.rot / 2;
  a.interleaved = p->interleaved != 0;
  a.hadamard = p->hadamard != 0;
  auto vectors = [](const void* b, int64_t ts, int64_t hs) { return vector_rows(b, ts) && hs % 8 == 0; };
  a.vec = vectors(p->q, a.qts, a.qhs) && vectors(p->q_out, a.qots, a.qohs) &&
          (!keys || (vectors(p->k, a.kts, a.khs) && vectors(p->k_out, a.kots, a.kohs)));
  if (a.cos_sin) a.vec = a.vec && aligned_to(p->cos_sin, 16) && a.half % (a.interleaved ? 4 : 8) == 0;
  hipError_t e;  // (the cache's type plays no part)
  switch (p->dtype) {
    case ORBIT_BF16: e = launch_append<__bf16, __bf16, true>(a, stream); break;
    case ORBIT_F16: e = launch_append<_Float16, _Float16, true>(a, stream); break;
    default: e = launch_append<float, __bf16, true>(a, stream);
  }
  return hip_status(e);
}
