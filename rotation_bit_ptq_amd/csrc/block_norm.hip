// orbit_block_norm: argument checks and the 16-bit residual streams (see
// block_norm_impl.h for the kernel).
#include "block_norm_impl.h"

#include <cmath>

using namespace orbit;
using namespace orbit::block;

namespace {

bool is_norm(int n) { return n == ORBIT_NORM_NONE || n == ORBIT_NORM_RMS || n == ORBIT_NORM_LAYER; }

orbit_status check(const orbit_block_norm_args* p) {
  if (!p) return ORBIT_E_ARG;
  if (p->rows < 0 || p->rows >= ORBIT_MAX_ROWS || p->dim < 1 || p->dim > ORBIT_MAX_D) return ORBIT_E_SHAPE;
  if (!is_norm(p->norm) || !is_norm(p->post)) return ORBIT_E_ARG;
  if (!is_dtype(p->x_dtype)) return ORBIT_E_DTYPE;
  if (!(p->eps >= 0.0f) || !std::isfinite(p->eps)) return ORBIT_E_ARG;
  const bool branch = p->branch != nullptr, norm = p->norm != ORBIT_NORM_NONE;
  if (!branch && !norm) return ORBIT_E_ARG;
  if (!branch && (p->post != ORBIT_NORM_NONE || p->post_weight || p->gate)) return ORBIT_E_ARG;
  if (!norm && (p->weight || p->scale || p->shift)) return ORBIT_E_ARG;
  if (branch && (!is_dtype(p->branch_dtype) || (p->x_dtype != ORBIT_F32 && p->branch_dtype != p->x_dtype)))
    return ORBIT_E_DTYPE;
  if (norm && (!is_dtype(p->y_dtype) || (p->x_dtype != ORBIT_F32 && p->y_dtype != p->x_dtype)))
    return ORBIT_E_DTYPE;
  const bool mod = p->gate || p->scale || p->shift;
  if ((mod || p->weight || p->post_weight) && !is_dtype(p->p_dtype)) return ORBIT_E_DTYPE;
  if (mod && (p->groups < 1 || p->groups >= (1LL << 31))) return ORBIT_E_SHAPE;
  if (p->group_ids && !aligned_to(p->group_ids, 4)) return ORBIT_E_ARG;
  if (p->rows == 0) return ORBIT_OK;
  if (!p->x || (branch && !p->r_out) || (norm && !p->y_out)) return ORBIT_E_ARG;
  const int64_t xb = dtype_bytes(p->x_dtype), pb = dtype_bytes(p->p_dtype);
  if (!aligned_to(p->x, xb) || (branch && (!aligned_to(p->branch, dtype_bytes(p->branch_dtype)) || !aligned_to(p->r_out, xb))) ||
      (norm && !aligned_to(p->y_out, dtype_bytes(p->y_dtype))))
    return ORBIT_E_ARG;
  for (const void* q : {p->weight, p->post_weight, p->gate, p->scale, p->shift})
    if (q && !aligned_to(q, pb)) return ORBIT_E_ARG;
  if (p->x_stride < 0 || p->branch_stride < 0 || p->gate_stride < 0 || p->scale_stride < 0 || p->shift_stride < 0)
    return ORBIT_E_SHAPE;
  // output rows that overlap would race
  if (p->rows > 1 && ((branch && p->r_stride < p->dim) || (norm && p->y_stride < p->dim))) return ORBIT_E_SHAPE;
  return ORBIT_OK;
}

}  // namespace

extern "C" orbit_status orbit_block_norm(const orbit_block_norm_args* p, hipStream_t stream) {
  const orbit_status st = check(p);
  if (st != ORBIT_OK || p->rows == 0) return st;
  const bool norm = p->norm != ORBIT_NORM_NONE, mod = p->gate || p->scale || p->shift;
  NormArgs a = {};
  a.x = (const char*)p->x;
  a.branch = (const char*)p->branch;
  a.r = (char*)p->r_out;
  a.y = (char*)p->y_out;
  a.weight = (const char*)p->weight;
  a.post_weight = (const char*)p->post_weight;
  a.gate = (const char*)p->gate;
  a.scale = (const char*)p->scale;
  a.shift = (const char*)p->shift;
  a.group_ids = mod ? p->group_ids : nullptr;
  a.xs = p->x_stride;
  a.bs = p->branch_stride;
  a.rs = p->r_stride;
  a.ys = p->y_stride;
  a.gs = p->gate_stride;
  a.scs = p->scale_stride;
  a.shs = p->shift_stride;
  a.rows = (uint32_t)p->rows;
  a.groups = mod ? (uint32_t)p->groups : 1u;
  a.rows_per_group = mod ? (uint32_t)((p->rows + p->groups - 1) / p->groups) : a.rows;
  a.dim = (int)p->dim;
  a.p_dtype = p->p_dtype;
  a.norm = p->norm;
  a.post = p->post;
  a.rho = p->residual_scale;
  a.eps = p->eps;
  a.width = (float)p->dim;
  hipError_t e;
  switch (p->x_dtype) {
    case ORBIT_BF16: e = launch_norm<__bf16, __bf16, __bf16>(a, stream); break;
    case ORBIT_F16: e = launch_norm<_Float16, _Float16, _Float16>(a, stream); break;
    default: e = launch_norm_f32(a, p->branch ? p->branch_dtype : ORBIT_F32, norm ? p->y_dtype : ORBIT_F32, stream);
  }
  return hip_status(e);
}
