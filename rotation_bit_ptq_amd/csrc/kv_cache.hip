// orbit_kv_append and orbit_kv_read: tokens into the paged cache and back.
//
// Append, per token and head of dimension D:
//   a' = a cos - b sin, b' = a sin + b cos        (keys and queries)
//   x' = H_D x / sqrt(D)                          (rotated cache)
//   scale = fp16(max|x'| / 127), code = rint(x' / scale)  (INT8 cache)
//
// Bound: memory.  Eight neighbouring elements per lane (16-byte accesses),
// so a head is a group of D / 8 lanes (a power of two of them, the rest
// idle) and a wave holds several heads; the Hadamard transform is three
// register stages and log2(D / 8) exchanges between lanes of the group, the
// row maximum one reduction over it.  The other half of a pair (x[i + rot/2])
// is loaded a second time rather than exchanged: the line is in L1, and any
// rot_dim works alike.  16384 tokens of 32 + 8 + 8 heads of 128 in bf16: 88
// us (4.7 TB/s); 4099 of 24 + 4 + 4 in the int8 cache 17 us, read back 5.
#include "kv_append_impl.h"

using namespace orbit;
using namespace orbit::block;
using namespace orbit::block::append;

namespace {

struct ReadArgs {
  Cache c;
  const int64_t* slots;
  char *k, *v;
  long long vectors;  // tokens * kv_heads * (head_dim / 8)
};

// A thread takes one vector of a key and the same one of the value.
template <class CT, class OT>
__global__ __launch_bounds__(256) void read_kernel(ReadArgs a) {
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  if (i >= a.vectors) return;
  const uint32_t per_head = (uint32_t)a.c.head_dim >> 3, per_token = per_head * (uint32_t)a.c.kv_heads;
  const uint32_t token = (uint32_t)(i / per_token);
  const uint32_t rest = (uint32_t)(i - (long long)token * per_token);
  const uint32_t head = rest / per_head;
  const int e0 = (int)(rest - head * per_head) * 8;
  const long long slot = a.slots[token];
  Vec8<OT> ko, vo;
  if (slot >= 0 && slot < ((long long)a.c.pages << a.c.page_shift)) {
    const long long row = cache_row(a.c, (uint32_t)slot >> a.c.page_shift, (int)head, (uint32_t)slot & a.c.page_mask);
    const long long at = row * a.c.head_dim + e0;
    if constexpr (sizeof(CT) == 1) {
      union {
        u32x2 w;
        signed char b[8];
      } kc, vc;
      kc.w = *(const u32x2*)(a.c.k + at);
      vc.w = *(const u32x2*)(a.c.v + at);
      const float ks = (float)a.c.ks[row], vs = (float)a.c.vs[row];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        ko.e[j] = (OT)((float)kc.b[j] * ks);
        vo.e[j] = (OT)((float)vc.b[j] * vs);
      }
    } else {
      const Vec8<CT> kc = *(const Vec8<CT>*)((const CT*)a.c.k + at), vc = *(const Vec8<CT>*)((const CT*)a.c.v + at);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        ko.e[j] = (OT)(float)kc.e[j];
        vo.e[j] = (OT)(float)vc.e[j];
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) ko.e[j] = vo.e[j] = (OT)0.0f;
  }
  *(Vec8<OT>*)((OT*)a.k + i * 8) = ko;
  *(Vec8<OT>*)((OT*)a.v + i * 8) = vo;
}

template <class CT>
hipError_t launch_read(const ReadArgs& a, int out_dtype, hipStream_t stream) {
  const unsigned blocks = (unsigned)((a.vectors + 255) / 256);
  switch (out_dtype) {
    case ORBIT_BF16: read_kernel<CT, __bf16><<<dim3(blocks), dim3(256), 0, stream>>>(a); break;
    case ORBIT_F16: read_kernel<CT, _Float16><<<dim3(blocks), dim3(256), 0, stream>>>(a); break;
    default: read_kernel<CT, float><<<dim3(blocks), dim3(256), 0, stream>>>(a);
  }
  return hipGetLastError();
}

}  // namespace

orbit_status orbit::block::append::fill(const orbit_kv_append_args& args, AppendArgs& a) {
  const orbit_kv_append_args* const p = &args;
  const orbit_status st = check_cache(p->cache);
  if (st != ORBIT_OK) return st;
  if (p->tokens < 0 || p->tokens >= ORBIT_MAX_ROWS) return ORBIT_E_SHAPE;
  if (!is_dtype(p->in_dtype)) return ORBIT_E_DTYPE;
  const int dim = p->cache.head_dim;
  const bool table = p->cos_sin != nullptr, queries = p->q != nullptr;
  if (queries && (p->q_heads < 1 || p->q_heads > 65536)) return ORBIT_E_SHAPE;
  if (table && (p->rot_dim < 0 || p->rot_dim > dim || p->rot_dim % 2 || p->table_len < 1)) return ORBIT_E_SHAPE;
  if (p->hadamard && (dim & (dim - 1))) return ORBIT_E_SHAPE;
  if (p->k_token_stride < 0 || p->k_head_stride < 0 || p->v_token_stride < 0 || p->v_head_stride < 0) return ORBIT_E_SHAPE;
  if (queries && (p->q_token_stride < 0 || p->q_head_stride < 0)) return ORBIT_E_SHAPE;
  if (p->tokens == 0) return ORBIT_OK;
  const int64_t eb = dtype_bytes(p->in_dtype);
  if (!p->k || !p->v || !p->slots || !aligned_to(p->k, eb) || !aligned_to(p->v, eb) || !aligned_to(p->slots, 8)) return ORBIT_E_ARG;
  if (table && (!p->positions || !aligned_to(p->positions, 8) || !aligned_to(p->cos_sin, 4))) return ORBIT_E_ARG;
  if (queries && (!aligned_to(p->q, eb) || !p->q_out || !aligned_to(p->q_out, 16) || p->q_out == p->q)) return ORBIT_E_ARG;
  a = AppendArgs{};
  a.c = cache_of(p->cache);
  a.k = (const char*)p->k;
  a.v = (const char*)p->v;
  a.q = (const char*)p->q;
  a.q_out = (char*)p->q_out;
  a.slots = p->slots;
  a.positions = p->positions;
  a.cos_sin = table && p->rot_dim > 0 ? p->cos_sin : nullptr;
  a.kts = p->k_token_stride;
  a.khs = p->k_head_stride;
  a.vts = p->v_token_stride;
  a.vhs = p->v_head_stride;
  a.qts = p->q_token_stride;
  a.qhs = p->q_head_stride;
  a.table_len = p->table_len;
  a.tokens = (uint32_t)p->tokens;
  a.q_heads = queries ? (int)p->q_heads : 0;
  a.tasks = a.q_heads + 2 * p->cache.kv_heads;
  a.rot = a.cos_sin ? p->rot_dim : 0;
  a.half = a.rot / 2;
  a.interleaved = p->interleaved != 0;
  a.hadamard = p->hadamard != 0;
  a.vec = vector_rows(p->k, p->k_token_stride) && vector_rows(p->v, p->v_token_stride) && p->k_head_stride % 8 == 0 &&
          p->v_head_stride % 8 == 0 && (!queries || (vector_rows(p->q, p->q_token_stride) && p->q_head_stride % 8 == 0));
  // halves lie whole vectors apart, interleaved pairs take four cosines
  if (a.cos_sin) a.vec = a.vec && aligned_to(p->cos_sin, 16) && a.half % (a.interleaved ? 4 : 8) == 0;
  return ORBIT_OK;
}

extern "C" orbit_status orbit_kv_append(const orbit_kv_append_args* p, hipStream_t stream) {
  if (!p) return ORBIT_E_ARG;
  AppendArgs a = {};
  const orbit_status st = fill(*p, a);
  if (st != ORBIT_OK || p->tokens == 0) return st;
  hipError_t e;
  switch (p->in_dtype) {
    case ORBIT_BF16: e = append_by_format<__bf16, false>(a, p->cache.format, stream); break;
    case ORBIT_F16: e = append_by_format<_Float16, false>(a, p->cache.format, stream); break;
    default: e = append_by_format<float, false>(a, p->cache.format, stream);
  }
  return hip_status(e);
}

extern "C" orbit_status orbit_kv_read(const orbit_kv_cache* cache, const int64_t* slots, int64_t tokens, void* k_out,
                                      void* v_out, orbit_dtype out_dtype, hipStream_t stream) {
  if (!cache) return ORBIT_E_ARG;
  const orbit_status st = check_cache(*cache);
  if (st != ORBIT_OK) return st;
  if (!is_dtype(out_dtype)) return ORBIT_E_DTYPE;
  if (tokens < 0 || tokens >= ORBIT_MAX_ROWS) return ORBIT_E_SHAPE;
  if (tokens == 0) return ORBIT_OK;
  if (!slots || !k_out || !v_out || !aligned_to(slots, 8) || !aligned_to(k_out, 16) || !aligned_to(v_out, 16))
    return ORBIT_E_ARG;
  ReadArgs a = {};
  a.c = cache_of(*cache);
  a.slots = slots;
  a.k = (char*)k_out;
  a.v = (char*)v_out;
  a.vectors = tokens * cache->kv_heads * (cache->head_dim / 8);
  if (a.vectors >= (1LL << 32)) return ORBIT_E_SHAPE;
  hipError_t e;
  switch (cache->format) {
    case ORBIT_KV_BF16: e = launch_read<__bf16>(a, out_dtype, stream); break;
    case ORBIT_KV_F16: e = launch_read<_Float16>(a, out_dtype, stream); break;
    default: e = launch_read<signed char>(a, out_dtype, stream);
  }
  return hip_status(e);
}
