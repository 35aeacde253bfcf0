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
#include "kv_cache.h"

using namespace orbit;
using namespace orbit::block;

namespace {

struct AppendArgs {
  Cache c;
  const char *k, *v, *q;
  char* q_out;
  const int64_t *slots, *positions;
  const float* cos_sin;
  long long kts, khs, vts, vhs, qts, qhs;
  long long table_len;
  uint32_t tokens;
  int q_heads, tasks, tokens_per_block;
  int rot, half, interleaved, hadamard;
  int vec;  // rows, partners and table rows in 16-byte words
};

template <class T>
__device__ __forceinline__ Vec8<T> load8(const T* p, bool vec) {
  Vec8<T> r;
  if (vec) {
    r = *(const Vec8<T>*)p;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) r.e[j] = p[j];
  }
  return r;
}

template <int M>
__device__ __forceinline__ float lane_xor(float v) {
  const int b = __builtin_bit_cast(int, v);
  if constexpr (M == 1) return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, b, kXor1, 0xf, 0xf, true));
  if constexpr (M == 2) return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, b, kXor2, 0xf, 0xf, true));
  return __builtin_bit_cast(float, __builtin_amdgcn_ds_swizzle(b, (M << 10) | 0x1f));
}

template <int M>
__device__ __forceinline__ void butterfly(float (&f)[8], int lane) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float o = lane_xor<M>(f[j]);
    f[j] = lane & M ? o - f[j] : f[j] + o;
  }
}

// H_D over the group's lanes, D = 8 * (lanes in use).
template <int LPH>
__device__ __forceinline__ void hadamard(float (&f)[8], int lane, int dim) {
#pragma unroll
  for (int s = 1; s < 8; s *= 2)
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (!(j & s)) {
        const float a = f[j], b = f[j | s];
        f[j] = a + b;
        f[j | s] = a - b;
      }
  if (dim > 8) butterfly<1>(f, lane);
  if (dim > 16) butterfly<2>(f, lane);
  if (dim > 32) butterfly<4>(f, lane);
  if (LPH > 8 && dim > 64) butterfly<8>(f, lane);
  if (LPH > 16 && dim > 128) butterfly<16>(f, lane);
  const float s = rsqrtf((float)dim);
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] *= s;
}

template <int M>
__device__ __forceinline__ unsigned umax_xor(unsigned v) {
  const unsigned o = __builtin_bit_cast(unsigned, lane_xor<M>(__builtin_bit_cast(float, v)));
  return v > o ? v : o;
}

// One vector of eight as the cache holds it.
template <class CT>
__device__ __forceinline__ void put(char* base, long long row, int dim, int e0, const float (&f)[8]) {
  Vec8<CT> o;
#pragma unroll
  for (int j = 0; j < 8; ++j) o.e[j] = (CT)f[j];
  *(Vec8<CT>*)((CT*)base + row * dim + e0) = o;
}

// A group of LPH lanes takes one head of one token: blockIdx.y the heads in
// pieces of 256 / LPH, or a workgroup several tokens where they have fewer.
// VEC: rows, partners and table rows in 16-byte words.  One head per group
// and not several in turn: fewer registers (48) keep twice the waves in
// flight, which hides the chain position -> cosines -> result (16384 tokens
// of 32 + 8 + 8 heads of 128: two heads in turn 119 us, three with all their
// loads ahead 214, one 88: 4.7 TB/s).
template <class IT, class CT, int LPH, bool VEC>
__global__ __launch_bounds__(256) void append_kernel(AppendArgs a) {
  constexpr int kGroups = 256 / LPH;
  const int lane = threadIdx.x & (LPH - 1), grp = threadIdx.x / LPH;
  const int dim = a.c.head_dim, e0 = lane * 8;
  int t = (int)blockIdx.y * kGroups + grp;
  uint32_t token = blockIdx.x;
  if (a.tokens_per_block > 1) {
    const int sub = grp / a.tasks;
    t = grp - sub * a.tasks;
    if (sub >= a.tokens_per_block) return;
    token = blockIdx.x * (uint32_t)a.tokens_per_block + sub;
  }
  if (token >= a.tokens || t >= a.tasks || e0 >= dim) return;
  const int last_k = a.q_heads + a.c.kv_heads;
  const bool turned = a.cos_sin && t < last_k;  // this head takes the position rotation
  const bool rotated = turned && e0 < a.rot;    // and these coordinates
  const long long slot = a.slots[token];
  const long long pos = a.cos_sin ? a.positions[token] : 0;

  const IT* p = t < a.q_heads ? (const IT*)a.q + token * a.qts + t * a.qhs
                : t < last_k  ? (const IT*)a.k + token * a.kts + (t - a.q_heads) * a.khs
                              : (const IT*)a.v + token * a.vts + (t - last_k) * a.vhs;
  const Vec8<IT> own = load8<IT>(p + e0, VEC);
  Vec8<IT> pair;
  if (rotated && !a.interleaved) {
    if constexpr (VEC) {
      pair = load8<IT>(p + (e0 < a.half ? e0 + a.half : e0 - a.half), true);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int e = e0 + j;
        pair.e[j] = e < a.half ? p[e + a.half] : e < a.rot ? p[e - a.half] : (IT)0.0f;
      }
    }
  }
  const bool known = !a.cos_sin || (pos >= 0 && pos < a.table_len);
  float f[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] = (float)own.e[j];
  if (rotated) {
    const float* row = a.cos_sin + (known ? pos : 0) * (long long)a.rot;
    if (a.interleaved) {
      float c[4], s[4];
      if constexpr (VEC) {
        *(f32x4*)c = *(const f32x4*)(row + (e0 >> 1));
        *(f32x4*)s = *(const f32x4*)(row + a.half + (e0 >> 1));
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const bool in = e0 + 2 * j < a.rot;
          c[j] = in ? row[(e0 >> 1) + j] : 1.0f;
          s[j] = in ? row[a.half + (e0 >> 1) + j] : 0.0f;
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float x = f[2 * j], y = f[2 * j + 1];
        f[2 * j] = x * c[j] - y * s[j];
        f[2 * j + 1] = x * s[j] + y * c[j];
      }
    } else {
      float c[8], s[8];
      if constexpr (VEC) {
        const int i0 = e0 < a.half ? e0 : e0 - a.half;
        *(f32x4*)c = *(const f32x4*)(row + i0);
        *(f32x4*)(c + 4) = *(const f32x4*)(row + i0 + 4);
        *(f32x4*)s = *(const f32x4*)(row + a.half + i0);
        *(f32x4*)(s + 4) = *(const f32x4*)(row + a.half + i0 + 4);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int e = e0 + j, i = e < a.half ? e : e - a.half;
          c[j] = e < a.rot ? row[i] : 1.0f;
          s[j] = e < a.rot ? row[a.half + i] : 0.0f;
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = f[j] * c[j] + (float)pair.e[j] * (e0 + j < a.half ? -s[j] : s[j]);
    }
  }
  if (a.hadamard && t < last_k) hadamard<LPH>(f, lane, dim);
  if (t < a.q_heads) {
    if (!known) {
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = __builtin_nanf("");
    }
    put<IT>(a.q_out, (long long)token * a.q_heads + t, dim, e0, f);
    return;
  }
  const long long room = (long long)a.c.pages << a.c.page_shift;
  if (slot < 0 || slot >= room || !known) return;
  const bool key = t < last_k;
  const long long row = cache_row(a.c, (uint32_t)slot >> a.c.page_shift, key ? t - a.q_heads : t - last_k,
                                  (uint32_t)slot & a.c.page_mask);
  char* const base = key ? a.c.k : a.c.v;
  if constexpr (sizeof(CT) == 1) {
    // bit patterns of |x| order like the values, infinities and NaN last
    unsigned m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const unsigned b = __builtin_bit_cast(unsigned, f[j]) & 0x7fffffffu;
      m = m > b ? m : b;
    }
    // a group's idle lanes hold no part of the head and have left: the
    // exchanges stay below the lanes in use
    const int used = dim >> 3;
    if ((used & (used - 1)) == 0) {
      if (used > 1) m = umax_xor<1>(m);
      if (used > 2) m = umax_xor<2>(m);
      if (used > 4) m = umax_xor<4>(m);
      if (LPH > 8 && used > 8) m = umax_xor<8>(m);
      if (LPH > 16 && used > 16) m = umax_xor<16>(m);
    } else {
      const int first = (threadIdx.x & 63) & ~(LPH - 1);
      unsigned all = 0;
      for (int l = 0; l < used; ++l) {
        const unsigned o = (unsigned)__shfl((int)m, first + l);
        all = all > o ? all : o;
      }
      m = all;
    }
    const _Float16 scale = (_Float16)(__builtin_bit_cast(float, m) / 127.0f);
    const float s = (float)scale;
    union {
      signed char b[8];
      u32x2 w;
    } o;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float q = s == 0.0f ? 0.0f : rintf(f[j] / s);
      o.b[j] = (signed char)(int)fminf(fmaxf(q, -127.0f), 127.0f);
    }
    *(u32x2*)(base + row * dim + e0) = o.w;
    if (lane == 0) (key ? a.c.ks : a.c.vs)[row] = scale;
  } else {
    put<CT>(base, row, dim, e0, f);
  }
}

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

template <class IT, class CT>
hipError_t launch_append(AppendArgs& a, hipStream_t stream) {
  const int lph = a.c.head_dim <= 64 ? 8 : a.c.head_dim <= 128 ? 16 : 32;
  const int groups = 256 / lph;
  a.tokens_per_block = a.tasks >= groups ? 1 : groups / a.tasks;
  const dim3 grid((a.tokens + a.tokens_per_block - 1) / a.tokens_per_block, (a.tasks + groups - 1) / groups);
  if (a.vec) {
    if (lph == 8) append_kernel<IT, CT, 8, true><<<grid, dim3(256), 0, stream>>>(a);
    else if (lph == 16) append_kernel<IT, CT, 16, true><<<grid, dim3(256), 0, stream>>>(a);
    else append_kernel<IT, CT, 32, true><<<grid, dim3(256), 0, stream>>>(a);
  } else {
    if (lph == 8) append_kernel<IT, CT, 8, false><<<grid, dim3(256), 0, stream>>>(a);
    else if (lph == 16) append_kernel<IT, CT, 16, false><<<grid, dim3(256), 0, stream>>>(a);
    else append_kernel<IT, CT, 32, false><<<grid, dim3(256), 0, stream>>>(a);
  }
  return hipGetLastError();
}

template <class IT>
hipError_t append_by_format(AppendArgs& a, int format, hipStream_t stream) {
  switch (format) {
    case ORBIT_KV_BF16: return launch_append<IT, __bf16>(a, stream);
    case ORBIT_KV_F16: return launch_append<IT, _Float16>(a, stream);
    default: return launch_append<IT, signed char>(a, stream);
  }
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

extern "C" orbit_status orbit_kv_append(const orbit_kv_append_args* p, hipStream_t stream) {
  if (!p) return ORBIT_E_ARG;
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
  AppendArgs a = {};
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
  hipError_t e;
  switch (p->in_dtype) {
    case ORBIT_BF16: e = append_by_format<__bf16>(a, p->cache.format, stream); break;
    case ORBIT_F16: e = append_by_format<_Float16>(a, p->cache.format, stream); break;
    default: e = append_by_format<float>(a, p->cache.format, stream);
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
