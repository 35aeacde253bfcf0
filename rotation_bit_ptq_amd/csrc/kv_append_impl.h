// The kernel of orbit_kv_append, orbit_kv_append_normed and orbit_qk_norm (see
// kv_cache.hip).
#pragma once

#include "kv_cache.h"

namespace orbit {
namespace block {
namespace append {

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
  // norms of queries and keys
  const char *q_weight, *k_weight;  // of w_dtype, may be null
  long long q_weight_stride, k_weight_stride;  // from head to head
  int norm, w_dtype, w_vec;
  float eps;
  char* k_out;  // keys as rows instead of into the cache (and no values)
  long long qots, qohs, kots, kohs;
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

// One vector of eight as a row holds it.
template <class T, bool VEC>
__device__ __forceinline__ void put_row(T* p, const float (&f)[8]) {
  Vec8<T> o;
#pragma unroll
  for (int j = 0; j < 8; ++j) o.e[j] = (T)f[j];
  if constexpr (VEC) {
    *(Vec8<T>*)p = o;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) p[j] = o.e[j];
  }
}

// Sum over a group of LPH lanes.
template <int LPH>
__device__ __forceinline__ float group_sum(float v) {
  v = dpp_add<kXor1>(v);
  v = dpp_add<kXor2>(v);
  v = dpp_add<kHalfMirror>(v);
  if (LPH > 8) v = dpp_add<kRowMirror>(v);
  if (LPH > 16) v = add_rows16(v);
  return v;
}

// Eight weights from element e on (those past the head: 0); none: ones.
__device__ __forceinline__ void weights8(float (&w)[8], const char* base, long long e, int left, int dtype, bool vec) {
#pragma unroll
  for (int j = 0; j < 8; ++j) w[j] = 1.0f;
  if (!base) return;
  if (dtype == ORBIT_F32) {
    const float* const p = (const float*)base + e;
    if (vec) {
      *(f32x4*)w = *(const f32x4*)p;
      *(f32x4*)(w + 4) = *(const f32x4*)(p + 4);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = j < left ? p[j] : 0.0f;
    }
    return;
  }
  Vec8<uint16_t> v;
  const uint16_t* const p = (const uint16_t*)base + e;
  if (vec) {
    v = *(const Vec8<uint16_t>*)p;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v.e[j] = j < left ? p[j] : 0;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j)
    w[j] = dtype == ORBIT_BF16 ? __builtin_bit_cast(float, (uint32_t)v.e[j] << 16) : (float)__builtin_bit_cast(_Float16, v.e[j]);
}

// A group of LPH lanes takes one head of one token: blockIdx.y the heads in
// pieces of 256 / LPH, or a workgroup several tokens where they have fewer.
// VEC: rows, partners and table rows in 16-byte words.  One head per group
// and not several in turn: fewer registers (48) keep twice the waves in
// flight, which hides the chain position -> cosines -> result (16384 tokens
// of 32 + 8 + 8 heads of 128: two heads in turn 119 us, three with all their
// loads ahead 214, one 88: 4.7 TB/s).
// NORM: queries and keys are normed first, x^ = (x - mean) / sqrt(mean (x -
// mean)^2 + eps) w (rms: without the mean), by sums over the group in float32;
// the partner of a pair is normed by the same sums and its own weight.
template <class IT, class CT, int LPH, bool VEC, bool NORM>
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
  // a group's idle lanes stay for the norm's sums
  if (token >= a.tokens || t >= a.tasks || (!NORM && e0 >= dim)) return;
  const bool idle = NORM && e0 >= dim;
  const int last_k = a.q_heads + a.c.kv_heads;
  const bool turned = a.cos_sin && t < last_k;  // this head takes the position rotation
  const bool rotated = turned && e0 < a.rot;    // and these coordinates
  const long long slot = NORM && a.k_out ? -1 : a.slots[token];
  const long long pos = a.cos_sin ? a.positions[token] : 0;

  const IT* p = t < a.q_heads ? (const IT*)a.q + token * a.qts + t * a.qhs
                : t < last_k  ? (const IT*)a.k + token * a.kts + (t - a.q_heads) * a.khs
                              : (const IT*)a.v + token * a.vts + (t - last_k) * a.vhs;
  const Vec8<IT> own = load8<IT>(p + (idle ? 0 : e0), VEC);
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
  float other[8];  // the partners
  if (rotated && !a.interleaved) {
#pragma unroll
    for (int j = 0; j < 8; ++j) other[j] = (float)pair.e[j];
  }
  if constexpr (NORM) {
    // what is written may lie where this group read
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (t < last_k) {
      float sum = 0.0f, mean = 0.0f;
      if (a.norm == ORBIT_NORM_LAYER) {
#pragma unroll
        for (int j = 0; j < 8; ++j) sum += f[j];
        mean = group_sum<LPH>(idle ? 0.0f : sum) / (float)dim;
        sum = 0.0f;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) sum = fmaf(f[j] - mean, f[j] - mean, sum);
      const float scale = 1.0f / sqrtf(group_sum<LPH>(idle ? 0.0f : sum) / (float)dim + a.eps);
      const bool query = t < a.q_heads;
      const char* const wb = query ? a.q_weight : a.k_weight;
      const long long we = query ? t * a.q_weight_stride : (t - a.q_heads) * a.k_weight_stride;
      float w[8];
      if (!idle) {
        weights8(w, wb, we + e0, 8, a.w_dtype, a.w_vec);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = (f[j] - mean) * scale * w[j];
      }
      if (rotated && !a.interleaved) {
        if constexpr (VEC) {
          weights8(w, wb, we + (e0 < a.half ? e0 + a.half : e0 - a.half), 8, a.w_dtype, a.w_vec);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int e = e0 + j, x = e < a.half ? e + a.half : e - a.half;
            float one[8];
            weights8(one, wb, we + (e < a.rot ? x : 0), 1, a.w_dtype, false);
            w[j] = one[0];
          }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) other[j] = (other[j] - mean) * scale * w[j];
      }
    }
    if (idle) return;
  }
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
      for (int j = 0; j < 8; ++j) f[j] = f[j] * c[j] + other[j] * (e0 + j < a.half ? -s[j] : s[j]);
    }
  }
  if (a.hadamard && t < last_k) hadamard<LPH>(f, lane, dim);
  if (t < a.q_heads) {
    if (!known) {
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = __builtin_nanf("");
    }
    if constexpr (NORM) put_row<IT, VEC>((IT*)a.q_out + token * a.qots + t * a.qohs + e0, f);
    else put<IT>(a.q_out, (long long)token * a.q_heads + t, dim, e0, f);
    return;
  }
  if (NORM && a.k_out) {
    if (!known) {
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = __builtin_nanf("");
    }
    put_row<IT, VEC>((IT*)a.k_out + token * a.kots + (t - a.q_heads) * a.kohs + e0, f);
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

template <class IT, class CT, bool NORM>
hipError_t launch_append(AppendArgs& a, hipStream_t stream) {
  const int lph = a.c.head_dim <= 64 ? 8 : a.c.head_dim <= 128 ? 16 : 32;
  const int groups = 256 / lph;
  a.tokens_per_block = a.tasks >= groups ? 1 : groups / a.tasks;
  const dim3 grid((a.tokens + a.tokens_per_block - 1) / a.tokens_per_block, (a.tasks + groups - 1) / groups);
  if (a.vec) {
    if (lph == 8) append_kernel<IT, CT, 8, true, NORM><<<grid, dim3(256), 0, stream>>>(a);
    else if (lph == 16) append_kernel<IT, CT, 16, true, NORM><<<grid, dim3(256), 0, stream>>>(a);
    else append_kernel<IT, CT, 32, true, NORM><<<grid, dim3(256), 0, stream>>>(a);
  } else {
    if (lph == 8) append_kernel<IT, CT, 8, false, NORM><<<grid, dim3(256), 0, stream>>>(a);
    else if (lph == 16) append_kernel<IT, CT, 16, false, NORM><<<grid, dim3(256), 0, stream>>>(a);
    else append_kernel<IT, CT, 32, false, NORM><<<grid, dim3(256), 0, stream>>>(a);
  }
  return hipGetLastError();
}

template <class IT, bool NORM>
hipError_t append_by_format(AppendArgs& a, int format, hipStream_t stream) {
  switch (format) {
    case ORBIT_KV_BF16: return launch_append<IT, __bf16, NORM>(a, stream);
    case ORBIT_KV_F16: return launch_append<IT, _Float16, NORM>(a, stream);
    default: return launch_append<IT, signed char, NORM>(a, stream);
  }
}

// What the entry points share: the checks of the arguments, and the kernel's.
orbit_status fill(const orbit_kv_append_args& p, AppendArgs& a);

}  // namespace append
}  // namespace block
}  // namespace orbit
