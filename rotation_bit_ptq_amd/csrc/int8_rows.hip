// orbit_int8_quant_rows: rows to 8 bits with one float32 scale each, rotated
// on the way:
//   x' = Pi x (or x),  s = max|x'| / 127,  q = rint(x' * 127 / max|x'|).
//
// Bound: vector instructions, in one pass over memory: a row stays in registers
// between the rotation, its maximum and its codes.  4096 bf16 rows of 3072,
// blocks of 128: 17 us (2.2 TB/s); 16 such rows 4.6 us; not rotated 9.6 us.
//
// A workgroup takes a row at a time, a wave of it 1024 coordinates: lane l
// holds coordinates 16 l .. 16 l + 15 of those, so that four of the Hadamard's
// stages are in registers, six between lanes, and codes leave as 16-byte
// words.  Blocks of 2048 and 4096 take their last two stages between the
// waves, through LDS.  The gather goes through an LDS copy of the row; its
// offsets (with the signs) are kept in registers for all rows of a workgroup.
// Rows of 4352 (9164, fp16) take 67 us, of 6336 (13404, fp16) 124, of 12288
// (4096, bf16) 83, of 16384 (2048, float32) 63.
//
// Rows of every type are rotated in float64.  In float32 the sums of 16-bit
// values are not exact either (terms some 2^9 below a block's largest lose
// bits), which moved some 10^-6 of the codes across a half, and finite bfloat16
// rows left its range; it took 14 us for the 4096 rows above.
//
// Codes: t = fma(x', 127 / max, 1.5 * 2^8) in float64 is 127 x' / max to 44
// bits behind the point, t + 1.5 * 2^52 - 1.5 * 2^8 holds that, rounded half to
// even, in its low byte (|x'| <= max, so there is nothing to clamp).  16-bit rows
// have ties (one of 10^4 codes of unrotated bf16 rows); the factor's rounding,
// 2^-46 here, would decide them, and is gone with what lies behind 44 bits.
// A row with an infinity or a NaN takes s = NaN and codes 0, so that all that
// is made of it is NaN.
#include "block_common.h"
#include "int8_rows.h"

using namespace orbit;
using namespace orbit::block;

namespace {

template <int M>
__device__ __forceinline__ int lane_xor(int b) {
  if constexpr (M == 1) return __builtin_amdgcn_update_dpp(0, b, kXor1, 0xf, 0xf, true);
  if constexpr (M == 2) return __builtin_amdgcn_update_dpp(0, b, kXor2, 0xf, 0xf, true);
  return __builtin_amdgcn_ds_swizzle(b, (M << 10) | 0x1f);
}
typedef int i32x2 __attribute__((ext_vector_type(2)));
template <int M>
__device__ __forceinline__ double lane_xor(double v) {
  const i32x2 b = __builtin_bit_cast(i32x2, v);
  return __builtin_bit_cast(double, i32x2{lane_xor<M>(b.x), lane_xor<M>(b.y)});
}
// with the sign bit flipped where `sign` is 2^31
__device__ __forceinline__ float flipped(float v, uint32_t sign) { return __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, v) ^ sign); }
// Between lanes the upper one of a pair, whose result is the other's less its own, takes its own less the other's: one
// product and sum in place.  A lane's coordinates are then negated where it was an upper one an odd number of times.
template <int M>
__device__ __forceinline__ void butterfly(double (&f)[16], int lane) {
  const double sign = lane & M ? -1.0 : 1.0;
#pragma unroll
  for (int j = 0; j < 16; ++j) f[j] = __builtin_fma(lane_xor<M>(f[j]), sign, f[j]);
}
// of lane l % 32 and of lane 32 + l % 32
__device__ __forceinline__ void halves(double v, double& lo, double& hi) {
  const i32x2 b = __builtin_bit_cast(i32x2, v);
  const auto x = __builtin_amdgcn_permlane32_swap((unsigned)b.x, (unsigned)b.x, false, false);
  const auto y = __builtin_amdgcn_permlane32_swap((unsigned)b.y, (unsigned)b.y, false, false);
  lo = __builtin_bit_cast(double, i32x2{(int)x[0], (int)y[0]});
  hi = __builtin_bit_cast(double, i32x2{(int)x[1], (int)y[1]});
}
__device__ __forceinline__ void butterfly32(double (&f)[16], int lane) {
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    double lo, hi;
    halves(f[j], lo, hi);
    f[j] = lane & 32 ? hi - lo : lo + hi;
  }
}

// Magnitudes as bit patterns, which order like the values, infinities and NaN last.
__device__ __forceinline__ uint32_t size_of(float v) { return __builtin_bit_cast(uint32_t, v) & 0x7fffffffu; }
__device__ __forceinline__ uint64_t size_of(double v) { return __builtin_bit_cast(uint64_t, v) & 0x7fffffffffffffffull; }
__device__ __forceinline__ double value_of(uint32_t b) { return (double)__builtin_bit_cast(float, b); }
__device__ __forceinline__ double value_of(uint64_t b) { return __builtin_bit_cast(double, b); }
__device__ __forceinline__ uint32_t other_lane(uint32_t b, int s) { return (uint32_t)__shfl_xor((int)b, s); }
__device__ __forceinline__ uint64_t other_lane(uint64_t b, int s) { return (uint64_t)__shfl_xor((long long)b, s); }

// A barrier for LDS alone: loads and stores of memory may be on their way.
__device__ __forceinline__ void meet() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// What rows are rotated in: 64 bits hold a block's sums without loss (fp16, and bfloat16 values
// within 2^33 of each other in blocks of 4096) and without leaving their range.
template <bool ROT>
using Sum = std::conditional_t<ROT, double, float>;

// A wave for each 1024 coordinates of a row, up to 16.
template <class IT, bool ROT>
__global__ __launch_bounds__(1024, 5) void rows_kernel(Int8RowArgs a) {
  extern __shared__ __align__(16) char smem[];
  typedef Sum<ROT> A;
  typedef decltype(size_of(A())) Size;
  Size* const top = (Size*)(smem + a.lds_row);  // the waves' maxima, behind the row's copy
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6, waves = (int)blockDim.x >> 6;
  const bool negated = ROT && __popc(lane & ((a.h >> 4) - 1)) & 1;  // see butterfly
  // where each coordinate comes from (times two, in 15 bits), bit 15: with its sign flipped
  uint32_t from[8];
  if constexpr (ROT) {
    const int k0 = wave * 1024 + lane * 16;
#pragma unroll
    for (int j = 0; j < 8; ++j) from[j] = 0;
    if (k0 < a.d) {
      const uint32_t sign = a.sign_bits[k0 >> 5] >> (k0 & 31);
#pragma unroll
      for (int j = 0; j < 16; ++j)
        from[j >> 1] |= ((uint32_t)a.perm[k0 + j] << 1 | ((sign >> j) & 1u) << 15) << (16 * (j & 1));
    }
  }
  const IT* const base = (const IT*)a.in;
  for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const IT* const x = base + row * a.stride;
    A f[16];
    if constexpr (ROT) {
      IT* const copy = (IT*)smem;
#pragma unroll
      for (int j = 0; j < 8; ++j) asm volatile("" : "+v"(from[j]));  // what is made of them is not kept in registers
      if (a.vec) {
        for (int i = t * 8; i < a.d; i += (int)blockDim.x * 8) *(Vec8<IT>*)(copy + i) = *(const Vec8<IT>*)(x + i);
      } else {
        for (int i = t; i < a.d; i += (int)blockDim.x) copy[i] = x[i];
      }
      meet();
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const uint32_t w = from[j >> 1] >> (16 * (j & 1));
        if constexpr (sizeof(IT) == 2) {
          const uint16_t v = *(const uint16_t*)(smem + (w & 0x7fffu));
          f[j] = (float)__builtin_bit_cast(IT, (uint16_t)(v ^ (w & 0x8000u)));
        } else {
          f[j] = flipped(*(const float*)(smem + (w & 0x7fffu) * 2), (w & 0x8000u) << 16);
        }
      }
    } else {
      const int k0 = wave * 1024 + lane * 16;
      Vec8<IT> v[2];
      if (k0 < a.d) {
        if (a.vec) {
          v[0] = *(const Vec8<IT>*)(x + k0);
          v[1] = *(const Vec8<IT>*)(x + k0 + 8);
        } else {
#pragma unroll
          for (int j = 0; j < 16; ++j) v[j >> 3].e[j & 7] = x[k0 + j];
        }
      }
#pragma unroll
      for (int j = 0; j < 16; ++j) f[j] = k0 < a.d ? (A)v[j >> 3].e[j & 7] : (A)0;
    }
    Size m = 0;
    if constexpr (ROT) {
      // lanes past the row hold the first coordinate again, and whole blocks of it: cleared below
#pragma unroll
      for (int s = 1; s < 16; s *= 2)
#pragma unroll
        for (int j = 0; j < 16; ++j)
          if (!(j & s)) {
            const A p = f[j], q = f[j | s];
            f[j] = p + q;
            f[j | s] = p - q;
          }
      if (a.h > 16) butterfly<1>(f, lane);
      if (a.h > 32) butterfly<2>(f, lane);
      if (a.h > 64) butterfly<4>(f, lane);
      if (a.h > 128) butterfly<8>(f, lane);
      if (a.h > 256) butterfly<16>(f, lane);
      if (a.h > 512) butterfly32(f, lane);
#pragma unroll 1
      for (int s = 1; s * 1024 < a.h; s *= 2) {  // between neighbouring waves
        A* const all = (A*)smem;                 // [wave][j][lane], over the row's copy
        meet();
#pragma unroll
        for (int j = 0; j < 16; ++j) all[(wave * 16 + j) * 64 + lane] = f[j];
        meet();
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const A o = all[((wave ^ s) * 16 + j) * 64 + lane];
          f[j] = wave & s ? o - f[j] : f[j] + o;
        }
      }
    }
    if constexpr (ROT) {
      // an infinity or a NaN makes each coordinate of its block one, a lane's first among them
      double most = 0.0;
#pragma unroll
      for (int j = 0; j < 16; ++j) most = __builtin_fmax(most, __builtin_fabs(f[j]));
      m = size_of(f[0] - f[0] == 0.0 ? most : __builtin_inf());
    } else {
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const Size b = size_of(f[j]);
        m = b > m ? b : m;
      }
    }
    if (wave * 1024 + lane * 16 >= a.d) m = 0;
#pragma unroll
    for (int s = 1; s < 64; s *= 2) {
      const Size o = other_lane(m, s);
      m = o > m ? o : m;
    }
    if (waves > 1) {
      if (lane == 0) top[wave] = m;
      meet();  // and every lane has gathered: the copy may be overwritten
      m = top[0];
      for (int w = 1; w < waves; ++w) m = top[w] > m ? top[w] : m;
    }
    const double most = value_of(m);
    const bool fine = most < __builtin_inf();
    const float scale = fine ? (float)(most * a.inv_sqrt_h / 127.0) : __builtin_nanf("");
    if (t == 0) a.s_out[row] = scale;
    const double inv = scale > 0.0f ? (ROT && negated ? -127.0 : 127.0) / most : 0.0;
    const uint32_t keep = fine ? 0xffffffffu : 0u;
    const int k0 = wave * 1024 + lane * 16;
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t b[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) b[i] = (uint32_t)__builtin_bit_cast(uint64_t, __builtin_fma((double)f[4 * j + i], inv, 384.0) + (6755399441055744.0 - 384.0));
      const uint32_t lo = __builtin_amdgcn_perm(b[1], b[0], 0x0c0c0400u), hi = __builtin_amdgcn_perm(b[3], b[2], 0x04000c0cu);
      w[j] = (lo | hi) & keep;
    }
    if (k0 < a.d) *(u32x4*)(a.q_out + row * a.d + k0) = u32x4{w[0], w[1], w[2], w[3]};
    if (ROT || waves > 1) meet();  // the row's copy and the maxima have been read
  }
}

template <class IT, bool ROT>
hipError_t launch(Int8RowArgs a, hipStream_t stream) {
  const int waves = (a.d + 1023) / 1024;
  int lds = 0;
  if (ROT) {
    lds = a.d * (int)sizeof(IT);
    const int all = waves * 1024 * (int)sizeof(double);
    if (a.h > 1024 && lds < all) lds = all;
  }
  a.lds_row = lds;
  lds += 16 * 8;
  // as many workgroups as are resident (five waves to a SIMD, by their registers:
  // 51.0 us with the product, 52.8 with 24 waves to a unit), so that the offsets are read
  // once for many rows; unrotated rows have none to keep
  const long long cap = ROT ? (long long)kUnits * (20 / waves) : a.rows;
  const dim3 grid((unsigned)(a.rows < cap ? a.rows : cap)), block(64 * waves);
  auto kern = rows_kernel<IT, ROT>;
  static LaunchCache cache;
  const hipError_t e = prepare_launch(cache, (const void*)kern, 64 * waves, lds, nullptr);
  if (e != hipSuccess) return e;
  kern<<<grid, block, lds, stream>>>(a);
  return hipGetLastError();
}

}  // namespace

namespace orbit {
hipError_t launch_int8_rows(const Int8RowArgs& a, int dtype, bool rotated, hipStream_t stream) {
  switch (dtype) {
    case ORBIT_BF16: return rotated ? launch<__bf16, true>(a, stream) : launch<__bf16, false>(a, stream);
    case ORBIT_F16: return rotated ? launch<_Float16, true>(a, stream) : launch<_Float16, false>(a, stream);
    default: return rotated ? launch<float, true>(a, stream) : launch<float, false>(a, stream);
  }
}
}  // namespace orbit
