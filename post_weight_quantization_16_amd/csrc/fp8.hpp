// Block-scaled e4m3 matrices: device helpers shared by the 8-bit kernels.
//
// A value is code·scale, the code in e4m3 (bias 7, three mantissa bits, no
// infinities, largest 448), the scale fp32 for each block of 128 columns and
// 1 or 128 rows: s = max(fl32(amax/448), 2^-126), code = e4m3 nearest to x/s,
// ties to even.  448 reaches the last code, so nothing saturates; the lower
// limit keeps s normal (an all-zero block gets zero codes).  A block that
// holds a NaN or an infinity gets s = NaN and NaN codes, so whatever is
// computed from it is NaN.
#pragma once

#include "common.hpp"

namespace gq {

typedef __attribute__((ext_vector_type(8))) int i32x8;

constexpr int kFp8Block = 128;        // columns of a block (and rows, for weights)

// Scale of a block from its largest magnitude (NaN or infinite: NaN).  For an
// fp32 amax the product with 1/448 rounds to fp32 as the quotient does: amax/7
// is either exact in fp32 or at least 2^-28 of itself away from a border.
__device__ __forceinline__ float e4m3_scale(double amax) {
  const float s = fmaxf((float)(amax * (1.0 / 448.0)), 1.17549435e-38f);
  return __builtin_isfinite(amax) ? s : __builtin_nanf("");
}

// 1/s for e4m3_quotient, to 2^-40 or better (the estimate's 2^-20 or better,
// squared): what is left enters the quotient squared again.
__device__ __forceinline__ double e4m3_inverse(float s) {
  const double sd = (double)s, r = __builtin_amdgcn_rcp(sd);
  return __builtin_fma(__builtin_fma(-sd, r, 1.0), r, r);
}

// x as a float that rounds to 16 bits or fewer as x does: its last 32 bits
// folded into a sticky bit above them, which leaves 21 bits, a value fp32 holds
// exactly (from 2^-126 up), and keeps the side of every border.
__device__ __forceinline__ float sticky_float(double x) {
  const uint64_t b = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = (uint32_t)b, hi = (uint32_t)(b >> 32) | (lo < 1u ? lo : 1u);
  return (float)__builtin_bit_cast(double, (uint64_t)hi << 32);
}

// x/s as a float that rounds to e4m3 as the exact quotient does: the quotient
// in fp64, with one correction by the exact remainder, so ties stay ties.  fp32
// alone would move about one code in 10^6 over a border.
__device__ __forceinline__ float e4m3_quotient(double x, double s, double inv) {
  double q = x * inv;
  return sticky_float(__builtin_fma(__builtin_fma(-q, s, x), inv, q));
}

// Four floats to four e4m3 codes, byte i from argument i (round to nearest
// even; NaN stays NaN; |x| <= 464 assumed).
__device__ __forceinline__ uint32_t e4m3_pack4(float a, float b, float c, float d) {
  int r = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, r, true);
}

// Another lane's value, by a DPP control.
template <int CTRL> __device__ __forceinline__ double dpp_d(double x) {
  const uint64_t b = __builtin_bit_cast(uint64_t, x);
  const int lo = (int)(uint32_t)b, hi = (int)(uint32_t)(b >> 32);
  const uint32_t l = (uint32_t)__builtin_amdgcn_update_dpp(lo, lo, CTRL, 0xF, 0xF, false);
  const uint32_t h = (uint32_t)__builtin_amdgcn_update_dpp(hi, hi, CTRL, 0xF, 0xF, false);
  return __builtin_bit_cast(double, ((uint64_t)h << 32) | l);
}
// row_ror:n rotates inside each row of 16 lanes
constexpr int kRor8 = 0x128, kRor4 = 0x124, kRor2 = 0x122, kRor1 = 0x121;
// Maximum over the 16 lanes of a DPP row (every lane gets it).
__device__ __forceinline__ uint32_t row16_max_u32(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, kRor8, 0xF, 0xF, false));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, kRor4, 0xF, 0xF, false));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, kRor2, 0xF, 0xF, false));
  return max(v, (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, kRor1, 0xF, 0xF, false));
}

// ---------------------------------------------------------------- 16/32-bit elements
template <int DT> struct Elem;
template <> struct Elem<GPTQ_F32> {
  typedef float type;
  static __device__ __forceinline__ float up(float x) { return x; }
  static __device__ __forceinline__ float down(float x) { return x; }
};
template <> struct Elem<GPTQ_BF16> {
  typedef __bf16 type;
  static __device__ __forceinline__ float up(__bf16 x) { return (float)x; }
  static __device__ __forceinline__ __bf16 down(float x) { return (__bf16)x; }
};
template <> struct Elem<GPTQ_F16> {
  typedef _Float16 type;
  static __device__ __forceinline__ float up(_Float16 x) { return (float)x; }
  static __device__ __forceinline__ _Float16 down(float x) { return (_Float16)x; }
};

// Eight consecutive elements as stored, `n` of them present (the others are
// zero).
// Full pieces are copied whole at whatever alignment the caller's rows have:
// gfx950 loads and stores wide words at any byte address in global memory.
template <int DT>
__device__ __forceinline__ void load8_raw(const typename Elem<DT>::type* p, int n,
                                          typename Elem<DT>::type (&x)[8]) {
  typedef typename Elem<DT>::type T;
  if (n >= 8) {
    __builtin_memcpy(x, p, sizeof x);
  } else {
    // one element a load, all in flight together (a branch for each would
    // wait eight times)
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = (T)0.f;
    if (n > 0) {
      T y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = p[i < n ? i : n - 1];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = i < n ? y[i] : (T)0.f;
    }
  }
}
// The same, widened.
template <int DT>
__device__ __forceinline__ void load8(const typename Elem<DT>::type* p, int n, float (&v)[8]) {
  typename Elem<DT>::type x[8];
  load8_raw<DT>(p, n, x);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = Elem<DT>::up(x[i]);
}
template <int DT>
__device__ __forceinline__ void store8_raw(typename Elem<DT>::type* p, int n,
                                           const typename Elem<DT>::type (&x)[8]) {
  if (n >= 8) {
    __builtin_memcpy(p, x, sizeof x);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = x[i];
  }
}
template <int DT>
__device__ __forceinline__ void store8(typename Elem<DT>::type* p, int n, const float (&v)[8]) {
  typename Elem<DT>::type x[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = Elem<DT>::down(v[i]);
  store8_raw<DT>(p, n, x);
}
__device__ __forceinline__ void store_codes8(uint8_t* p, int n, uint32_t lo, uint32_t hi) {
  if (n >= 8) {
    const uint32_t x[2] = {lo, hi};
    __builtin_memcpy(p, x, 8);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = (uint8_t)((i < 4 ? lo : hi) >> (8 * (i & 3)));
  }
}

}  // namespace gq
