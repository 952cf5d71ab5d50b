// Kernels of the products of block-scaled e4m3 matrices (fp8.hpp has the
// format):
//   C[m,n] = Σ_kb sa[m,kb]·sb[n/128,kb]·Σ_{k in kb} a[m,k]·b[n,k],
// the gated projection act(A·Gᵀ)·(A·Uᵀ), and act(A·Bᵀ + bias) + residual,
// rounded to 16 or 32 bits or quantized again in 1 x 128 blocks; the first two
// also for rows that are sorted by expert, each with its expert's weights.
//
// A block of 128 along K is contracted on the matrix cores from a zero
// accumulator and comes in with one fma a value: acc += t·(sa·sb).  The
// weights are the instruction's first operand: a lane then holds one row m of
// C (its lane % 16) and four neighbouring columns n (4·(lane / 16) + 0..3), so
// sa is one register and four outputs are stored together.  Any order of k
// inside a block gives the same sum if both operands agree on it: lane l
// takes bytes 16·(l / 16).. and 64 + 16·(l / 16).. of its row's block.
//
// Two ways to contract a block:
//   fast   one v_mfma_f32_16x16x128_f8f6f4.  It aligns every eight
//          neighbouring products to the power of two of the largest, cuts the
//          others (toward zero) below 2^-13 of it, and adds the eights in
//          fp32 (the powers of two are those of the factors, 2^-6 for a
//          subnormal code, so beside one of these it cuts up to 2^3 higher).
//          Measured, an error of 1.5e-5 of the result's norm on normal
//          data and 3e-5 to 6e-5 where one column in fifty is an outlier.
//          Taken where C has 16 bits: beside the norm of C's own rounding
//          (fp16 2.1e-4, bf16 1.7e-3) that adds 1 to 4 % and nothing.  It is
//          a bound on the whole, not on each value: where a sum cancels, what
//          is cut can exceed the value's own half step (in about one of
//          twenty values in fp16, one of two hundred in bf16).
//   exact  e4m3 -> fp16 (every value is exact) in registers and four
//          v_mfma_f32_16x16x32_f16: products exact, sums in fp32 (measured
//          below 5·2^-24 of Σ|a||b| a block), at half the rate.  Taken for
//          fp32 results and for 8-bit ones, whose scales are fp32.
#pragma once

#include "fp8.hpp"

namespace gq {
namespace {

typedef __attribute__((ext_vector_type(2))) _Float16 f16x2;
typedef __attribute__((ext_vector_type(4))) int i32x4;

struct GArgs {
  const uint8_t* A; const float* sa; int64_t M, K, lda;
  const uint8_t* B[2]; const float* sb[2]; int64_t N, ldb[2];   // gate and up, or B alone
  void* C; int64_t ldc; int c_dt, act;
  uint8_t* codes; int64_t ld_codes; float* sc; int64_t nb;      // nb = blocks of N
  float* P;          // split-K partials [splits][1 or 2][M][N]
  int kb, kper;      // blocks of K, and of one split
  int tm, tn;        // tiles
  int wide;          // every row of A and B starts at a multiple of 16 bytes
  // kLinear: bias [N] or null, residual [M x N] of C's type or null; act < 0: none
  const void* bias; int bias_dt; const void* R; int64_t ldr;
  // rows sorted by expert: expert e has positions offsets[e] .. offsets[e+1],
  // position i the slot order[i] = token·topk + j
  const int32_t* offsets; const int32_t* order;
  int E, topk, slots;
  int64_t next[2];   // bytes from an expert's weights to the next one's
  int group;         // kScaled: columns that share a power of two
};

// What is computed: C = A·Bᵀ, act(A·Gᵀ)·(A·Uᵀ), act(A·Bᵀ + bias) + residual.
enum { kPlain = 0, kGated = 1, kLinear = 2 };
// Which rows of A a tile multiplies: neighbouring ones of one matrix; those of
// one expert's tokens, gathered; or neighbouring ones that are sorted by expert,
// their partial sums stored at their slots.
enum { kDense = 0, kGather = 1, kSorted = 2 };
// Elements of fp16 that hold n of them, the fp32 numbers behind them aligned.
__host__ __device__ inline int64_t align_scaled(int64_t n) { return (n + 7) / 8 * 8; }

// ---------------------------------------------------------------- a block's contraction
// 128 bytes of a row, this lane's 32 of them.
template <bool FAST> struct Frag;
template <> struct Frag<true> {
  i32x8 v;
  __device__ __forceinline__ void set(const i32x4& x, const i32x4& y) {
    v = __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
  }
};
template <> struct Frag<false> {
  f16x8 v[4];
  static __device__ __forceinline__ f16x8 up(int lo, int hi) {
    const f16x2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.f, false);
    const f16x2 b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.f, true);
    const f16x2 c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.f, false);
    const f16x2 d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.f, true);
    return f16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
  }
  __device__ __forceinline__ void set(const i32x4& x, const i32x4& y) {
    v[0] = up(x[0], x[1]); v[1] = up(x[2], x[3]);
    v[2] = up(y[0], y[1]); v[3] = up(y[2], y[3]);
  }
};
// q[g] = the block's products of b[g] and a
template <int G>
__device__ __forceinline__ void contract(const Frag<true>* b, const Frag<true>& a, f32x4 (&q)[G]) {
#pragma unroll
  for (int g = 0; g < G; ++g)
    q[g] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b[g].v, a.v, f32x4{0.f, 0.f, 0.f, 0.f}, 0,
                                                            0, 0, 0, 0, 0);
}
template <int G>
__device__ __forceinline__ void contract(const Frag<false>* b, const Frag<false>& a, f32x4 (&q)[G]) {
#pragma unroll
  for (int g = 0; g < G; ++g) q[g] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int g = 0; g < G; ++g)
      q[g] = __builtin_amdgcn_mfma_f32_16x16x32_f16(b[g].v[i], a.v[i], q[g], 0, 0, 0);
}

// 16 bytes of a row from byte k on, zeros past the row's K bytes.  A piece that
// K cuts is loaded so that it ends at K, and shifted.
__device__ __forceinline__ i32x4 piece16(const uint8_t* row, int64_t k, int64_t K) {
  i32x4 v = {0, 0, 0, 0};
  if (k >= K) return v;
  if (K >= 16) {
    const int cut = (int)max((int64_t)0, k + 16 - K);   // bytes past K
    uint64_t q[2];
    __builtin_memcpy(q, row + k - cut, 16);
    const int sh = 8 * (cut & 7);
    if (cut >= 8) {
      q[0] = q[1];
      q[1] = 0;
    }
    if (sh) q[0] = (q[0] >> sh) | (q[1] << (64 - sh));
    q[1] >>= sh;
    v = i32x4{(int)(uint32_t)q[0], (int)(uint32_t)(q[0] >> 32), (int)(uint32_t)q[1], (int)(uint32_t)(q[1] >> 32)};
  } else {
    uint64_t q[2] = {0, 0};   // k == 0
#pragma unroll 1
    for (int i = 0; i < (int)K; ++i) {
      const uint64_t x = (uint64_t)row[i] << (8 * (i & 7));
      if (i < 8) q[0] |= x; else q[1] |= x;
    }
    v = i32x4{(int)(uint32_t)q[0], (int)(uint32_t)(q[0] >> 32), (int)(uint32_t)q[1], (int)(uint32_t)(q[1] >> 32)};
  }
  return v;
}

// The source of a wide copy past a row's end, where K ends between two pieces
// of 16 bytes: zeros.
__device__ const uint32_t kNothing[4] __attribute__((aligned(16))) = {0, 0, 0, 0};
__device__ __forceinline__ const uint8_t* within(const uint8_t* p, bool inside) {
  return inside ? p : reinterpret_cast<const uint8_t*>(kNothing);
}

// ---------------------------------------------------------------- epilogues
// Sigmoids by the hardware's exp2 and reciprocal.  What counts is the rounding
// of the exponent: silu is within |x| + 4 units of 2^-23, gelu_tanh, whose
// exponent is 1.6x + 0.07x³ after three roundings, within 2.5|x| + |x|³/9 + 4
// (15 at -3, 81 at -8), of values that e^-|x| makes small there.
__device__ __forceinline__ float over_one_plus_exp2(float x, float z) {   // x/(1 + 2^z)
  return x * __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(z));
}
__device__ __forceinline__ float activate(float x, int act) {
  if (act == GPTQ_ACT_SILU) return over_one_plus_exp2(x, x * -1.44269504f);
  if (act == GPTQ_ACT_GELU) return 0.5f * x * erfcf(x * -0.70710678f);   // Φ(x) without cancellation
  return over_one_plus_exp2(x, -2.30220820f * (x + 0.044715f * x * x * x));   // (1 + tanh y)/2 = 1/(1 + e^-2y)
}

// The same for many values in registers.  silu and gelu_tanh are one formula,
// x/(1 + 2^(x·(a + b·x²))), so their values need no jumps; gelu's code stands
// apart.  A choice at every value made the code longer than the instruction
// cache: 4096 x 16384 x 4096 with gelu_tanh 344 us, this way 293.  (x² is limited
// so that 0·x² stays 0.)
struct Activation {
  int act;
  float a, b;
  __device__ __forceinline__ explicit Activation(int k)
      : act(k), a(k == GPTQ_ACT_SILU ? -1.44269504f : -2.30220820f),
        b(k == GPTQ_ACT_SILU ? 0.f : -2.30220820f * 0.044715f) {}
  __device__ __forceinline__ f32x4 operator()(f32x4 x) const {
    if (__builtin_expect(act == GPTQ_ACT_GELU, 0)) {
#pragma unroll
      for (int r = 0; r < 4; ++r) x[r] = activate(x[r], GPTQ_ACT_GELU);
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        x[r] = over_one_plus_exp2(x[r], x[r] * __builtin_fmaf(fminf(x[r] * x[r], 1e38f), b, a));
    }
    return x;
  }
};

// Codes of four values of a block.  1/s and the product round by 2^-24 each, so
// a code is that of the fp32 value over its scale but within 2^-22 of a border.
// The values and the block's largest, its scale, carry fp32's rounding already;
// one more in the quotient moves no more codes over a border (1024 x 8192 x
// 2048: 50 of 8.4 million differ from those of exact sums, 49 with quotients in
// fp64, which took 1487 us where this takes 1447, 2048 x 28672 x 8192 to codes).
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d, float inv) {
  return e4m3_pack4(a * inv, b * inv, c * inv, d * inv);
}

// The same with quotients to within 2^-24 (one correction by the remainder): a
// code differs from that of the exact quotient only next to a border.
__device__ __forceinline__ float near_quotient(float x, float s, float inv) {
  const float q = x * inv;
  return __builtin_fmaf(__builtin_fmaf(-q, s, x), inv, q);
}
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d, float s, float inv) {
  return e4m3_pack4(near_quotient(a, s, inv), near_quotient(b, s, inv), near_quotient(c, s, inv),
                    near_quotient(d, s, inv));
}

// Four neighbouring values of a row, `n` of them present.
template <int DT> __device__ __forceinline__ void put4(void* C, int64_t at, int n, const f32x4& x) {
  typedef typename Elem<DT>::type T;
  T v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = Elem<DT>::down(x[i]);
  T* p = static_cast<T*>(C) + at;
  if (n >= 4) {
    __builtin_memcpy(p, v, sizeof v);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) p[i] = v[i];
  }
}
// The same for two tiles that are 16 columns apart, of a 16-bit type: the odd
// quarters of the wave change their columns of the first for the even ones' of the
// second, so that a lane stores eight neighbouring columns (the first of them
// eight_at(lane) from the first tile's own first) and the wave 64 bytes of a row in
// place of 32: stores into many rows cost by their number (products to bf16, 8192 x
// 8192 x 1024: 96.4 -> 82.4 us, 4096 x 16384 x 4096: 262.5 -> 248.4).  All lanes take
// part; n counts from the lane's first column, none for a row that does not exist.
// One wide store, written as such: as eight elements the compiler takes it apart.
__device__ __forceinline__ int eight_at(int lane) { return 16 * (lane >> 4 & 1) + 8 * (lane >> 5); }
template <int DT>
__device__ __forceinline__ void put8(void* C, int64_t at, int n, const f32x4& x, const f32x4& y) {
  typedef typename Elem<DT>::type T;
  T v[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = Elem<DT>::down(x[i]);
    v[4 + i] = Elem<DT>::down(y[i]);
  }
  unsigned u[4];
  __builtin_memcpy(u, v, sizeof u);
  const auto lo = __builtin_amdgcn_permlane16_swap(u[0], u[2], false, false);
  const auto hi = __builtin_amdgcn_permlane16_swap(u[1], u[3], false, false);
  const i32x4 w = {(int)lo[0], (int)hi[0], (int)lo[1], (int)hi[1]};
  T* p = static_cast<T*>(C) + at;
  if (n >= 8) {
    __builtin_memcpy(p, &w, sizeof w);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint16_t h = (uint16_t)((unsigned)w[i / 2] >> (16 * (i & 1)));
      if (i < n) __builtin_memcpy(p + i, &h, sizeof h);
    }
  }
}
// The way back: eight neighbouring columns of a lane, those past n zeros, added to
// its columns of the two tiles.
template <int DT> __device__ __forceinline__ i32x4 get8_of(const void* p, int64_t at, int n) {
  typedef typename Elem<DT>::type T;
  const T* q = static_cast<const T*>(p) + at;
  i32x4 w = {0, 0, 0, 0};
  if (n >= 8) {
    __builtin_memcpy(&w, q, sizeof w);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint16_t h = 0;
      if (i < n) __builtin_memcpy(&h, q + i, sizeof h);
      w[i / 2] |= (int)((unsigned)h << (16 * (i & 1)));
    }
  }
  return w;
}
template <int DT> __device__ __forceinline__ void add8(const i32x4& w, f32x4& x, f32x4& y) {
  typedef typename Elem<DT>::type T;
  const auto lo = __builtin_amdgcn_permlane16_swap((unsigned)w[0], (unsigned)w[2], false, false);
  const auto hi = __builtin_amdgcn_permlane16_swap((unsigned)w[1], (unsigned)w[3], false, false);
  const unsigned u[4] = {lo[0], hi[0], lo[1], hi[1]};
  T v[8];
  __builtin_memcpy(v, u, sizeof v);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[i] += Elem<DT>::up(v[i]);
    y[i] += Elem<DT>::up(v[4 + i]);
  }
}
// Piece i of the rows of a wave's sums, NO tiles of columns, n of them present; at:
// of the lane's row, the wave's first column.
template <int DT, int NO, int NI, int MI>
__device__ __forceinline__ void put_row(void* C, int64_t at, int n, const f32x4 (&acc)[NI][MI], int i, int lane) {
  if constexpr (DT != GPTQ_F32 && NO % 2 == 0) {
#pragma unroll
    for (int j = 0; j < NO; j += 2) {
      const int c = j * 16 + eight_at(lane);
      put8<DT>(C, at + c, n - c, acc[j][i], acc[j + 1][i]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < NO; ++j) {
      const int c = j * 16 + 4 * (lane >> 4);
      put4<DT>(C, at + c, n - c, acc[j][i]);
    }
  }
}
// Four neighbouring elements of type dt, widened; those past n are zeros.
template <int DT> __device__ __forceinline__ f32x4 get4_of(const void* p, int64_t at, int n) {
  typedef typename Elem<DT>::type T;
  const T* q = static_cast<const T*>(p) + at;
  T v[4] = {(T)0.f, (T)0.f, (T)0.f, (T)0.f};
  if (n >= 4) {
    __builtin_memcpy(v, q, sizeof v);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) v[i] = q[i];
  }
  return f32x4{Elem<DT>::up(v[0]), Elem<DT>::up(v[1]), Elem<DT>::up(v[2]), Elem<DT>::up(v[3])};
}
__device__ __forceinline__ f32x4 get4(const void* p, int dt, int64_t at, int n) {
  if (dt == GPTQ_F32) return get4_of<GPTQ_F32>(p, at, n);
  return dt == GPTQ_BF16 ? get4_of<GPTQ_BF16>(p, at, n) : get4_of<GPTQ_F16>(p, at, n);
}
__device__ __forceinline__ void put1(void* p, int dt, int64_t at, float x) {
  if (dt == GPTQ_F32) static_cast<float*>(p)[at] = x;
  else if (dt == GPTQ_BF16) static_cast<__bf16*>(p)[at] = (__bf16)x;
  else static_cast<_Float16*>(p)[at] = (_Float16)x;
}
// The largest of the four values that lanes 16 apart hold, in all of them.
__device__ __forceinline__ uint32_t quarters_max(uint32_t v) {
  const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  v = max(a[0], a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return max(b[0], b[1]);
}
// The largest of m, |a| and |b|, without what is NaN.
__device__ __forceinline__ float largest(float m, float a, float b) {
  asm("v_max3_f32 %0, %0, |%1|, |%2|" : "+v"(m) : "v"(a), "v"(b));
  return m;
}
// Magnitudes as integers: finite < infinity < NaN.
__device__ __forceinline__ uint32_t mag_bits(float x) {
  return __builtin_bit_cast(uint32_t, x) & 0x7FFFFFFFu;
}

// ---------------------------------------------------------------- tile kernel
// Bound: 4096 x 28672 x 8192 to bf16 (fp8 instructions, 256 x 256 tiles) takes
// 0.84 to 0.90 ms by the machine, 2.14 to 2.28 PFLOP/s; the matrix cores are
// busy 55 % of the cycles, the LDS and the vector units 35 % each, at the 1.7
// GHz that the power budget leaves; the stages' copies out of L2 (64 KB a stage
// and CU, 9 TB/s in all) run beside them.  The exact form (2048 x 28672 x 8192
// gated to codes: 1.44 to 1.52 ms, 1.27 to 1.33 PFLOP/s) is at 0.90 to 0.95 of
// the rate that a large bf16 product reaches here; the issue of its conversions
// and adds takes 46 % of the cycles, the products 55 %.
// BM x BN tile of C per workgroup, waves of WM x WN, K in stages of one block
// in a ring of NS stage buffers.  Stages go from memory straight into LDS
// (global_load_lds: no registers, no LDS store instructions), NS-1 ahead.
// LDS per stage: BM + BN rows of 128 bytes (16-byte piece p of row r in slot
// p ^ ((r >> 1) & 7): the 16 rows that a lane group reads together cover all
// 64 banks).  Scales come eight blocks of K at a time, 8 rows x 8 blocks a
// copy (a copy of one block's scales touches a cache line for each row: with
// those, 4096 x 28672 x 8192 took 917 us instead of 843), into two buffers of
// [BM + 2][8]: the rows of A, then the tile's one or two blocks of B.
// GATED: the B rows are BN/2 gate rows, then BN/2 up rows of the same
// columns, and a wave's columns are half gate, half up.
template <int BM, int BN, int WM, int WN, int NS> struct Tile {
  static constexpr int WAVES = (BM / WM) * (BN / WN), NT = WAVES * 64;
  static constexpr int MI = WM / 16, NI = WN / 16;
  static constexpr int SEGS = (BM + BN) / 8;            // 1-KB copies per stage
  static constexpr int PER = (SEGS + WAVES - 1) / WAVES;   // ... per wave
  static constexpr int SB = (BM + BN) * 128;            // bytes per stage
  static constexpr int SCALES = NS * SB;                // two buffers of scales
  static constexpr int SCB = BM * 32 + 256;
  static constexpr int SMEM = SCALES + 2 * SCB;
  static constexpr int SCOPIES = BM / 8 + 1;            // copies of eight blocks' scales
  static_assert(NS >= 2 && NS <= 4, "copy plan");
  // Copy i of wave w; where the waves do not share the copies out evenly, some
  // make the last one again, with the same bytes.
  static __device__ __forceinline__ int seg(int w, int i) {
    return SEGS % WAVES ? min(w * PER + i, SEGS - 1) : w * PER + i;
  }
  static_assert((NS - 2) * PER <= 63, "vmcnt range");
  // waves a SIMD gets from the workgroups that fit in a CU's LDS: the
  // registers must leave room for them
  static constexpr int WPE = 163840 / SMEM * WAVES / 4;
};

// Waits until all copies but the last `ahead` stages' (loads complete in issue
// order; copies of scales among them only make the wait longer) have landed
// and this wave's LDS reads are done, then for the other waves.
template <int NW> __device__ __forceinline__ void stage_barrier(int ahead) {
  if (ahead <= 0) asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
  else if (ahead == 1) asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" :: "i"(NW) : "memory");
  else asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" :: "i"(2 * NW) : "memory");
}

// Tile of a workgroup.  Workgroup L runs on XCD L % 8: each XCD takes one
// stretch of the tile order, which goes down strips of eight tile rows, so
// the tiles an XCD's L2 serves at a time share rows of A and of B.
__device__ __forceinline__ void tile_of(uint32_t L, uint32_t total, uint32_t tm, uint32_t tn,
                                        uint32_t& bm, uint32_t& bn) {
  const uint32_t q = total / 8, r = total % 8, x = L % 8;
  const uint32_t u = x * q + min(x, r) + L / 8;
  const uint32_t strip = u / (8 * tn), rows = min(8u, tm - strip * 8), in = u - strip * 8 * tn;
  bm = strip * 8 + in % rows;
  bn = in / rows;
}

// Results as they are, fp32 sums to be joined, codes; and sums for bf16 results
// in fp16, each row of a group of columns times a power of two of its own.
enum { kStore = 0, kPartial = 1, kCodes = 2, kScaled = 3 };

// The power of two for kScaled, from the largest finite magnitude of a row's sums
// over a group of columns (the wave's own; an infinity beside them shall not take
// their bits): that one comes to 2^14 .. 2^15, which fp16 holds, and all down to
// 2^-28 of it keep fp16's 11 bits; below, half a step is 2^-39 of it.  (A bound of
// the sums from their scales instead would take the bits of those whose codes are
// small.)  The limit keeps the power's reciprocal an fp32 number; fp32's smallest
// sums then come to 2^-23 and more.
__device__ __forceinline__ int scaled_exponent(uint32_t mag) { return max((int)(mag >> 23) - 127 - 14, -126); }
constexpr float kInfinity = __builtin_inff();
__device__ __forceinline__ float power_of_two(int e) {
  return __builtin_bit_cast(float, (uint32_t)(e + 127) << 23);
}

// ---------------------------------------------------------------- rows by expert
// The sorted positions in stretches of up to BM rows of one expert, numbered
// along the order.  Found by every wave for itself: lane l counts the stretches
// of experts l·per .. (l+1)·per - 1, and a scan over the lanes gives what lies
// before them.  Offsets are clamped to the slots there are, and the counts to the
// most stretches that sorted slots can make (most_stretches; the grid is made for
// them), so that no table makes a kernel read outside its rows or a count pass 32
// bits: offsets that go up and down over 2^30 slots of 1024 experts would count
// 2^32 stretches of 128.  Sums that saturate leave no stretch below the total
// without a lane that finds it.
struct Stretch { int expert, row, rows; };
__device__ __forceinline__ int offset_of(const GArgs& a, int e) {
  return min(max(a.offsets[min(e, a.E)], 0), a.slots);
}
// The most stretches of bm rows that `slots` rows of E experts can make.
template <typename T> __host__ __device__ __forceinline__ T most_stretches(T slots, T E, T bm) {
  const T n = slots / bm + (E < slots ? E : slots);
  return n < slots ? n : slots;
}
template <int BM> struct Stretches {
  int per, e0, sum, below, total;
  // offsets: clamped, [E + 1]
  __device__ __forceinline__ Stretches(const int* offsets, int E, int slots) {
    const int lane = threadIdx.x & 63, most = most_stretches(slots, E, BM);
    per = (E + 63) >> 6;
    e0 = lane * per;
    sum = 0;
    int o = offsets[min(e0, E)];
#pragma unroll 1
    for (int j = 1; j <= per; ++j) {
      const int p = offsets[min(e0 + j, E)];
      sum = min(sum + max(p - o + BM - 1, 0) / BM, most);
      o = p;
    }
    int in = sum;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int y = __shfl_up(in, d);
      if (lane >= d) in = min(in + y, most);
    }
    below = in - sum;
    total = __builtin_amdgcn_readlane(in, 63);
  }
  // stretch u < total
  __device__ __forceinline__ Stretch find(const int* offsets, int E, int u) const {
    Stretch s{0, 0, 0};
    int left = u - below, o = offsets[min(e0, E)];
    const bool here = left >= 0 && left < sum;
    bool open = here;
#pragma unroll 1
    for (int j = 1; j <= per; ++j) {
      const int p = offsets[min(e0 + j, E)], n = max(p - o + BM - 1, 0) / BM;
      if (open && left < n) {
        s = {e0 + j - 1, o + left * BM, min(BM, p - o - left * BM)};
        open = false;
      }
      left -= n;
      o = p;
    }
    const int src = (int)__builtin_ctzll(__ballot(here) | (1ull << 63));
    s.expert = __builtin_amdgcn_readlane(s.expert, src);
    s.row = __builtin_amdgcn_readlane(s.row, src);
    s.rows = __builtin_amdgcn_readlane(s.rows, src);
    return s;
  }
};

template <int BM, int BN, int WM, int WN, int NS, bool FAST, int FORM, int EPI, int DT>
__global__ __launch_bounds__((Tile<BM, BN, WM, WN, NS>::NT), (Tile<BM, BN, WM, WN, NS>::WPE)) void tile_kernel(GArgs a) {
  using T = Tile<BM, BN, WM, WN, NS>;
  constexpr bool GATED = FORM == kGated;
  constexpr int MI = T::MI, NI = T::NI, NB = GATED ? 2 : 1;
  // B pieces a step takes: the exact form's four instructions depend on each
  // other, so two pieces run side by side where registers allow
  constexpr int G = !FAST && MI * NI < 32 && NI % 2 == 0 ? 2 : 1;
  // Copies issued at a stage's start; the others follow an A piece later.  The
  // fp8 form of the largest tile gains by it (4096 x 28672 x 8192: 847 -> 824
  // us), the exact one does not.
  constexpr int FIRST = FAST && MI * NI == 32 ? T::PER / 2 : T::PER;
  constexpr int BC = BN / NB;      // columns of C
  constexpr int WC = WN / NB;      // ... of a wave
  __shared__ __attribute__((aligned(1024))) char S[T::SMEM];
  const int t = threadIdx.x, lane = t & 63;
  const int w = __builtin_amdgcn_readfirstlane(t >> 6);
  const int wm = w / (BN / WN), wn = w % (BN / WN);
  uint32_t bm, bn;
  const uint32_t tiles = (uint32_t)a.tm * a.tn, split = blockIdx.x / tiles;
  tile_of(blockIdx.x - split * tiles, tiles, a.tm, a.tn, bm, bn);
  const int64_t m0 = (int64_t)bm * BM;
  const int mleft = (int)min((int64_t)BM, a.M - m0);
  const int64_t n0 = (int64_t)bn * BC;
  const int kbeg = (int)split * a.kper, kend = min(a.kb, kbeg + a.kper);
  const int nst = kend - kbeg;
  const int nleft = (int)min((int64_t)BC, a.N - n0);

  // Copy plan: wave w's copy i fills KB w·PER + i of the stage: eight rows,
  // lane l row l/8 of them, slot l%8.  Rows past the matrix copy its last
  // row (their results are never stored).
  auto seg_base = [&](int seg) -> const uint8_t* {   // wave-uniform
    if (seg < BM / 8) return a.A + m0 * a.lda;
    const int half = GATED && seg >= (BM + BC) / 8;
    return a.B[half] + n0 * a.ldb[half];
  };
  auto seg_offset = [&](int seg, int l) -> int64_t {   // row and piece of lane l
    const int row = seg * 8 + (l >> 3), p16 = (((l & 7) ^ (l >> 4)) << 4) ^ ((seg & 1) << 6);
    if (seg < BM / 8) return (int64_t)min(row, mleft - 1) * a.lda + p16;
    const int half = GATED && seg >= (BM + BC) / 8;
    return (int64_t)min(row - BM - half * BC, nleft - 1) * a.ldb[half] + p16;
  };
  // The exact form with the largest tile has no registers left to keep its
  // offsets in (a spill would wait for the copies in flight) and computes them
  // anew each stage.
  constexpr bool KEEP = FAST || MI * NI < 32;
  uint32_t voff[KEEP ? T::PER : 1];
  if constexpr (KEEP) {
#pragma unroll
    for (int i = 0; i < T::PER; ++i) voff[i] = (uint32_t)seg_offset(T::seg(w, i), lane);
  }
  const unsigned sbase = (unsigned)(uintptr_t)(__attribute__((address_space(3))) char*)S;
  const int last_wide = a.wide ? (a.K % 128 ? a.kb - 1 : a.kb) : 0;   // blocks from here on: through registers
  // the wave's copies of the scales of blocks 8·g.. of this split
  auto copy_scales = [&](int g) {
    int l = lane;
    asm volatile("" : "+v"(l));   // eight stages apart: not worth registers
    const int r = l >> 3, k = min(kbeg + 8 * g + (l & 7), a.kb - 1);
#pragma unroll
    for (int idx = w; idx < T::SCOPIES; idx += T::WAVES) {
      const float* p;
      if (idx < BM / 8) p = a.sa + (m0 + min(idx * 8 + r, mleft - 1)) * a.kb;
      else if (GATED) p = (r == 0 ? a.sb[0] : a.sb[NB - 1]) + n0 / 128 * a.kb;
      else p = a.sb[0] + min(n0 / 128 + min(r, 1), a.nb - 1) * a.kb;
      lds_copy4(sbase + T::SCALES + (unsigned)((g & 1) * T::SCB + idx * 256), p + k);
    }
  };
  // copies i0 .. i1 - 1 of a stage (through registers: all of them with the first)
  auto copy = [&](int st, int i0, int i1) {
    const unsigned buf = (unsigned)((st % NS) * T::SB);
    if (kbeg + st < last_wide) {
      int l = lane;
      if constexpr (!KEEP) asm volatile("" : "+v"(l));   // not hoisted
#pragma unroll
      for (int i = i0; i < i1; ++i) {
        const int seg = T::seg(w, i);
        // ordered before the reads by the stage barriers
        lds_copy16(sbase + buf + (unsigned)seg * 1024u, seg_base(seg) + (int64_t)(kbeg + st) * 128,
                   KEEP ? voff[KEEP ? i : 0] : (uint32_t)seg_offset(seg, l));
      }
    } else if (i0 == 0) {
      // rows that end inside this block, or start at odd addresses: through
      // registers, few at a time (more would cost workgroups a CU)
      constexpr int U = FAST && T::PER % 2 == 0 ? 2 : 1;
#pragma unroll 1
      for (int g = 0; g < T::PER; g += U) {
        i32x4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int seg = T::seg(w, g + u);
          const int p16 = (((lane & 7) ^ (lane >> 4)) << 4) ^ ((seg & 1) << 6);
          v[u] = piece16(seg_base(seg) + seg_offset(seg, lane) - p16, (int64_t)(kbeg + st) * 128 + p16, a.K);
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
          *reinterpret_cast<i32x4*>(S + buf + T::seg(w, g + u) * 1024 + lane * 16) = v[u];
      }
      asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    }
  };

  f32x4 acc[NI][MI];
#pragma unroll
  for (int j = 0; j < NI; ++j)
#pragma unroll
    for (int i = 0; i < MI; ++i) acc[j][i] = f32x4{0.f, 0.f, 0.f, 0.f};

  const int l15 = lane & 15, sw = ((lane >> 4) ^ ((l15 >> 1) & 7)) << 4;
  const int arow = (wm * WM + l15) * 128 + sw;
  const int brow = (BM + wn * WC + l15) * 128 + sw;
  const int soff = T::SCALES + (wm * WM + l15) * 32;
  const int boff = T::SCALES + BM * 32 + (GATED ? 0 : wn * WC / 128 * 32);
  auto scales_of = [&](int st) { return S + ((st >> 3) & 1) * T::SCB + (st & 7) * 4; };

  // Operands of a stage: raw bytes from LDS, then the instruction's form.
  struct Raw { i32x4 x, y; };
  auto read_b = [&](const char* b, int j) -> Raw {
    const int off = brow + (GATED ? (j / (NI / 2)) * BC * 128 + (j % (NI / 2)) * 2048 : j * 2048);
    return {*reinterpret_cast<const i32x4*>(b + off), *reinterpret_cast<const i32x4*>(b + (off ^ 64))};
  };
  auto read_a = [&](const char* b, int i) -> Raw {
    const int off = arow + i * 2048;
    return {*reinterpret_cast<const i32x4*>(b + off), *reinterpret_cast<const i32x4*>(b + (off ^ 64))};
  };

  if (nst > 0) {
    copy_scales(0);
    for (int s0 = 0; s0 < NS - 1 && s0 < nst; ++s0) copy(s0, 0, T::PER);
    stage_barrier<T::PER>(min(nst - 1, NS - 2));
    // The loop is software-pipelined by hand: step (i, j) multiplies A piece i
    // by B piece j and adds the product of the step before, so the matrix
    // core works while the adds run; A pieces are read one ahead, and the
    // next stage's first pieces after the barrier that is placed before the
    // last A piece's steps.
    Frag<FAST> fb[NI], fa;
    Raw ra;
    float sb[NB], sa, sn;
#pragma unroll
    for (int j = 0; j < NI; ++j) { const Raw r = read_b(S, j); fb[j].set(r.x, r.y); }
    ra = read_a(S, 0);
    sn = *reinterpret_cast<const float*>(S + soff);
#pragma unroll
    for (int q = 0; q < NB; ++q) sb[q] = *reinterpret_cast<const float*>(S + boff + 32 * q);
    for (int st = 0; st < nst; ++st) {
      if (st + NS - 1 < nst) copy(st + NS - 1, 0, FIRST);
      if ((st & 7) == 0 && st + 8 < nst) copy_scales((st >> 3) + 1);
      const char* sc = scales_of(st);
      const char* sc_ = scales_of(st + 1);
      const char* b = S + (st % NS) * T::SB;
      const char* bn_ = S + ((st + 1) % NS) * T::SB;
      f32x4 p[G];
      float sp[G] = {}, s[NB];
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        if (i == 1 && FIRST < T::PER && st + NS - 1 < nst) copy(st + NS - 1, FIRST, T::PER);
        fa.set(ra.x, ra.y);
        sa = sn;
#pragma unroll
        for (int q = 0; q < NB; ++q) s[q] = sa * sb[q];
        if (i + 1 < MI) {
          ra = read_a(b, i + 1);
          sn = *reinterpret_cast<const float*>(sc + soff + (i + 1) * 512);
        } else {
          stage_barrier<T::PER>(min(nst - 1, st + NS - 1) - (st + 1));
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = 0; j < NI; j += G) {
          f32x4 q[G];
          contract(&fb[j], fa, q);
          // keeps the adds below behind these products
#pragma unroll
          for (int g = 0; g < G; ++g) {
            if (i + j > 0) asm volatile("" : "+v"(q[g]), "+v"(p[g]));
            else asm volatile("" : "+v"(q[g]));
          }
          if (i + 1 == MI) {   // the next stage's pieces (past the last stage: unused bytes)
#pragma unroll
            for (int g = 0; g < G; ++g) {
              const Raw r = read_b(bn_, j + g);
              fb[j + g].set(r.x, r.y);
            }
            if (j == 0) {
              ra = read_a(bn_, 0);
              sn = *reinterpret_cast<const float*>(sc_ + soff);
#pragma unroll
              for (int h = 0; h < NB; ++h) sb[h] = *reinterpret_cast<const float*>(sc_ + boff + 32 * h);
            }
          }
          const int pi = j > 0 ? i : i - 1, pj = j > 0 ? j - G : NI - G;
          if (pi >= 0) {
#pragma unroll
            for (int g = 0; g < G; ++g) {
#pragma unroll
              for (int r = 0; r < 4; ++r)
                acc[pj + g][pi][r] = __builtin_fmaf(p[g][r], sp[g], acc[pj + g][pi][r]);
              asm volatile("" : "+v"(acc[pj + g][pi]));   // ... and here
            }
          }
#pragma unroll
          for (int g = 0; g < G; ++g) {
            p[g] = q[g];
            sp[g] = s[GATED ? (j + g) / (NI / 2) : 0];
          }
          __builtin_amdgcn_sched_barrier(0);
        }
      }
#pragma unroll
      for (int g = 0; g < G; ++g)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          acc[NI - G + g][MI - 1][r] = __builtin_fmaf(p[g][r], sp[g], acc[NI - G + g][MI - 1][r]);
    }
    __syncthreads();   // the epilogue reuses the stage buffers
  }

  const int nl = wn * WC + 4 * (lane >> 4);   // this lane's first column in the tile
  if constexpr (EPI == kPartial) {
    if constexpr (GATED && !FAST && BC < 128) {   // codes of a tile below a block: here unsplit too
      if (a.kper >= a.kb) {   // h itself
#pragma unroll
        for (int i = 0; i < MI; ++i) {
          const int ml = wm * WM + i * 16 + l15;
#pragma unroll
          for (int j = 0; j < NI / NB; ++j) {
#pragma unroll
            for (int r = 0; r < 4; ++r)
              acc[j][i][r] = activate(acc[j][i][r], a.act) * acc[NI / NB + j][i][r];
            if (ml < mleft)
              put4<GPTQ_F32>(a.P, (m0 + ml) * a.N + n0 + nl + j * 16, nleft - nl - j * 16, acc[j][i]);
          }
        }
        return;
      }
    }
    float* P = a.P + (int64_t)split * NB * a.M * a.N;
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      const int ml = wm * WM + i * 16 + l15;
      if (ml >= mleft) continue;
#pragma unroll
      for (int j = 0; j < NI; ++j) {
        const int half = GATED ? j / (NI / 2) : 0, c = nl + (GATED ? j % (NI / 2) : j) * 16;
        put4<GPTQ_F32>(P, ((int64_t)half * a.M + m0 + ml) * a.N + n0 + c, nleft - c, acc[j][i]);
      }
    }
    return;
  }
  constexpr int NO = GATED ? NI / 2 : NI;   // 16-column pieces of C
  if constexpr (GATED) {
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NO; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[j][i][r] = activate(acc[j][i][r], a.act) * acc[NO + j][i][r];
  }
  if constexpr (FORM == kLinear) {
    if (a.bias) {
#pragma unroll
      for (int j = 0; j < NI; ++j) {
        const f32x4 b = get4(a.bias, a.bias_dt, n0 + nl + j * 16, nleft - nl - j * 16);
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[j][i][r] += b[r];
      }
    }
    if (a.act >= 0) {
      const Activation act(a.act);
#pragma unroll
      for (int j = 0; j < NI; ++j)
#pragma unroll
        for (int i = 0; i < MI; ++i) acc[j][i] = act(acc[j][i]);
    }
  }
  if constexpr (EPI == kStore && FORM == kLinear) {
    // residuals of as many rows together as 32 registers hold: who waits for a load
    // waits for the stores before it too (8192 x 8192 x 1024, bf16, gelu: one piece
    // of rows at a time 213 us, four 190, all eight, which spills, 216)
    constexpr bool PAIRS = DT != GPTQ_F32 && NO % 2 == 0;
    constexpr int CH = PAIRS ? (MI > 4 ? 4 : MI) : (MI * NI > 8 ? 8 / NI : MI);
    static_assert(MI % CH == 0, "chunks of rows");
#pragma unroll
    for (int i0 = 0; i0 < MI; i0 += CH) {
      if (a.R) {
        if constexpr (PAIRS) {
          i32x4 x[CH][NO / 2];
#pragma unroll
          for (int i = 0; i < CH; ++i) {
            const int ml = wm * WM + (i0 + i) * 16 + l15;
#pragma unroll
            for (int j = 0; j < NO; j += 2) {
              const int n = wn * WC + j * 16 + eight_at(lane);
              x[i][j / 2] = get8_of<DT>(a.R, (m0 + ml) * a.ldr + n0 + n, ml < mleft ? nleft - n : 0);
            }
          }
#pragma unroll
          for (int i = 0; i < CH; ++i)
#pragma unroll
            for (int j = 0; j < NO; j += 2) add8<DT>(x[i][j / 2], acc[j][i0 + i], acc[j + 1][i0 + i]);
        } else {
          f32x4 x[CH][NI];
#pragma unroll
          for (int i = 0; i < CH; ++i) {
            const int ml = wm * WM + (i0 + i) * 16 + l15;
#pragma unroll
            for (int j = 0; j < NI; ++j)
              x[i][j] = get4_of<DT>(a.R, (m0 + ml) * a.ldr + n0 + nl + j * 16, ml < mleft ? nleft - nl - j * 16 : 0);
          }
#pragma unroll
          for (int i = 0; i < CH; ++i)
#pragma unroll
            for (int j = 0; j < NI; ++j)
#pragma unroll
              for (int r = 0; r < 4; ++r) acc[j][i0 + i][r] += x[i][j][r];
        }
      }
#pragma unroll
      for (int i = i0; i < i0 + CH; ++i) {
        const int ml = wm * WM + i * 16 + l15;
        put_row<DT, NO>(a.C, (m0 + ml) * a.ldc + n0 + wn * WC, ml < mleft ? nleft - wn * WC : 0, acc, i, lane);
      }
    }
  } else if constexpr (EPI == kStore) {
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      const int ml = wm * WM + i * 16 + l15;
      put_row<DT, NO>(a.C, (m0 + ml) * a.ldc + n0 + wn * WC, ml < mleft ? nleft - wn * WC : 0, acc, i, lane);
    }
  } else {
    // the tile is one or two blocks of 128 columns wide, a wave within one
    static_assert(EPI != kCodes || (BC % 128 == 0 && 128 % WC == 0), "whole blocks");
    constexpr int WPB = EPI == kCodes ? 128 / WC : 1;   // waves across a block
    const int first = wn / WPB * WPB;
    uint32_t* top = reinterpret_cast<uint32_t*>(S);   // [BN / WN][BM]
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      uint32_t u = 0;
#pragma unroll
      for (int j = 0; j < NO; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (nl + j * 16 + r < nleft) u = max(u, mag_bits(acc[j][i][r]));
      u = max(u, (uint32_t)__shfl_xor((int)u, 16));
      u = max(u, (uint32_t)__shfl_xor((int)u, 32));
      if (lane < 16) top[wn * BM + wm * WM + i * 16 + l15] = u;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      const int ml = wm * WM + i * 16 + l15;
      uint32_t u = 0;
#pragma unroll
      for (int q = 0; q < WPB; ++q) u = max(u, top[(first + q) * BM + ml]);
      const float s = e4m3_scale((double)__builtin_bit_cast(float, u));
      const float inv = 1.f / s;
      if (ml >= mleft) continue;
      if (wn == first && lane < 16 && (BC == 128 || n0 + wn * WC < a.N))
        a.sc[(m0 + ml) * a.nb + (BC == 128 ? bn : (uint32_t)((n0 + wn * WC) / 128))] = s;
#pragma unroll
      for (int j = 0; j < NO; ++j) {
        uint32_t c;
        if constexpr (FORM == kLinear) c = codes4(acc[j][i][0], acc[j][i][1], acc[j][i][2], acc[j][i][3], s, inv);
        else c = codes4(acc[j][i][0], acc[j][i][1], acc[j][i][2], acc[j][i][3], inv);
        uint8_t* o = a.codes + (m0 + ml) * a.ld_codes + n0 + nl + j * 16;
        const int n = nleft - nl - j * 16;
        if (n >= 4) {
          __builtin_memcpy(o, &c, 4);
        } else {
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (r < n) o[r] = (uint8_t)(c >> (8 * r));
        }
      }
    }
  }
}

// ---------------------------------------------------------------- few rows
// Up to 64 rows of A: the weights' bytes are what counts.  A workgroup owns 16
// columns (of gate and of up for GATED) and each of its waves a stretch of K.
// A wave copies its blocks into a ring of its own in LDS, FD ahead, and waits
// for its own copies alone: no barrier in the loop, no registers in flight,
// and whole 128-byte lines (loads straight into registers, in the
// instruction's layout of 16 rows by 64 bytes, reached 35 bytes a ns and CU;
// this reaches 75).  The waves' sums are added in wave order.
// Bound: the weights' bytes, and at more than 16 rows the copies of A beside
// them.  28672 x 8192 at 16 rows: 34 us, 6.8 TB/s out of the memory-side
// cache.  Kernel times with the weights there / from memory: 11008 x 4096 gate
// and up at 4 rows 18.6 / 21.4 us (4.2 TB/s), 4096 x 4096 at one row 5.5 / 6.0,
// 37 x 4000 x 11008 to fp32 13.9 / 16.8.
// NA: 8-row copies of A.
constexpr int kFewRows = 64, kFewDepth = 2;

template <int NA, bool GATED> struct Few {
  static constexpr int NB = GATED ? 2 : 1, MT = (NA + 1) / 2;
  static constexpr int WAVES = NB + MT <= 4 ? 8 : NB + MT == 5 ? 6 : 5;   // as many as LDS holds
  static constexpr int PER = 2 * NB + NA;                 // copies a block
  static constexpr int SLOT = (NB + MT) * 2048;           // B rows, then A rows
  static constexpr int SCB = MT * 512 + 256;              // scales of eight blocks: A rows, then B
  static constexpr int RING = kFewDepth * SLOT + 2 * SCB; // bytes of a wave
  static constexpr int PART = NB * MT * 16 * 17;          // a wave's sums (floats)
  static constexpr int SMEM = WAVES * (RING > PART * 4 ? RING : PART * 4);
};

template <int NA, bool FAST, int FORM, int EPI>
__global__ __launch_bounds__((Few<NA, FORM == kGated>::WAVES * 64)) void few_rows_kernel(GArgs a) {
  constexpr bool GATED = FORM == kGated;
  using F = Few<NA, GATED>;
  constexpr int NB = F::NB, MT = F::MT;
  __shared__ __attribute__((aligned(1024))) char S[F::SMEM];
  const int t = threadIdx.x, lane = t & 63, l15 = lane & 15;
  const int w = __builtin_amdgcn_readfirstlane(t >> 6);
  const int64_t n0 = (int64_t)blockIdx.x * 16;
  const int nleft = (int)min((int64_t)16, a.N - n0), mleft = (int)a.M;
  const int per = (a.kb + F::WAVES - 1) / F::WAVES;
  const int kbeg = w * per, nblk = min(per, a.kb - kbeg);   // may be 0 or less
  char* ring = S + w * F::RING;
  const unsigned rbase = (unsigned)(uintptr_t)(__attribute__((address_space(3))) char*)ring;

  // copy i of a block: eight rows of B (i < 2·NB) or A, lane l row l/8 of them,
  // piece l%8 to slot l%8 as in the tile kernel; rows that do not exist copy
  // the last one (their results are never stored)
  auto base = [&](int i) -> const uint8_t* {
    return i < 2 * NB ? a.B[i / 2] + n0 * a.ldb[i / 2] : a.A;
  };
  auto offset = [&](int i) -> int64_t {
    const int p16 = (((lane & 7) ^ (lane >> 4)) << 4) ^ ((i & 1) << 6);
    return i < 2 * NB ? (int64_t)min((i & 1) * 8 + (lane >> 3), nleft - 1) * a.ldb[i / 2] + p16
                      : (int64_t)min((i - 2 * NB) * 8 + (lane >> 3), mleft - 1) * a.lda + p16;
  };
  auto dest = [&](int slot, int i) { return slot * F::SLOT + i * 1024; };
  uint32_t voff[F::PER];
#pragma unroll
  for (int i = 0; i < F::PER; ++i) voff[i] = (uint32_t)offset(i);
  const int last_wide = a.wide ? (a.K % 128 ? a.kb - 1 : a.kb) : 0;   // blocks from here on: through registers
  auto copy = [&](int j) {
    const int slot = j % kFewDepth;
    if (kbeg + j < last_wide) {
#pragma unroll
      for (int i = 0; i < F::PER; ++i)
        lds_copy16(rbase + (unsigned)dest(slot, i), base(i) + (int64_t)(kbeg + j) * 128, voff[i]);
    } else if (FORM == kLinear && a.wide && a.K % 16 == 0) {
      // K ends between two pieces (to codes, us, in brackets through registers, at 8 / 33
      // / 64 rows: 11008 x 4000 13.7 (15.4) / 24.9 (28.6) / 31.6 (33.5), 9000 x 1504 9.1
      // (10.0) / 15.7 (19.7) / 19.0 (24.1), 1024 x 5392 8.6 (8.5) / 11.2 (11.1) / 13.4
      // (13.4)).  The plain and gated products' kernels are without it.
#pragma unroll
      for (int i = 0; i < F::PER; ++i) {
        const int p16 = (((lane & 7) ^ (lane >> 4)) << 4) ^ ((i & 1) << 6);
        const int64_t k = (int64_t)(kbeg + j) * 128;
        lds_copy16(rbase + (unsigned)dest(slot, i), within(base(i) + offset(i) + k, k + p16 < a.K));
      }
    } else {
      i32x4 v[F::PER];
#pragma unroll
      for (int i = 0; i < F::PER; ++i) {
        const int p16 = (((lane & 7) ^ (lane >> 4)) << 4) ^ ((i & 1) << 6);
        v[i] = piece16(base(i) + offset(i) - p16, (int64_t)(kbeg + j) * 128 + p16, a.K);
      }
#pragma unroll
      for (int i = 0; i < F::PER; ++i) *reinterpret_cast<i32x4*>(ring + dest(slot, i) + lane * 16) = v[i];
      asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    }
  };
  // scales of blocks 8·g..: eight rows by eight blocks a copy
  auto copy_scales = [&](int g) {
    const int r = lane >> 3, k = min(kbeg + 8 * g + (lane & 7), a.kb - 1);
#pragma unroll
    for (int i = 0; i < 2 * MT + 1; ++i) {
      const float* p = i < 2 * MT ? a.sa + (int64_t)min(i * 8 + r, mleft - 1) * a.kb
                                  : (r == 0 ? a.sb[0] : a.sb[NB - 1]) + n0 / 128 * a.kb;
      lds_copy4(rbase + (unsigned)(kFewDepth * F::SLOT + (g & 1) * F::SCB + i * 256), p + k);
    }
  };

  f32x4 acc[MT][NB];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int b = 0; b < NB; ++b) acc[i][b] = f32x4{0.f, 0.f, 0.f, 0.f};
  if (nblk > 0) {
    copy_scales(0);
#pragma unroll
    for (int j = 0; j < kFewDepth; ++j)
      if (j < nblk) copy(j);
  }
  const int row = l15 * 128 + (((lane >> 4) ^ ((l15 >> 1) & 7)) << 4);
  for (int j = 0; j < nblk; ++j) {
    // this block's copies have landed when no more are in flight than the
    // later blocks' (scales among them only make the wait longer)
    if (j + kFewDepth <= nblk) asm volatile("s_waitcnt vmcnt(%0)" :: "i"((kFewDepth - 1) * F::PER) : "memory");
    else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    const char* q = ring + (j % kFewDepth) * F::SLOT + row;
    const char* sc = ring + kFewDepth * F::SLOT + ((j >> 3) & 1) * F::SCB + (j & 7) * 4;
    i32x4 x[NB + MT], y[NB + MT];
#pragma unroll
    for (int i = 0; i < NB + MT; ++i) {
      x[i] = *reinterpret_cast<const i32x4*>(q + i * 2048);
      y[i] = *reinterpret_cast<const i32x4*>(ring + (j % kFewDepth) * F::SLOT + (row ^ 64) + i * 2048);
    }
    float sa[MT], sb[NB];
#pragma unroll
    for (int i = 0; i < MT; ++i) sa[i] = *reinterpret_cast<const float*>(sc + (i * 16 + l15) * 32);
#pragma unroll
    for (int b = 0; b < NB; ++b) sb[b] = *reinterpret_cast<const float*>(sc + MT * 512 + b * 32);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // read: the slot may be written again
    if ((j & 7) == 0 && j + 8 < nblk) copy_scales((j >> 3) + 1);
    if (j + kFewDepth < nblk) copy(j + kFewDepth);
    Frag<FAST> fb[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) fb[b].set(x[b], y[b]);
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      Frag<FAST> fa;
      fa.set(x[NB + i], y[NB + i]);
      f32x4 p[NB];
      contract(fb, fa, p);
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const float s = sa[i] * sb[b];
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[i][b][r] = __builtin_fmaf(p[b][r], s, acc[i][b][r]);
      }
    }
  }
  __syncthreads();   // the sums go where the rings were
  float* part = reinterpret_cast<float*>(S);
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        part[w * F::PART + ((b * MT + i) * 16 + l15) * 17 + 4 * (lane >> 4) + r] = acc[i][b][r];
  __syncthreads();
  const int c = t & 15;
  if (c >= nleft) return;
  const int64_t n = n0 + c;
  for (int m = t >> 4; m < MT * 16 && m < mleft; m += F::WAVES * 4) {
    float h[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      h[b] = 0.f;
#pragma unroll
      for (int v = 0; v < F::WAVES; ++v) h[b] += part[v * F::PART + (b * MT * 16 + m) * 17 + c];
    }
    float o = h[0];
    if constexpr (GATED) o = activate(h[0], a.act) * h[NB - 1];
    if constexpr (EPI == kPartial) {
      a.P[(int64_t)m * a.N + n] = o;     // h itself: one partial, activated (kLinear: the sum)
    } else {
      if constexpr (FORM == kLinear) {
        if (a.bias) o += get1(a.bias, a.bias_dt, n);
        if (a.act >= 0) o = activate(o, a.act);
        if (a.R) o += get1(a.R, a.c_dt, m * a.ldr + n);
      }
      put1(a.C, a.c_dt, m * a.ldc + n, o);
    }
  }
}

// ---------------------------------------------------------------- joining partial sums
// One thread per eight columns: the partials in split order, then the
// activation (gated, not yet activated) and C, or a block's codes and scale
// (16 lanes a block).  A launch of its own, 2 to 4 us where the partials are
// small; the cost model charges it to every split.
template <int FORM, bool CODES, int ROWS = kDense>
__global__ __launch_bounds__(256) void join_kernel(GArgs a, int splits) {
  constexpr bool GATED = FORM == kGated;
  constexpr int NB = GATED ? 2 : 1;
  const int t = threadIdx.x, lane = t & 15;
  const int64_t g = (int64_t)blockIdx.x * 16 + (t >> 4);
  const int64_t m = g / a.nb, blk = g - m * a.nb;
  if (m >= a.M) return;
  if constexpr (ROWS != kDense) {
    if (m >= offset_of(a, a.E)) return;   // behind the last expert's rows
  }
  const int64_t n = blk * 128 + lane * 8;
  const int c = (int)max((int64_t)0, min((int64_t)8, a.N - n));
  float h[NB][8];
#pragma unroll
  for (int b = 0; b < NB; ++b) {
#pragma unroll
    for (int i = 0; i < 8; ++i) h[b][i] = 0.f;
    // four splits' loads in flight: 322 x 448 x 8960 in 12 splits 17.3 -> 15.2 us
    for (int s = 0; s < splits; s += 4) {
      float v[4][8];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        load8<GPTQ_F32>(a.P + (((int64_t)min(s + u, splits - 1) * NB + b) * a.M + m) * a.N + n, c, v[u]);
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (s + u < splits) {
#pragma unroll
          for (int i = 0; i < 8; ++i) h[b][i] += v[u][i];
        }
    }
  }
  if constexpr (GATED) {
#pragma unroll
    for (int i = 0; i < 8; ++i) h[0][i] = activate(h[0][i], a.act) * h[NB - 1][i];
  }
  if constexpr (FORM == kLinear) {
    if (a.bias) {
      const f32x4 b = get4(a.bias, a.bias_dt, n, c), b2 = get4(a.bias, a.bias_dt, n + 4, c - 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        h[0][i] += b[i];
        h[0][4 + i] += b2[i];
      }
    }
    if (a.act >= 0) {
#pragma unroll
      for (int i = 0; i < 8; ++i) h[0][i] = activate(h[0][i], a.act);
    }
    if (a.R) {
      const f32x4 b = get4(a.R, a.c_dt, m * a.ldr + n, c), b2 = get4(a.R, a.c_dt, m * a.ldr + n + 4, c - 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        h[0][i] += b[i];
        h[0][4 + i] += b2[i];
      }
    }
  }
  if constexpr (CODES) {
    uint32_t u = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) u = max(u, mag_bits(h[0][i]));
    const float s = e4m3_scale((double)__builtin_bit_cast(float, row16_max_u32(u)));
    const float inv = 1.f / s;
    if constexpr (FORM == kLinear || ROWS != kDense)
      store_codes8(a.codes + m * a.ld_codes + n, c, codes4(h[0][0], h[0][1], h[0][2], h[0][3], s, inv),
                   codes4(h[0][4], h[0][5], h[0][6], h[0][7], s, inv));
    else
      store_codes8(a.codes + m * a.ld_codes + n, c, codes4(h[0][0], h[0][1], h[0][2], h[0][3], inv),
                   codes4(h[0][4], h[0][5], h[0][6], h[0][7], inv));
    if (lane == 0) a.sc[m * a.nb + blk] = s;
  } else {
    if (a.c_dt == GPTQ_F32) store8<GPTQ_F32>(static_cast<float*>(a.C) + m * a.ldc + n, c, h[0]);
    else if (a.c_dt == GPTQ_BF16) store8<GPTQ_BF16>(static_cast<__bf16*>(a.C) + m * a.ldc + n, c, h[0]);
    else store8<GPTQ_F16>(static_cast<_Float16*>(a.C) + m * a.ldc + n, c, h[0]);
  }
}

}  // namespace
}  // namespace gq
