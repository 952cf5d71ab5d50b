// Products of block-scaled e4m3 matrices (fp8.hpp has the format):
//   C[m,n] = Σ_kb sa[m,kb]·sb[n/128,kb]·Σ_{k in kb} a[m,k]·b[n,k]
// and the gated projection act(A·Gᵀ)·(A·Uᵀ), rounded to 16 or 32 bits or
// quantized again in 1 x 128 blocks.
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
};

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

// Codes of four values of a block.  1/s and the product round by 2^-24 each, so
// a code is that of the fp32 value over its scale but within 2^-22 of a border.
// The values and the block's largest, its scale, carry fp32's rounding already;
// one more in the quotient moves no more codes over a border (1024 x 8192 x
// 2048: 50 of 8.4 million differ from those of exact sums, 49 with quotients in
// fp64, which took 1487 us where this takes 1447, 2048 x 28672 x 8192 to codes).
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d, float inv) {
  return e4m3_pack4(a * inv, b * inv, c * inv, d * inv);
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
  static constexpr int PER = SEGS / WAVES;              // ... per wave
  static constexpr int SB = (BM + BN) * 128;            // bytes per stage
  static constexpr int SCALES = NS * SB;                // two buffers of scales
  static constexpr int SCB = BM * 32 + 256;
  static constexpr int SMEM = SCALES + 2 * SCB;
  static constexpr int SCOPIES = BM / 8 + 1;            // copies of eight blocks' scales
  static_assert(SEGS % WAVES == 0 && NS >= 2 && NS <= 4, "copy plan");
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

enum { kStore = 0, kPartial = 1, kCodes = 2 };

template <int BM, int BN, int WM, int WN, int NS, bool FAST, bool GATED, int EPI, int DT>
__global__ __launch_bounds__((Tile<BM, BN, WM, WN, NS>::NT), (Tile<BM, BN, WM, WN, NS>::WPE)) void tile_kernel(GArgs a) {
  using T = Tile<BM, BN, WM, WN, NS>;
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
  const int64_t m0 = (int64_t)bm * BM, n0 = (int64_t)bn * BC;
  const int kbeg = (int)split * a.kper, kend = min(a.kb, kbeg + a.kper);
  const int nst = kend - kbeg;
  const int mleft = (int)min((int64_t)BM, a.M - m0), nleft = (int)min((int64_t)BC, a.N - n0);

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
    for (int i = 0; i < T::PER; ++i) voff[i] = (uint32_t)seg_offset(w * T::PER + i, lane);
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
        const int seg = w * T::PER + i;
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
          const int seg = w * T::PER + g + u;
          const int p16 = (((lane & 7) ^ (lane >> 4)) << 4) ^ ((seg & 1) << 6);
          v[u] = piece16(seg_base(seg) + seg_offset(seg, lane) - p16, (int64_t)(kbeg + st) * 128 + p16, a.K);
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
          *reinterpret_cast<i32x4*>(S + buf + (w * T::PER + g + u) * 1024 + lane * 16) = v[u];
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
  if constexpr (EPI == kStore) {
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      const int ml = wm * WM + i * 16 + l15;
      if (ml >= mleft) continue;
#pragma unroll
      for (int j = 0; j < NO; ++j)
        put4<DT>(a.C, (m0 + ml) * a.ldc + n0 + nl + j * 16, nleft - nl - j * 16, acc[j][i]);
    }
  } else {
    // the tile's 128 columns are one block of its rows
    static_assert(EPI != kCodes || BC == 128, "a tile is one block wide");
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
      for (int q = 0; q < BN / WN; ++q) u = max(u, top[q * BM + ml]);
      const float s = e4m3_scale((double)__builtin_bit_cast(float, u));
      const float inv = 1.f / s;
      if (ml >= mleft) continue;
      if (wn == 0 && lane < 16) a.sc[(m0 + ml) * a.nb + bn] = s;
#pragma unroll
      for (int j = 0; j < NO; ++j) {
        const uint32_t c = codes4(acc[j][i][0], acc[j][i][1], acc[j][i][2], acc[j][i][3], inv);
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

template <int NA, bool FAST, bool GATED, int EPI>
__global__ __launch_bounds__((Few<NA, GATED>::WAVES * 64)) void few_rows_kernel(GArgs a) {
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
      a.P[(int64_t)m * a.N + n] = o;     // h itself: one partial, activated
    } else {
      if (a.c_dt == GPTQ_F32) static_cast<float*>(a.C)[m * a.ldc + n] = o;
      else if (a.c_dt == GPTQ_BF16) static_cast<__bf16*>(a.C)[m * a.ldc + n] = (__bf16)o;
      else static_cast<_Float16*>(a.C)[m * a.ldc + n] = (_Float16)o;
    }
  }
}

// ---------------------------------------------------------------- joining partial sums
// One thread per eight columns: the partials in split order, then the
// activation (gated, not yet activated) and C, or a block's codes and scale
// (16 lanes a block).  A launch of its own, 2 to 4 us where the partials are
// small; the cost model charges it to every split.
template <bool GATED, bool CODES>
__global__ __launch_bounds__(256) void join_kernel(GArgs a, int splits) {
  constexpr int NB = GATED ? 2 : 1;
  const int t = threadIdx.x, lane = t & 15;
  const int64_t g = (int64_t)blockIdx.x * 16 + (t >> 4);
  const int64_t m = g / a.nb, blk = g - m * a.nb;
  if (m >= a.M) return;
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
  if constexpr (CODES) {
    uint32_t u = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) u = max(u, mag_bits(h[0][i]));
    const float s = e4m3_scale((double)__builtin_bit_cast(float, row16_max_u32(u)));
    const float inv = 1.f / s;
    store_codes8(a.codes + m * a.ld_codes + n, c, codes4(h[0][0], h[0][1], h[0][2], h[0][3], inv),
                 codes4(h[0][4], h[0][5], h[0][6], h[0][7], inv));
    if (lane == 0) a.sc[m * a.nb + blk] = s;
  } else {
    if (a.c_dt == GPTQ_F32) store8<GPTQ_F32>(static_cast<float*>(a.C) + m * a.ldc + n, c, h[0]);
    else if (a.c_dt == GPTQ_BF16) store8<GPTQ_BF16>(static_cast<__bf16*>(a.C) + m * a.ldc + n, c, h[0]);
    else store8<GPTQ_F16>(static_cast<_Float16*>(a.C) + m * a.ldc + n, c, h[0]);
  }
}

// ---------------------------------------------------------------- choice and launch
// The kernel for a product is the one that this model says is quickest.  Its
// times are microseconds on MI355X (fp8 instructions / exact form): a stage of a
// tile with one workgroup on each of the 256 CUs, and with as many as fit; a
// round's start and epilogue.  Fitted to every kernel and split of 240 products
// of random sizes (M to 2900, K to 10 944): what it picks takes 0.7 % longer
// than the quickest on average, a third longer at worst (40 x 5760 x 1216: few
// rows 10.0, 32-tiles 7.3).  Small tiles win
// where there are few (512 x 4096: 64-tiles 18.7 / 29.1 us, 128-tiles in two
// splits 25.2 / 31.3, 256-tiles in eight 39 / 45), large ones where there are
// many (4096 x 4096: 131 / 201, 83 / 140, 67 / 118).
struct TileCost { int bm, bn, fit; double one[2], full[2], ends; };   // [0] fp8, [1] exact
constexpr TileCost kTiles[] = {
    {32, 64, 3, {0.29, 0.44}, {0.53, 0.73}, 1.25},
    {64, 64, 2, {0.36, 0.64}, {0.51, 0.81}, 1.45},
    {128, 128, 2, {0.70, 1.13}, {1.14, 1.81}, 2.1},
    {256, 256, 1, {1.77, 3.45}, {1.77, 3.45}, 2.3},
};
constexpr int kTileKinds = 4;
// us, us, us for each four splits' loads, bytes per us
constexpr double kLaunch = 2.7, kJoin = 2.2, kJoinLoads = 0.5, kJoinBytes = 4.0e6;
// Few rows, the same way: a workgroup's start and end, its copies at the rate
// one CU takes them (KB a us), or its waves' instructions (two waves a SIMD;
// cycles a block and wave: conversions, products, the rest), or all weights
// from memory (KB a us).
constexpr double kFewLaunch = 1.8, kFewGroup = 1.3, kFewCopies = 81.0, kFewWeights = 7e3, kClock = 2100.0;

struct Plan { int tile; int splits, kper; };   // tile -1: few rows

// join: the result goes through the workspace in any case (codes of a tile
// that is not a block wide).  Without a workspace one split of the 256-tile
// runs for codes, any unsplit kernel otherwise.
Plan plan_of(int64_t M, int64_t N, int64_t K, bool gated, bool exact, bool codes, bool ws) {
  const int nb = gated ? 2 : 1, e = exact ? 1 : 0;
  const int64_t kb = ceil_div(K, 128);
  Plan best{kTileKinds - 1, 1, (int)kb};
  double least = 1e300;
  if (M <= kFewRows && (!codes || ws)) {
    const int mt = (int)ceil_div(M, 16), waves = nb + mt <= 4 ? 8 : nb + mt == 5 ? 6 : 5;
    const int64_t groups = ceil_div(N, 16);
    const int fit = nb + mt == 2 ? 2 : 1, here = (int)std::min<int64_t>(fit, ceil_div(groups, 256));
    const double copied = 2.0 * kb * (nb + (M <= 8 ? 0.5 : mt)) / kFewCopies;
    const double cycles = exact ? 92 * (nb + mt) + 115 * nb * mt + 65 : 48 * nb * mt + 200;
    const double issued = 2.0 * (double)ceil_div(kb, waves) * cycles / kClock;
    least = kFewLaunch + (codes ? kJoin : 0) +
            std::max((double)ceil_div(groups, 256 * here) * (kFewGroup + here * std::max(copied, issued)),
                     2.0 * groups * kb * nb / kFewWeights);
    best = {-1, 1, (int)kb};
  }
  for (int i = 0; i < kTileKinds; ++i) {
    const TileCost& c = kTiles[i];
    const bool join = codes && c.bn < 256;
    if (join && !ws) continue;
    const int64_t tiles = ceil_div(M, c.bm) * ceil_div(N, c.bn / nb);
    for (const int s : {1, 2, 3, 4, 6, 8, 12, 16}) {
      if (s > 1 && (!ws || tiles * s > 1024 || 2 * s > kb)) break;
      const int kper = ((int)kb + s - 1) / s, splits = ((int)kb + kper - 1) / kper;
      const int64_t load = (tiles * splits + 255) >> 8;   // workgroups of a CU
      const int64_t rest = load % c.fit;                  // those of its last round, if not full
      double stage = (double)(load / c.fit) * c.full[e];
      if (rest) stage += c.one[e] + (rest > 1 ? (c.full[e] - c.one[e]) * (double)(rest - 1) / (c.fit - 1) : 0);
      double t = kLaunch + stage * kper + c.ends * (double)ceil_div(load, c.fit);
      if (splits > 1 || join)
        t += kJoin + (splits > 1 ? kJoinLoads * nb * (double)ceil_div(splits, 4) : 0) +
             (double)(splits > 1 ? splits * nb : 1) * M * N * 8 / kJoinBytes;
      if (t < least) {
        least = t;
        best = {i, splits, kper};
      }
    }
  }
  return best;
}

size_t plan_bytes(const Plan& p, int64_t M, int64_t N, bool gated, bool codes) {
  if (p.splits > 1) return (size_t)p.splits * (gated ? 2 : 1) * M * N * 4;
  return codes && p.tile != kTileKinds - 1 ? (size_t)M * N * 4 : 0;
}

template <int BM, int BN, int WM, int WN, int NS, bool FAST, bool GATED, int EPI, int DT>
hipError_t launch_tile(GArgs& a, int splits, hipStream_t s) {
  using T = Tile<BM, BN, WM, WN, NS>;
  a.tm = (int)ceil_div(a.M, BM);
  a.tn = (int)ceil_div(a.N, GATED ? BN / 2 : BN);
  const int64_t grid = (int64_t)a.tm * a.tn * splits;
  if (grid > INT32_MAX) return hipErrorInvalidValue;
  tile_kernel<BM, BN, WM, WN, NS, FAST, GATED, EPI, DT><<<(unsigned)grid, T::NT, 0, s>>>(a);
  return hipGetLastError();
}

template <bool FAST, bool GATED, int EPI, int DT>
hipError_t launch_kind(GArgs& a, const Plan& p, hipStream_t s) {
  switch (p.tile) {
    case 0: return launch_tile<32, 64, 16, 32, 4, FAST, GATED, EPI, DT>(a, p.splits, s);
    case 1: return launch_tile<64, 64, 32, 32, 4, FAST, GATED, EPI, DT>(a, p.splits, s);
    case 2: return launch_tile<128, 128, 64, 32, 2, FAST, GATED, EPI, DT>(a, p.splits, s);
    default: return launch_tile<256, 256, 128, 64, 2, FAST, GATED, EPI, DT>(a, p.splits, s);
  }
}

template <bool FAST, bool GATED, int EPI> hipError_t launch_few(const GArgs& a, hipStream_t s) {
  const unsigned grid = (unsigned)ceil_div(a.N, 16);
#define GQ_FEW(NA) few_rows_kernel<NA, FAST, GATED, EPI><<<grid, Few<NA, GATED>::WAVES * 64, 0, s>>>(a)
  if (a.M <= 8) GQ_FEW(1);
  else if (a.M <= 16) GQ_FEW(2);
  else if (a.M <= 32) GQ_FEW(4);
  else if (a.M <= 48) GQ_FEW(6);
  else GQ_FEW(8);
#undef GQ_FEW
  return hipGetLastError();
}

// One output form: EPI with DT (FAST goes with the 16-bit types).
template <bool GATED, int EPI, int DT>
hipError_t run(GArgs& a, void* ws, hipStream_t s) {
  constexpr bool FAST = EPI == kStore && DT != GPTQ_F32, codes = EPI == kCodes;
  const Plan p = plan_of(a.M, a.N, a.K, GATED, !FAST, codes, ws != nullptr);
  a.nb = ceil_div(a.N, 128);
  a.kb = (int)ceil_div(a.K, 128);
  a.kper = p.kper;
  a.P = static_cast<float*>(ws);
  // the wide copies' 32-bit offsets span a tile's rows
  auto wide = [](const uint8_t* q, int64_t rows, int64_t ld) {
    return (uintptr_t)q % 16 == 0 && (rows == 1 || (ld % 16 == 0 && ld < ((int64_t)1 << 23)));
  };
  a.wide = wide(a.A, a.M, a.lda) && wide(a.B[0], a.N, a.ldb[0]) && (!GATED || wide(a.B[1], a.N, a.ldb[1]));
  const bool join = p.splits > 1 || (codes && p.tile != kTileKinds - 1);
  hipError_t e;
  if (p.tile < 0) e = launch_few<FAST, GATED, codes ? kPartial : kStore>(a, s);
  else if (join) e = launch_kind<FAST, GATED, kPartial, GPTQ_F32>(a, p, s);
  else if constexpr (codes) e = launch_tile<256, 256, 128, 64, 2, false, true, kCodes, DT>(a, 1, s);
  else e = launch_kind<FAST, GATED, EPI, DT>(a, p, s);
  if (e != hipSuccess || !join) return e;
  const unsigned grid = (unsigned)ceil_div(a.M * a.nb, 16);
  if (p.splits > 1) join_kernel<GATED, codes><<<grid, 256, 0, s>>>(a, p.splits);
  else join_kernel<false, codes><<<grid, 256, 0, s>>>(a, 1);   // h itself
  return hipGetLastError();
}

template <bool GATED> hipError_t run_dt(GArgs& a, void* ws, hipStream_t s) {
  if constexpr (GATED)
    if (a.codes) return run<true, kCodes, GPTQ_F32>(a, ws, s);
  switch (a.c_dt) {
    case GPTQ_F32: return run<GATED, kStore, GPTQ_F32>(a, ws, s);
    case GPTQ_BF16: return run<GATED, kStore, GPTQ_BF16>(a, ws, s);
    default: return run<GATED, kStore, GPTQ_F16>(a, ws, s);
  }
}

// enough for every output form; 256, which no real need rounds up to, if none
// uses a workspace
size_t ws_bytes(int64_t M, int64_t N, int64_t K, bool gated) {
  size_t most = 0;
  for (int form = 0; form < (gated ? 3 : 2); ++form) {   // 16 bits, fp32, codes
    const Plan p = plan_of(M, N, K, gated, form > 0, form == 2, true);
    most = std::max(most, plan_bytes(p, M, N, gated, form == 2));
  }
  return most ? std::max<size_t>(512, align_up(most)) : 256;
}

}  // namespace

size_t fp8_gemm_ws_bytes(int64_t M, int64_t N, int64_t K) { return ws_bytes(M, N, K, false); }
size_t fp8_gated_ws_bytes(int64_t M, int64_t N, int64_t K) { return ws_bytes(M, N, K, true); }

hipError_t fp8_gemm_launch(const uint8_t* A, const float* sa, int64_t M, int64_t K, int64_t lda,
                           const uint8_t* B, const float* sb, int64_t N, int64_t ldb, void* C,
                           int c_dt, int64_t ldc, void* ws, hipStream_t s) {
  GArgs a{};
  a.A = A; a.sa = sa; a.M = M; a.K = K; a.lda = lda;
  a.B[0] = B; a.sb[0] = sb; a.N = N; a.ldb[0] = ldb;
  a.C = C; a.ldc = ldc; a.c_dt = c_dt;
  return run_dt<false>(a, ws, s);
}

hipError_t fp8_gated_launch(const uint8_t* A, const float* sa, int64_t M, int64_t K, int64_t lda,
                            const uint8_t* G, const float* sg, int64_t ldg, const uint8_t* U,
                            const float* su, int64_t ldu, int64_t N, int act, void* C, int c_dt,
                            int64_t ldc, uint8_t* codes, int64_t ld_codes, float* sc, void* ws,
                            hipStream_t s) {
  GArgs a{};
  a.A = A; a.sa = sa; a.M = M; a.K = K; a.lda = lda;
  a.B[0] = G; a.sb[0] = sg; a.ldb[0] = ldg;
  a.B[1] = U; a.sb[1] = su; a.ldb[1] = ldu; a.N = N;
  a.C = C; a.ldc = ldc; a.c_dt = c_dt; a.act = act;
  a.codes = codes; a.ld_codes = ld_codes; a.sc = sc;
  return run_dt<true>(a, ws, s);
}

}  // namespace gq
