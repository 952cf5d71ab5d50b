// Producers of block-scaled e4m3 matrices (fp8.hpp has the format):
//   quantize  a layer's weights (128 x 128 blocks) or activations (1 x 128)
//   rmsnorm   h = round(x + r), y = h·γ/sqrt(mean h² + ε), y in 1 x 128 blocks
// Both read their input once and keep it in registers between the pass that
// finds a block's largest magnitude and the pass that rounds.
#include "fp8.hpp"

namespace gq {
namespace {

struct QArgs {
  const void* X; int64_t rows, cols, ld_x;
  uint8_t* codes; int64_t ld_c;
  float* scales; int64_t kb;   // blocks along a row
};

__device__ __forceinline__ uint32_t mag_bits(float x) {
  return __builtin_bit_cast(uint32_t, x) & 0x7FFFFFFFu;   // orders finite < inf < NaN
}

__device__ __forceinline__ void encode8(const float (&v)[8], float s, uint32_t& lo, uint32_t& hi) {
  const double sd = (double)s, inv = e4m3_inverse(s);
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = e4m3_quotient((double)v[i], sd, inv);
  lo = e4m3_pack4(q[0], q[1], q[2], q[3]);
  hi = e4m3_pack4(q[4], q[5], q[6], q[7]);
}

// Activations: 16 lanes per 1 x 128 block, eight columns a lane.  A workgroup
// of 256 threads takes 2^lg blocks of a row side by side and 16 >> lg rows.
// Bound by memory: 517 x 11008 fp16 in 6.8 us (2.5 TB/s, mostly the launch's
// ramp), 1 x 4096 in 2.0 us (a launch).
template <int DT>
__global__ __launch_bounds__(256) void quantize_rows_kernel(QArgs a, int lg, uint32_t chunks) {
  typedef typename Elem<DT>::type T;
  const int t = threadIdx.x, g = t >> 4, lane = t & 15;
  const int64_t kb = (int64_t)(blockIdx.x % chunks) * (1 << lg) + (g & ((1 << lg) - 1));
  const int64_t row = (int64_t)(blockIdx.x / chunks) * (16 >> lg) + (g >> lg);
  if (kb >= a.kb || row >= a.rows) return;   // whole 16-lane rows leave together
  const int64_t col = kb * kFp8Block + lane * 8;
  const int n = (int)max((int64_t)0, min((int64_t)8, a.cols - col));
  float v[8];
  load8<DT>(static_cast<const T*>(a.X) + row * a.ld_x + col, n, v);
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, mag_bits(v[i]));
  const float s = e4m3_scale((double)__builtin_bit_cast(float, row16_max_u32(m)));
  uint32_t lo, hi;
  encode8(v, s, lo, hi);
  store_codes8(a.codes + row * a.ld_c + col, n, lo, hi);
  if (lane == 0) a.scales[row * a.kb + kb] = s;
}

// Weights: one workgroup per 128 x 128 block, 16 lanes across and 16 rows at
// a time, the whole block in registers (64 values a thread), so the input is
// read once.  Bound by memory: 28672 x 8192 bf16 in 137 to 139 us, 5.1 TB/s, the rate
// of a large copy; the fp64 quotients (about twelve instructions a value) hide
// behind it.
template <int DT>
__global__ __launch_bounds__(256) void quantize_block_kernel(QArgs a) {
  typedef typename Elem<DT>::type T;
  __shared__ uint32_t part[4];
  const int t = threadIdx.x, g = t >> 4, lane = t & 15;
  const int64_t kb = blockIdx.x % (uint32_t)a.kb, rb = blockIdx.x / (uint32_t)a.kb;
  const int64_t col = kb * kFp8Block + lane * 8;
  const int n = (int)max((int64_t)0, min((int64_t)8, a.cols - col));
  const int nr = (int)min((int64_t)kFp8Block, a.rows - rb * kFp8Block);
  float v[8][8];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = g + 16 * i;
    load8<DT>(static_cast<const T*>(a.X) + (rb * kFp8Block + r) * a.ld_x + col, r < nr ? n : 0, v[i]);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, mag_bits(v[i][j]));
  m = row16_max_u32(m);
  m = max(m, (uint32_t)__shfl_xor((int)m, 16));
  m = max(m, (uint32_t)__shfl_xor((int)m, 32));
  if ((t & 63) == 0) part[t >> 6] = m;
  __syncthreads();
  m = max(max(part[0], part[1]), max(part[2], part[3]));
  const float s = e4m3_scale((double)__builtin_bit_cast(float, m));
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = g + 16 * i;
    uint32_t lo, hi;
    encode8(v[i], s, lo, hi);
    if (r < nr) store_codes8(a.codes + (rb * kFp8Block + r) * a.ld_c + col, n, lo, hi);
  }
  if (t == 0) a.scales[rb * a.kb + kb] = s;
}

struct NArgs {
  const void* X; int64_t ld_x;
  const void* R; int64_t ld_r;   // residual or null
  const void* gamma;
  int64_t rows, cols; double inv_cols, eps;
  void* S; int64_t ld_s;         // h, or null
  void* Y; int64_t ld_y;         // y in h's type, or null
  uint8_t* codes; int64_t ld_c;  // or null, with scales
  float* scales; int64_t kb;
};

// One row per workgroup of NT threads; thread t holds the pieces t, t + NT,
// ... (P of them, eight columns each), so 16 neighbouring lanes hold a block.
// The sum of squares, 1/sqrt and y are fp64: the sum because rows are long,
// y because codes next to a border of e4m3 would change with fp32's rounding
// (the fp64 rate of gfx950 is that of unpacked fp32).  Many rows are bound by
// memory: 16384 x 4096 bf16 with a residual in 99 us, 4.8 TB/s, against 4.9 of
// a large copy.  A few hundred are not: 333 x 8190 fp16, y too, takes 11.8, four
// times its bytes' time, since a row is one workgroup's chain of load, sum and
// about 500 fp64 instructions a wave, with nothing to hide it (77 of 256 CUs
// have two rows).  One row takes 3.8 us.
template <int DT, int GDT, int NT, int P>
__global__ __launch_bounds__(NT) void rmsnorm_kernel(NArgs a) {
  typedef typename Elem<DT>::type T;
  typedef typename Elem<GDT>::type G;
  __shared__ double part[NT / 64];
  const int t = threadIdx.x;
  const int64_t row = blockIdx.x;
  auto col = [&](int i) { return (t + i * NT) * 8; };
  auto width = [&](int i) { return max(0, min(8, (int)a.cols - col(i))); };
  T v[P][8];
#pragma unroll
  for (int i = 0; i < P; ++i)
    load8_raw<DT>(static_cast<const T*>(a.X) + row * a.ld_x + col(i), width(i), v[i]);
  // γ arrives with the row where registers allow, else from the cache later
  constexpr bool EARLY = P <= 2;
  G gm[EARLY ? P : 1][8];
  if constexpr (EARLY) {
#pragma unroll
    for (int i = 0; i < P; ++i) load8_raw<GDT>(static_cast<const G*>(a.gamma) + col(i), width(i), gm[i]);
  }
  if (a.R) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      T r[8];
      load8_raw<DT>(static_cast<const T*>(a.R) + row * a.ld_r + col(i), width(i), r);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = Elem<DT>::down(Elem<DT>::up(v[i][j]) + Elem<DT>::up(r[j]));
    }
  }
  double ss = 0.0;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    if (a.S) store8_raw<DT>(static_cast<T*>(a.S) + row * a.ld_s + col(i), width(i), v[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const double x = (double)Elem<DT>::up(v[i][j]);
      ss = __builtin_fma(x, x, ss);
    }
  }
  ss += dpp_d<kRor8>(ss); ss += dpp_d<kRor4>(ss); ss += dpp_d<kRor2>(ss); ss += dpp_d<kRor1>(ss);
  ss += __shfl_xor(ss, 16);
  ss += __shfl_xor(ss, 32);
  if constexpr (NT > 64) {
    if ((t & 63) == 0) part[t >> 6] = ss;
    __syncthreads();
    ss = 0.0;
#pragma unroll
    for (int w = 0; w < NT / 64; ++w) ss += part[w];
  }
  // 1/sqrt: the estimate and two Newton steps (they would turn the estimates
  // of 0 and infinity, infinity and 0, into NaN)
  const double x = __builtin_fma(ss, a.inv_cols, a.eps);
  double rstd = __builtin_amdgcn_rsq(x);
  if (x > 0.0 && x < __builtin_inf()) {
    rstd *= __builtin_fma(-0.5 * x * rstd, rstd, 1.5);
    rstd *= __builtin_fma(-0.5 * x * rstd, rstd, 1.5);
  }
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int n = width(i);
    if constexpr (P >= 4) {   // widened anew: kept from the first pass, the row takes four times its size
      uint32_t u[sizeof v[i] / 4];
      __builtin_memcpy(u, v[i], sizeof u);
#pragma unroll
      for (int k = 0; k < (int)(sizeof u / 4); ++k) asm volatile("" : "+v"(u[k]));
      __builtin_memcpy(v[i], u, sizeof u);
    }
    G g[8];
    if constexpr (!EARLY) load8_raw<GDT>(static_cast<const G*>(a.gamma) + col(i), n, g);
    double y[8], m = 0.0, bad = 0.0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      y[j] = (double)Elem<DT>::up(v[i][j]) * rstd * (double)Elem<GDT>::up(EARLY ? gm[EARLY ? i : 0][j] : g[j]);
      m = __builtin_fmax(m, __builtin_fabs(y[j]));
      bad = __builtin_fma(y[j], 0.0, bad);   // NaN if y is NaN or infinite
    }
    // columns past the row are zeros, but with rstd = NaN or inf they are NaN:
    // then so is the row
    if (a.Y) {   // rounded once (bf16 below 2^-126: by way of fp32)
      T f[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = Elem<DT>::down(DT == GPTQ_F32 ? (float)y[j] : sticky_float(y[j]));
      store8_raw<DT>(static_cast<T*>(a.Y) + row * a.ld_y + col(i), n, f);
    }
    if (!a.codes) continue;   // the whole grid alike
    m = __builtin_fmax(m, dpp_d<kRor8>(m));
    m = __builtin_fmax(m, dpp_d<kRor4>(m));
    m = __builtin_fmax(m, dpp_d<kRor2>(m));
    m = __builtin_fmax(m, dpp_d<kRor1>(m));
    bad += dpp_d<kRor8>(bad); bad += dpp_d<kRor4>(bad);
    bad += dpp_d<kRor2>(bad); bad += dpp_d<kRor1>(bad);
    const float s = e4m3_scale(m + bad);
    const double sd = (double)s, inv = e4m3_inverse(s);
    float q[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) q[j] = e4m3_quotient(y[j], sd, inv);
    if (n > 0)
      store_codes8(a.codes + row * a.ld_c + col(i), n, e4m3_pack4(q[0], q[1], q[2], q[3]),
                   e4m3_pack4(q[4], q[5], q[6], q[7]));
    if ((t & 15) == 0 && n > 0) a.scales[row * a.kb + (t + i * NT) / 16] = s;
  }
}

template <int DT> hipError_t launch_quantize(const QArgs& a, int block_rows, hipStream_t s) {
  if (block_rows == 1) {
    int lg = 0;
    while (lg < 4 && (1 << lg) < a.kb) ++lg;
    const int64_t chunks = ceil_div(a.kb, 1 << lg), grid = chunks * ceil_div(a.rows, 16 >> lg);
    if (grid > INT32_MAX) return hipErrorInvalidValue;
    quantize_rows_kernel<DT><<<(unsigned)grid, 256, 0, s>>>(a, lg, (uint32_t)chunks);
  } else {
    const int64_t grid = a.kb * ceil_div(a.rows, kFp8Block);
    if (grid > INT32_MAX) return hipErrorInvalidValue;
    quantize_block_kernel<DT><<<(unsigned)grid, 256, 0, s>>>(a);
  }
  return hipGetLastError();
}

// Threads and pieces for a row: the fewest registers that hold it, with at
// least a wave and at most 16 of them.
template <int DT, int GDT> hipError_t launch_rmsnorm(const NArgs& a, hipStream_t s) {
  const int64_t pieces = ceil_div(a.cols, 8);
  const unsigned grid = (unsigned)a.rows;
#define GQ_NORM(NT, P) rmsnorm_kernel<DT, GDT, NT, P><<<grid, NT, 0, s>>>(a)
  if (pieces <= 64) GQ_NORM(64, 1);
  else if (pieces <= 128) GQ_NORM(128, 1);
  else if (pieces <= 256) GQ_NORM(256, 1);
  else if (pieces <= 512) GQ_NORM(256, 2);
  else if (pieces <= 1024) GQ_NORM(512, 2);
  else if (pieces <= 2048) GQ_NORM(512, 4);
  else if (pieces <= 4096) GQ_NORM(1024, 4);
  else GQ_NORM(1024, 8);
#undef GQ_NORM
  return hipGetLastError();
}

}  // namespace

hipError_t fp8_quantize_launch(const void* X, int dt, int64_t rows, int64_t cols, int64_t ld_x,
                               int block_rows, uint8_t* codes, int64_t ld_c, float* scales,
                               hipStream_t s) {
  const QArgs a{X, rows, cols, ld_x, codes, ld_c, scales, ceil_div(cols, kFp8Block)};
  switch (dt) {
    case GPTQ_F32: return launch_quantize<GPTQ_F32>(a, block_rows, s);
    case GPTQ_BF16: return launch_quantize<GPTQ_BF16>(a, block_rows, s);
    default: return launch_quantize<GPTQ_F16>(a, block_rows, s);
  }
}

hipError_t rmsnorm_fp8_launch(const void* X, int64_t ld_x, const void* R, int64_t ld_r, int dt,
                              const void* gamma, int g_dt, int64_t rows, int64_t cols, double eps,
                              void* S, int64_t ld_s, void* Y, int64_t ld_y, uint8_t* codes,
                              int64_t ld_c, float* scales, hipStream_t s) {
  const NArgs a{X, ld_x, R, ld_r, gamma, rows, cols, 1.0 / (double)cols, eps, S, ld_s, Y, ld_y, codes, ld_c, scales,
                ceil_div(cols, kFp8Block)};
  if (dt == GPTQ_F32) return launch_rmsnorm<GPTQ_F32, GPTQ_F32>(a, s);
  if (dt == GPTQ_BF16)
    return g_dt == GPTQ_F32 ? launch_rmsnorm<GPTQ_BF16, GPTQ_F32>(a, s)
                            : launch_rmsnorm<GPTQ_BF16, GPTQ_BF16>(a, s);
  return g_dt == GPTQ_F32 ? launch_rmsnorm<GPTQ_F16, GPTQ_F32>(a, s)
                          : launch_rmsnorm<GPTQ_F16, GPTQ_F16>(a, s);
}

}  // namespace gq
