// act(A·Bᵀ + bias) + residual of block-scaled e4m3 matrices, rounded to 16 or
// 32 bits or quantized again in 1 x 128 blocks (kernels: fp8_tile.hpp; choice
// among them: fp8_launch.hpp).
//
// Bias, activation and residual are applied to the fp32 sums in the registers
// that hold them (where K is split: by the kernel that joins the sums), so the
// value is rounded once and the sums never reach memory.  The products and
// sums are fp8_gemm's, and so is what bounds each kernel.
#include "fp8_launch.hpp"

namespace gq {
namespace {

template <int FORM> hipError_t run_dt(GArgs& a, void* ws, hipStream_t s) {
  if (a.codes) return run<FORM, kCodes, GPTQ_F32>(a, ws, s);
  switch (a.c_dt) {
    case GPTQ_F32: return run<FORM, kStore, GPTQ_F32>(a, ws, s);
    case GPTQ_BF16: return run<FORM, kStore, GPTQ_BF16>(a, ws, s);
    default: return run<FORM, kStore, GPTQ_F16>(a, ws, s);
  }
}

}  // namespace

// enough for every output form; 256 if none uses a workspace
size_t fp8_linear_ws_bytes(int64_t M, int64_t N, int64_t K) {
  size_t most = 0;
  for (int form = 0; form < 3; ++form) {   // 16 bits, fp32, codes
    const Plan p = plan_of(M, N, K, false, form > 0, form == 2, true);
    most = std::max(most, plan_bytes(p, M, N, false, form == 2));
  }
  return most ? std::max<size_t>(512, align_up(most)) : 256;
}

hipError_t fp8_linear_launch(const uint8_t* A, const float* sa, int64_t M, int64_t K, int64_t lda,
                             const uint8_t* B, const float* sb, int64_t N, int64_t ldb,
                             const void* bias, int bias_dt, int act, const void* R, int64_t ldr,
                             void* C, int c_dt, int64_t ldc, uint8_t* codes, int64_t ld_codes,
                             float* sc, void* ws, hipStream_t s) {
  GArgs a{};
  a.A = A; a.sa = sa; a.M = M; a.K = K; a.lda = lda;
  a.B[0] = B; a.sb[0] = sb; a.N = N; a.ldb[0] = ldb;
  a.bias = bias; a.bias_dt = bias_dt; a.act = act; a.R = R; a.ldr = ldr;
  a.C = C; a.c_dt = c_dt; a.ldc = ldc;
  a.codes = codes; a.ld_codes = ld_codes; a.sc = sc;
  return run_dt<kLinear>(a, ws, s);
}

}  // namespace gq
