// Products of block-scaled e4m3 matrices (kernels: fp8_tile.hpp; choice among
// them: fp8_launch.hpp): C = A·Bᵀ and the gated projection act(A·Gᵀ)·(A·Uᵀ).
#include "fp8_launch.hpp"

namespace gq {
namespace {

template <int FORM> hipError_t run_dt(GArgs& a, void* ws, hipStream_t s) {
  if constexpr (FORM == kGated)
    if (a.codes) return run<kGated, kCodes, GPTQ_F32>(a, ws, s);
  switch (a.c_dt) {
    case GPTQ_F32: return run<FORM, kStore, GPTQ_F32>(a, ws, s);
    case GPTQ_BF16: return run<FORM, kStore, GPTQ_BF16>(a, ws, s);
    default: return run<FORM, kStore, GPTQ_F16>(a, ws, s);
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
  return run_dt<kPlain>(a, ws, s);
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
  return run_dt<kGated>(a, ws, s);
}

}  // namespace gq
