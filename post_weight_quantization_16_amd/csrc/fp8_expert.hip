// The experts' products in 8-bit floating point (kernels: fp8_tile.hpp):
//   h[i] = act(x[t]·G_eᵀ)·(x[t]·U_eᵀ)   for each sorted position i: expert e, token t
//   y[t] = Σ_j w[t,j]·(h[i]·D_eᵀ) + residual[t]   over the positions i of token t
//
// Positions are sorted by expert, so a tile is up to BM of one expert's rows by
// its weights' columns.  How many rows an expert has is known on the device
// alone: the grid is the most tiles there can be, and each workgroup finds its
// own from the offsets.  The first product gathers its rows as it copies them
// into LDS (a copy's addresses are the lanes' own), so no sorted copy of the
// activations is ever made; the second stores each row's sums at its slot, and
// one pass adds a token's slots, with their weights, in the order of j.
#include "fp8_tile.hpp"

namespace gq {
namespace {

// ---------------------------------------------------------------- sum over a token's experts
// One thread per eight columns of a token.
template <int DT>
__global__ __launch_bounds__(256) void combine_kernel(const float* P, const int32_t* ids, const float* weights,
                                                      int64_t T, int64_t N, int k, int E, const void* R,
                                                      int64_t ldr, void* C, int64_t ldc) {
  typedef typename Elem<DT>::type Out;
  const int64_t g = (int64_t)blockIdx.x * 256 + threadIdx.x, per = (N + 7) / 8;
  const int64_t t = g / per, n = (g - t * per) * 8;
  if (t >= T) return;
  const int c = (int)min((int64_t)8, N - n);
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = 0.f;
  for (int j = 0; j < k; ++j) {
    const int id = ids[t * k + j];
    if (id < 0 || id >= E) continue;
    const float w = weights[t * k + j];
    float v[8];
    load8<GPTQ_F32>(P + (t * k + j) * N + n, c, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = __builtin_fmaf(w, v[i], y[i]);
  }
  if (R) {
    float v[8];
    load8<DT>(static_cast<const Out*>(R) + t * ldr + n, c, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] += v[i];
  }
  store8<DT>(static_cast<Out*>(C) + t * ldc + n, c, y);
}

// ---------------------------------------------------------------- launch
// The most stretches of BM rows that `slots` rows of E experts can make.
int64_t most_stretches(int64_t slots, int64_t E, int64_t bm) {
  return std::min(slots, slots / bm + std::min(E, slots));
}

template <int BM, int BN, int WM, int WN, int NS, bool FAST, int FORM, int EPI, int DT, int ROWS>
hipError_t launch_tile(GArgs& a, hipStream_t s) {
  using T = Tile<BM, BN, WM, WN, NS>;
  a.tn = (int)ceil_div(a.N, FORM == kGated ? BN / 2 : BN);
  const int64_t grid = most_stretches(a.slots, a.E, BM) * a.tn;
  if (grid > INT32_MAX) return hipErrorInvalidValue;
  tile_kernel<BM, BN, WM, WN, NS, FAST, FORM, EPI, DT, ROWS><<<(unsigned)grid, T::NT, 0, s>>>(a);
  return hipGetLastError();
}

void finish_args(GArgs& a) {
  a.nb = ceil_div(a.N, 128);
  a.kb = (int)ceil_div(a.K, 128);
  a.kper = a.kb;
}
bool wide_rows(const uint8_t* q, int64_t rows, int64_t ld, int64_t most) {
  return (uintptr_t)q % 16 == 0 && (rows == 1 || (ld % 16 == 0 && ld * std::min(rows, most) < ((int64_t)1 << 31)));
}

}  // namespace

size_t fp8_expert_gated_ws_bytes(int64_t T, int64_t k, int64_t E, int64_t N, int64_t K) {
  return 256;
}
size_t fp8_expert_gemm_ws_bytes(int64_t T, int64_t k, int64_t E, int64_t N, int64_t K) {
  return std::max<size_t>(512, align_up((size_t)(T * k) * N * 4));
}

hipError_t fp8_expert_gated_launch(const uint8_t* A, const float* sa, int64_t T, int64_t K, int64_t lda,
                                   int k, const int32_t* offsets, const int32_t* order, int E,
                                   const uint8_t* G, const float* sg, int64_t ldg, int64_t next_g,
                                   const uint8_t* U, const float* su, int64_t ldu, int64_t next_u,
                                   int64_t N, int act, void* C, int c_dt, int64_t ldc, uint8_t* codes,
                                   int64_t ld_codes, float* sc, void* ws, hipStream_t s) {
  GArgs a{};
  a.A = A; a.sa = sa; a.M = T * k; a.K = K; a.lda = lda;
  a.B[0] = G; a.sb[0] = sg; a.ldb[0] = ldg; a.next[0] = next_g;
  a.B[1] = U; a.sb[1] = su; a.ldb[1] = ldu; a.next[1] = next_u;
  a.N = N; a.act = act;
  a.C = C; a.ldc = ldc; a.c_dt = c_dt;
  a.codes = codes; a.ld_codes = ld_codes; a.sc = sc;
  a.offsets = offsets; a.order = order; a.E = E; a.topk = k; a.slots = (int)(T * k);
  finish_args(a);
  a.wide = wide_rows(A, T, lda, T) && wide_rows(G, 2, ldg, 256) && wide_rows(U, 2, ldu, 256) &&
           next_g % 16 == 0 && next_u % 16 == 0;
  if (codes) return launch_tile<64, 256, 32, 64, 3, false, kGated, kCodes, GPTQ_F32, kGather>(a, s);
  if (c_dt == GPTQ_F32) return launch_tile<64, 256, 32, 64, 3, false, kGated, kStore, GPTQ_F32, kGather>(a, s);
  if (c_dt == GPTQ_BF16) return launch_tile<64, 256, 32, 64, 3, true, kGated, kStore, GPTQ_BF16, kGather>(a, s);
  return launch_tile<64, 256, 32, 64, 3, true, kGated, kStore, GPTQ_F16, kGather>(a, s);
}

hipError_t fp8_expert_gemm_launch(const uint8_t* A, const float* sa, int64_t T, int64_t K, int64_t lda,
                                  int k, const int32_t* ids, const float* weights, const int32_t* offsets,
                                  const int32_t* order, int E, const uint8_t* B, const float* sb,
                                  int64_t ldb, int64_t next, int64_t N, const void* R, int64_t ldr,
                                  void* C, int c_dt, int64_t ldc, void* ws, hipStream_t s) {
  GArgs a{};
  a.A = A; a.sa = sa; a.M = T * k; a.K = K; a.lda = lda;
  a.B[0] = B; a.sb[0] = sb; a.ldb[0] = ldb; a.next[0] = next;
  a.N = N; a.P = static_cast<float*>(ws);
  a.offsets = offsets; a.order = order; a.E = E; a.topk = k; a.slots = (int)(T * k);
  finish_args(a);
  a.wide = wide_rows(A, 2, lda, 256) && wide_rows(B, 2, ldb, 256) && next % 16 == 0;
  hipError_t e;
  if (c_dt == GPTQ_F32) e = launch_tile<64, 128, 32, 32, 3, false, kPlain, kPartial, GPTQ_F32, kSorted>(a, s);
  else e = launch_tile<64, 128, 32, 32, 3, true, kPlain, kPartial, GPTQ_F32, kSorted>(a, s);
  if (e != hipSuccess) return e;
  const int64_t grid = ceil_div(T * ceil_div(N, 8), 256);
  if (grid > INT32_MAX) return hipErrorInvalidValue;
#define GQ_SUM(DT) combine_kernel<DT><<<(unsigned)grid, 256, 0, s>>>(a.P, ids, weights, T, N, k, E, R, ldr, C, ldc)
  if (c_dt == GPTQ_F32) GQ_SUM(GPTQ_F32);
  else if (c_dt == GPTQ_BF16) GQ_SUM(GPTQ_BF16);
  else GQ_SUM(GPTQ_F16);
#undef GQ_SUM
  return hipGetLastError();
}

}  // namespace gq
