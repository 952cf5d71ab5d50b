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
// one pass adds a token's slots, with their weights, in the order of j.  For
// bf16 results these sums are rounded to fp16 on their way (kScaled): 2^-11 of
// each term, an eighth of what the result's own rounding may lose, for half the
// bytes (4096 tokens, top 8, 2048 columns: 227 -> 170 us).
#include "fp8_tile.hpp"

namespace gq {
namespace {

// ---------------------------------------------------------------- sum over a token's experts
// One thread per eight columns of a token.  SCALED: the terms are kScaled's.
template <int DT, bool SCALED>
__global__ __launch_bounds__(256) void combine_kernel(const void* P, int64_t nb, const int32_t* ids,
                                                      const float* weights, int64_t T, int64_t N, int k, int E,
                                                      const void* R, int64_t ldr, void* C, int64_t ldc) {
  typedef typename Elem<DT>::type Out;
  const int64_t g = (int64_t)blockIdx.x * 256 + threadIdx.x, per = (N + 7) / 8;
  const int64_t t = g / per, n = (g - t * per) * 8;
  if (t >= T) return;
  const int c = (int)min((int64_t)8, N - n);
  const _Float16* H = static_cast<const _Float16*>(P);
  const float* F = reinterpret_cast<const float*>(H + align_scaled(T * k * N));
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = 0.f;
  // four slots' loads in flight
  for (int j0 = 0; j0 < k; j0 += 4) {
    float v[4][8], w[4];
    bool on[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int64_t s = t * k + min(j0 + u, k - 1);
      const int id = ids[s];
      on[u] = j0 + u < k && id >= 0 && id < E;
      w[u] = weights[s];
      if (!on[u]) continue;
      if constexpr (SCALED) {
        load8<GPTQ_F16>(H + s * N + n, c, v[u]);
        w[u] *= F[s * nb + n / 128];
      } else {
        load8<GPTQ_F32>(static_cast<const float*>(P) + s * N + n, c, v[u]);
      }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (on[u]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = __builtin_fmaf(w[u], v[u][i], y[i]);
      }
  }
  if (R) {
    float v[8];
    load8<DT>(static_cast<const Out*>(R) + t * ldr + n, c, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] += v[i];
  }
  store8<DT>(static_cast<Out*>(C) + t * ldc + n, c, y);
}

// ---------------------------------------------------------------- few tokens
// Up to 16 tokens: y in one kernel, no sums in memory.  A workgroup owns 16
// columns and goes through every expert that a token takes, its waves sharing
// out the blocks of all of them; a lane's row is its token (lane % 16), with the
// row of H that this expert's product takes and its weight, or none.  A token
// that has an expert twice gives that expert a second pass.  Copies as in
// few_rows_kernel: each wave's own ring in LDS, its own waits.
constexpr int kTokens = 16, kTokenSlots = 128, kTokenDepth = 3, kTokenWaves = 8;

template <int NA> struct Token {
  static constexpr int PER = 2 + NA + 1;                  // copies a block: B, A, scales
  static constexpr int SLOT = 4096 + 256;                 // 16 rows of B, 16 of A; scales
  static constexpr int RING = kTokenDepth * SLOT;
  static constexpr int SMEM = kTokenWaves * RING;
};

template <int NA, bool FAST>
__global__ __launch_bounds__(kTokenWaves * 64) void token_kernel(GArgs a, const int32_t* ids, const float* weights,
                                                                  int tokens) {
  using K = Token<NA>;
  __shared__ __attribute__((aligned(1024))) char S[K::SMEM];
  __shared__ int expert_of[kTokenSlots], pass_of[kTokenSlots], token_of[kTokenSlots], again[kTokenSlots];
  __shared__ int pass_expert[kTokenSlots], passes_;
  __shared__ short row_in[kTokenSlots][kTokens];      // pass, token: row of H or -1
  __shared__ float weight_in[kTokenSlots][kTokens];
  const int t = threadIdx.x, lane = t & 63, l15 = lane & 15;
  const int w = __builtin_amdgcn_readfirstlane(t >> 6);

  // passes: the sorted positions' experts, and how often the token had each before
  const int live = offset_of(a, a.E);
  for (int i = t; i < kTokenSlots * kTokens; i += kTokenWaves * 64) (&row_in[0][0])[i] = -1;
  if (t < kTokenSlots) {
    int e = -1, tok = 0;
    if (t < live) {
      const int o = a.order[t];
      if (o >= 0 && o < a.slots) {
        e = ids[o];
        tok = (int)((unsigned)o / (unsigned)a.topk);
        if (e < 0 || e >= a.E) e = -1;
        // the weight waits in the place of its own position
        weight_in[t >> 4][t & 15] = weights[o];
      }
    }
    expert_of[t] = e;
    token_of[t] = tok;
  }
  __syncthreads();
  float mine = 0.f;
  if (t < kTokenSlots) {
    mine = weight_in[t >> 4][t & 15];
    int n = 0;
    if (expert_of[t] >= 0)
      for (int i = t - 1; i >= 0 && expert_of[i] == expert_of[t]; --i) n += token_of[i] == token_of[t];
    again[t] = n;
  }
  __syncthreads();
  int first = t;   // the first position of this one's pass
  if (t < kTokenSlots && expert_of[t] >= 0) {
    for (int i = t - 1; i >= 0 && expert_of[i] == expert_of[t]; --i)
      if (again[i] == again[t]) first = i;
  }
  const bool leads = t < kTokenSlots && expert_of[t < kTokenSlots ? t : 0] >= 0 && first == t;
  const uint64_t lead = __ballot(leads);
  if (t == 0) passes_ = __builtin_popcountll(lead);
  __syncthreads();
  if (leads) {
    const int p = (w ? passes_ : 0) + __builtin_popcountll(lead & ((1ull << lane) - 1));
    pass_of[t] = p;
    pass_expert[p] = expert_of[t];
  }
  __syncthreads();
  if (t == 64) passes_ += __builtin_popcountll(lead);
  if (t < kTokenSlots && expert_of[t] >= 0) {
    const int p = pass_of[first];
    row_in[p][token_of[t]] = (short)t;
    weight_in[p][token_of[t]] = mine;
  }
  __syncthreads();
  const int passes = __builtin_amdgcn_readfirstlane(passes_);

  const int64_t n0 = (int64_t)blockIdx.x * 16;
  const int nleft = (int)min((int64_t)16, a.N - n0);
  const int blocks = passes * a.kb, per = (blocks + kTokenWaves - 1) / kTokenWaves;
  const int begin = w * per, nblk = min(per, blocks - begin);   // may be 0 or less
  char* ring = S + w * K::RING;
  const unsigned rbase = (unsigned)(uintptr_t)(__attribute__((address_space(3))) char*)ring;
  const int last_wide = a.wide ? (a.K % 128 ? a.kb - 1 : a.kb) : 0;   // blocks from here on: through registers
  // block j of this wave: pass and block of K
  int cp = nblk > 0 ? begin / a.kb : 0, ck = nblk > 0 ? begin - cp * a.kb : 0;   // of the next copy
  auto copy = [&](int j) {
    const int slot = j % kTokenDepth;
    const int e = __builtin_amdgcn_readfirstlane(pass_expert[cp]);
    const uint8_t* B = a.B[0] + e * a.next[0] + n0 * a.ldb[0];
    i32x4 v[2 + NA];
#pragma unroll
    for (int i = 0; i < 2 + NA; ++i) {
      const int row = (i & 1) * 8 + (lane >> 3);
      const int p16 = (((lane & 7) ^ (lane >> 4)) << 4) ^ ((i & 1) << 6);
      const uint8_t* at = i < 2 ? B + (int64_t)min(row, nleft - 1) * a.ldb[0] : a.A + (int64_t)max((int)row_in[cp][row], 0) * a.lda;
      if (ck < last_wide) lds_copy16(rbase + (unsigned)(slot * K::SLOT + i * 1024), at + (int64_t)ck * 128 + p16);
      else v[i] = piece16(at, (int64_t)ck * 128 + p16, a.K);
    }
    {   // scales: lanes 0..15 the rows', the others the weights'
      const float* p = lane < 16 ? a.sa + (int64_t)max((int)row_in[cp][l15], 0) * a.kb
                                 : a.sb[0] + ((int64_t)e * a.nb + n0 / 128) * a.kb;
      lds_copy4(rbase + (unsigned)(slot * K::SLOT + 4096), p + ck);
    }
    if (ck >= last_wide) {
#pragma unroll
      for (int i = 0; i < 2 + NA; ++i) *reinterpret_cast<i32x4*>(ring + slot * K::SLOT + i * 1024 + lane * 16) = v[i];
      asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    }
    if (++ck == a.kb) {
      ck = 0;
      ++cp;
    }
  };
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  int up = cp, uk = ck;   // pass and block of the next product
#pragma unroll
  for (int j = 0; j < kTokenDepth; ++j)
    if (j < nblk) copy(j);
  const int row = l15 * 128 + (((lane >> 4) ^ ((l15 >> 1) & 7)) << 4);
  for (int j = 0; j < nblk; ++j) {
    // this block's copies have landed when no more are in flight than the later blocks'
    if (j + kTokenDepth <= nblk) asm volatile("s_waitcnt vmcnt(%0)" :: "i"((kTokenDepth - 1) * K::PER) : "memory");
    else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    const char* q = ring + (j % kTokenDepth) * K::SLOT;
    const i32x4 bx = *reinterpret_cast<const i32x4*>(q + row), by = *reinterpret_cast<const i32x4*>(q + (row ^ 64));
    const i32x4 ax = *reinterpret_cast<const i32x4*>(q + 2048 + row), ay = *reinterpret_cast<const i32x4*>(q + 2048 + (row ^ 64));
    const float sa = *reinterpret_cast<const float*>(q + 4096 + l15 * 4), sb = *reinterpret_cast<const float*>(q + 4096 + 64);
    const bool on = row_in[up][l15] >= 0;
    const float wt = weight_in[up][l15];
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // read: the slot may be written again
    if (j + kTokenDepth < nblk) copy(j + kTokenDepth);
    Frag<FAST> fb[1], fa;
    fb[0].set(bx, by);
    fa.set(ax, ay);
    f32x4 p[1];
    contract(fb, fa, p);
    const float s = sa * sb * wt;
#pragma unroll
    for (int r = 0; r < 4; ++r) acc[r] = on ? __builtin_fmaf(p[0][r], s, acc[r]) : acc[r];
    if (++uk == a.kb) {
      uk = 0;
      ++up;
    }
  }
  __syncthreads();   // the sums go where the rings were
  float* part = reinterpret_cast<float*>(S);
#pragma unroll
  for (int r = 0; r < 4; ++r) part[(w * 16 + l15) * 17 + 4 * (lane >> 4) + r] = acc[r];
  __syncthreads();
  const int m = t >> 4, c = t & 15;
  if (m >= tokens || c >= nleft) return;
  float y = 0.f;
#pragma unroll
  for (int v = 0; v < kTokenWaves; ++v) y += part[(v * 16 + m) * 17 + c];
  if (a.R) y += get1(a.R, a.c_dt, m * a.ldr + n0 + c);
  put1(a.C, a.c_dt, m * a.ldc + n0 + c, y);
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

// Rows of an expert, on average over those that can have any.
double rows_each(const GArgs& a) { return (double)a.slots / (double)std::min(a.slots, a.E); }

// Tiles by the rows an expert has.  Up to 32 rows all of them wait for the
// weights and the smallest tile that holds most experts' rows is best: a second
// one reads the weights again, if only from the L2; above, the products count.
// Gated, codes (us; 64 experts of 1024 x 2048, top 8 / 8 of 11008 x 4096, top 2):
//   rows        2 / 1         8 / 16        32 / 64       128 / 256     512 / 1024
//   16 x 256    48.9 / 116.7  67.0 / 191.1  92.8 / 360    288 / 1199    954 / 4597
//   32 x 256    51.9 / 119.1  60.3 / 164.3  70.9 / 263    189 / 723     594 / 2727
//   128 x 256   73.3 / 166.2  67.5 / 188.8  79.6 / 209    116 / 455     320 / 1469
//   256 x 256   127 / 279     103 / 257     99 / 259      177 / 469     326 / 1493
template <int EPI, int DT> hipError_t run_gated(GArgs& a, hipStream_t s) {
  constexpr bool FAST = EPI == kStore && DT != GPTQ_F32;
  const double r = rows_each(a);
  if (r < 6) return launch_tile<16, 256, 16, 32, 4, FAST, kGated, EPI, DT, kGather>(a, s);
  if (r < 48) return launch_tile<32, 256, 32, 32, 4, FAST, kGated, EPI, DT, kGather>(a, s);
  return launch_tile<128, 256, 64, 64, 2, FAST, kGated, EPI, DT, kGather>(a, s);
}
// Back, to bf16 with the sum over the slots (2048 x 1024 / 4096 x 11008):
//   rows        2 / 4         8 / 16        32 / 64       128 / 256     512 / 1024
//   16 x 128    25.6 / 112.8  37.7 / 117    45.3 / 197    117 / 454     381 / 1554
//   32 x 128    26.8 / 95.2   33.7 / 98.1   41.2 / 136    95.4 / 293    307 / 1004
//   128 x 128   29.5 / 114.4  35.1 / 111    40.9 / 123    67.1 / 219    191 / 532
//   256 x 256   39.6 / 150.7  39.3 / 148    45.3 / 154    81.0 / 198    170 / 519
template <bool FAST, int EPI> hipError_t run_sorted(GArgs& a, hipStream_t s) {
  const double r = rows_each(a);
  if (r < 4) return launch_tile<16, 128, 16, 32, 2, FAST, kPlain, EPI, GPTQ_F32, kSorted>(a, s);
  if (r < 48) return launch_tile<32, 128, 32, 32, 3, FAST, kPlain, EPI, GPTQ_F32, kSorted>(a, s);
  if (r < 200) return launch_tile<128, 128, 64, 32, 2, FAST, kPlain, EPI, GPTQ_F32, kSorted>(a, s);
  return launch_tile<256, 256, 128, 64, 2, FAST, kPlain, EPI, GPTQ_F32, kSorted>(a, s);
}

}  // namespace

size_t fp8_expert_gated_ws_bytes() { return 256; }   // none
size_t fp8_expert_gemm_ws_bytes(int64_t T, int64_t k, int64_t N) {
  if (T <= kTokens && T * k <= kTokenSlots) return 256;
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
  a.P = static_cast<float*>(ws);
  if (codes) return run_gated<kCodes, GPTQ_F32>(a, s);
  if (c_dt == GPTQ_F32) return run_gated<kStore, GPTQ_F32>(a, s);
  if (c_dt == GPTQ_BF16) return run_gated<kStore, GPTQ_BF16>(a, s);
  return run_gated<kStore, GPTQ_F16>(a, s);
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
  a.R = R; a.ldr = ldr; a.C = C; a.c_dt = c_dt; a.ldc = ldc;
  if (T <= kTokens && T * k <= kTokenSlots) {
    const unsigned grid = (unsigned)ceil_div(N, 16);
#define GQ_TOKEN(NA, FAST) token_kernel<NA, FAST><<<grid, kTokenWaves * 64, 0, s>>>(a, ids, weights, (int)T)
    if (c_dt == GPTQ_F32) {
      if (T <= 8) GQ_TOKEN(1, false);
      else GQ_TOKEN(2, false);
    } else {
      if (T <= 8) GQ_TOKEN(1, true);
      else GQ_TOKEN(2, true);
    }
#undef GQ_TOKEN
    return hipGetLastError();
  }
  if (c_dt == GPTQ_F32) e = run_sorted<false, kPartial>(a, s);
  else if (c_dt == GPTQ_BF16) e = run_sorted<true, kScaled>(a, s);
  else e = run_sorted<true, kPartial>(a, s);
  if (e != hipSuccess) return e;
  const int64_t grid = ceil_div(T * ceil_div(N, 8), 256);
  if (grid > INT32_MAX) return hipErrorInvalidValue;
#define GQ_SUM(DT, SC) combine_kernel<DT, SC><<<(unsigned)grid, 256, 0, s>>>(a.P, a.nb, ids, weights, T, N, k, E, R, ldr, C, ldc)
  if (c_dt == GPTQ_F32) GQ_SUM(GPTQ_F32, false);
  else if (c_dt == GPTQ_F16) GQ_SUM(GPTQ_F16, false);
  else GQ_SUM(GPTQ_BF16, true);
#undef GQ_SUM
  return hipGetLastError();
}

}  // namespace gq
