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
// bf16 results these terms are rounded to fp16 on their way (kScaled), for half
// the bytes (4096 tokens, top 8, 2048 columns: 201 -> 156 us): up to 2^-11 of each
// term, where the result's own rounding loses up to 2^-8 of the sum.  That is an
// eighth as long as the terms do not cancel; where they or the residual do, it can
// be more than the result's half step, and a result in fp32 is the way out.
#include <cmath>

#include "fp8_tile.hpp"

namespace gq {
namespace {

// ---------------------------------------------------------------- sum over a token's experts
// One thread per eight columns of a token.  SCALED: the terms are kScaled's.
template <int DT, bool SCALED>
__global__ __launch_bounds__(256) void combine_kernel(const void* P, int group, const int32_t* ids,
                                                      const float* weights, int64_t T, int64_t N, int k, int E,
                                                      const void* R, int64_t ldr, void* C, int64_t ldc) {
  typedef typename Elem<DT>::type Out;
  const int64_t g = (int64_t)blockIdx.x * 256 + threadIdx.x, per = (N + 7) / 8;
  const int64_t t = g / per, n = (g - t * per) * 8;
  if (t >= T) return;
  const int c = (int)min((int64_t)8, N - n);
  const _Float16* H = static_cast<const _Float16*>(P);
  const float* F = reinterpret_cast<const float*>(H + align_scaled(T * k * N)) + (SCALED ? n / group : 0);
  const int64_t nf = SCALED ? (N + group - 1) / group : 0;
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = 0.f;
  // four slots' loads in flight
  for (int j0 = 0; j0 < k; j0 += 4) {
    float v[4][8], w[4], f[4];
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
        f[u] = F[s * nf];
      } else {
        load8<GPTQ_F32>(static_cast<const float*>(P) + s * N + n, c, v[u]);
      }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (on[u]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = __builtin_fmaf(w[u], SCALED ? v[u][i] * f[u] : v[u][i], y[i]);
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
// Bound: the weights' bytes (top 2 of 8 experts of 4096 x 11008, one token: 18.8
// us, 4.8 TB/s), with several tokens the waves' instructions beside them.  Us for
// 1 / 4 / 16 tokens, in brackets the stream of 32-row tiles and the sum after it:
//   top 8 of 64, 2048 x 1024      7.5 (15.5)   14.3 (19.9)   33.3 (31.4)
//   top 2 of 8, 4096 x 11008     19.0 (54.6)   53.8 (73.7)   90.0 (97.7)
//   top 8 of 256, 4096 x 512      7.7 (16.2)   15.1 (23.4)   42.6 (52.9)
//   top 4 of 16, 1024 x 4096      9.0 (25.4)   16.6 (25.8)   25.0 (26.0)
// From 8 tokens on the two are near each other and the tiles, with more waves for
// the same bytes, can win (8 / 9 / 12 / 16 tokens of two other runs: top 8 of 128, 2048
// x 768, 20.6 (27.0), 24.4 (27.7), 30.4 (31.9), 35.6 (35.7); top 4 of 128, 2880 x 2880,
// 63.8 (62.3), 70.9 (59.2), 76.2 (71.3), 89.7 (84.4)); the bound is one number all
// the same, so that a token's result does not change its terms' type with the size
// of the weights.
constexpr int kTokens = 16, kTokenSlots = 128;

// WAVES: 8, or 16 where there are few columns (16 tokens, top 4 of 16, 1024 x
// 4096: 50.7 us with 8 and the addresses above, 25.0 with 16).
template <int NA, int WAVES> struct Token {
  static constexpr int PER = 2 + NA + 1;                  // copies a block: B, A, scales
  static constexpr int DEPTH = WAVES == 16 ? 2 : 4;       // blocks in flight
  static constexpr int SC = 2048 + NA * 1024;             // 16 rows of B, 8·NA of A; scales
  static constexpr int SLOT = SC + 256;
  static constexpr int RING = DEPTH * SLOT;
  static constexpr int SMEM = WAVES * RING + (NA == 1 ? 1024 : 0);   // rows 8 to 15 of A: read, not used
};

template <int NA, bool FAST, int WAVES>
__global__ __launch_bounds__(WAVES * 64) void token_kernel(GArgs a, const int32_t* ids, const float* weights,
                                                           int tokens) {
  using K = Token<NA, WAVES>;
  __shared__ __attribute__((aligned(1024))) char S[K::SMEM];
  __shared__ int expert_of[kTokenSlots], pass_of[kTokenSlots], token_of[kTokenSlots], again[kTokenSlots];
  __shared__ int pass_expert[kTokenSlots], passes_;
  __shared__ short row_in[kTokenSlots][kTokens];      // pass, token: row of H or -1
  __shared__ float weight_in[kTokenSlots][kTokens];
  const int t = threadIdx.x, lane = t & 63, l15 = lane & 15;
  const int w = __builtin_amdgcn_readfirstlane(t >> 6);

  // passes: the sorted positions' experts, and how often the token had each before
  const int live = offset_of(a, a.E);
  for (int i = t; i < kTokenSlots * kTokens; i += WAVES * 64) (&row_in[0][0])[i] = -1;
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
  const int blocks = passes * a.kb, per = (blocks + WAVES - 1) / WAVES;
  const int begin = w * per, nblk = min(per, blocks - begin);   // may be 0 or less
  char* ring = S + w * K::RING;
  const unsigned rbase = (unsigned)(uintptr_t)(__attribute__((address_space(3))) char*)ring;
  // pass and block of K of the next copy, and what a pass has for it: the
  // expert's weights and scales, each lane's row of H.  A pass's addresses are
  // formed once: with new ones at every block the waves' instructions took
  // longer than the bytes (8 tokens, top 1 of 8, 2048 x 4096: 17.7 us, now 11.8).
  int cp = nblk > 0 ? begin / a.kb : 0, ck = nblk > 0 ? begin - cp * a.kb : 0;
  const uint8_t* B = nullptr;
  const float* scale = nullptr;
  uint32_t boff[2], aoff[NA];
  auto p16_of = [&](int i) { return (((lane & 7) ^ (lane >> 4)) << 4) ^ ((i & 1) << 6); };
#pragma unroll
  for (int i = 0; i < 2; ++i) boff[i] = (uint32_t)min(i * 8 + (lane >> 3), nleft - 1) * (uint32_t)a.ldb[0] + p16_of(i);
  auto turn = [&] {
    const int e = __builtin_amdgcn_readfirstlane(pass_expert[cp]);
    B = a.B[0] + (int64_t)e * a.next[0] + n0 * a.ldb[0];
#pragma unroll
    for (int i = 0; i < NA; ++i) aoff[i] = (uint32_t)max((int)row_in[cp][i * 8 + (lane >> 3)], 0) * (uint32_t)a.lda + p16_of(i);
    // lanes 0..15 the rows' scales, the others the weights'
    scale = lane < 16 ? a.sa + (int64_t)max((int)row_in[cp][l15], 0) * a.kb
                      : a.sb[0] + ((int64_t)e * a.nb + n0 / 128) * a.kb;
  };
  const int full = a.wide ? (int)(a.K / 128) : 0;   // blocks that are whole
  auto copy = [&](int j) {
    const unsigned to = (unsigned)((j % K::DEPTH) * K::SLOT);
    const int64_t k = (int64_t)ck * 128;
    if (ck < full) {
#pragma unroll
      for (int i = 0; i < 2; ++i) lds_copy16(rbase + to + i * 1024, B + k, boff[i]);
#pragma unroll
      for (int i = 0; i < NA; ++i) lds_copy16(rbase + to + 2048 + i * 1024, a.A + k, aoff[i]);
      lds_copy4(rbase + to + K::SC, scale + ck);
    } else if (a.wide && a.K % 16 == 0) {
#pragma unroll
      for (int i = 0; i < 2; ++i) lds_copy16(rbase + to + i * 1024, within(B + k + boff[i], k + p16_of(i) < a.K));
#pragma unroll
      for (int i = 0; i < NA; ++i)
        lds_copy16(rbase + to + 2048 + i * 1024, within(a.A + k + aoff[i], k + p16_of(i) < a.K));
      lds_copy4(rbase + to + K::SC, scale + ck);
    } else {   // through registers; rows at any stride
      i32x4 v[2 + NA];
#pragma unroll
      for (int i = 0; i < 2 + NA; ++i) {
        const int row = (i & 1) * 8 + (lane >> 3);
        const uint8_t* at = i < 2 ? B + (int64_t)min(row, nleft - 1) * a.ldb[0] : a.A + (int64_t)max((int)row_in[cp][row], 0) * a.lda;
        v[i] = piece16(at, k + p16_of(i), a.K);
      }
      lds_copy4(rbase + to + K::SC, scale + ck);
#pragma unroll
      for (int i = 0; i < 2 + NA; ++i) *reinterpret_cast<i32x4*>(ring + to + i * 1024 + lane * 16) = v[i];
      asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    }
    if (++ck == a.kb) {
      ck = 0;
      if (++cp < passes) turn();
    }
  };
  if (nblk > 0) turn();
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  int up = cp, uk = ck;   // pass and block of the next product; whether the lane's token takes it
  bool on = nblk > 0 && row_in[up][l15] >= 0;
  float wt = nblk > 0 ? weight_in[up][l15] : 0.f;
#pragma unroll
  for (int j = 0; j < K::DEPTH; ++j)
    if (j < nblk) copy(j);
  const int row = l15 * 128 + (((lane >> 4) ^ ((l15 >> 1) & 7)) << 4);
  for (int j = 0; j < nblk; ++j) {
    // this block's copies have landed when no more are in flight than the later blocks'
    if (j + K::DEPTH <= nblk) asm volatile("s_waitcnt vmcnt(%0)" :: "i"((K::DEPTH - 1) * K::PER) : "memory");
    else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    const char* q = ring + (j % K::DEPTH) * K::SLOT;
    const i32x4 bx = *reinterpret_cast<const i32x4*>(q + row), by = *reinterpret_cast<const i32x4*>(q + (row ^ 64));
    const i32x4 ax = *reinterpret_cast<const i32x4*>(q + 2048 + row), ay = *reinterpret_cast<const i32x4*>(q + 2048 + (row ^ 64));
    const float sa = *reinterpret_cast<const float*>(q + K::SC + l15 * 4), sb = *reinterpret_cast<const float*>(q + K::SC + 64);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // read: the slot may be written again
    if (j + K::DEPTH < nblk) copy(j + K::DEPTH);
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
      if (++up < passes) {
        on = row_in[up][l15] >= 0;
        wt = weight_in[up][l15];
      }
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
  for (int v = 0; v < WAVES; ++v) y += part[(v * 16 + m) * 17 + c];
  if (a.R) y += get1(a.R, a.c_dt, m * a.ldr + n0 + c);
  put1(a.C, a.c_dt, m * a.ldc + n0 + c, y);
}

// ---------------------------------------------------------------- few gated columns
// Gate and up for up to eight rows of one expert and 16 columns a workgroup, its
// waves sharing out the blocks of K, each with a ring of its own in LDS: for few
// tokens over few columns, where tiles of 128 columns leave most of the card idle.
// Codes, one and two tokens (us, with the join's launch; in brackets the tiles and
// their number): top 8 of 64 of 1024 x 2048 13.8 (16.3, 64), 20.9 (18.1, 120);
// top 8 of 256 of 512 x 4096 15.4 (26.7, 32), 19.8 (28.4, 62); top 1 of 8 of 4096
// x 2048 10.8 (16.1, 32), 14.6 (16.3, 60).
// WAVES: 8, or 4 with two workgroups a CU where there are more than 256.
template <int WAVES> struct FewGated {
  static constexpr int PER = 4 + 1 + 1;                   // copies a block: gate, up, rows, scales
  static constexpr int DEPTH = 3;
  static constexpr int SC = 5 * 1024, SLOT = SC + 256;
  static constexpr int RING = DEPTH * SLOT;
  static constexpr int SMEM = WAVES * RING + 1024;        // rows 8 to 15: read, not used
};

template <bool FAST, int EPI, int WAVES>
__global__ __launch_bounds__(WAVES * 64) void few_gated_kernel(GArgs a) {
  using K = FewGated<WAVES>;
  __shared__ __attribute__((aligned(1024))) char S[K::SMEM];
  __shared__ int offs[kMaxExperts + 1];
  const int t = threadIdx.x, lane = t & 63, l15 = lane & 15;
  const int w = __builtin_amdgcn_readfirstlane(t >> 6);
  for (int e = t; e <= a.E; e += WAVES * 64) offs[e] = offset_of(a, e);
  __syncthreads();
  const uint32_t u = blockIdx.x / (uint32_t)a.tn;
  const Stretches<8> all(offs, a.E, a.slots);
  if (u >= (uint32_t)all.total) return;
  const int64_t n0 = (int64_t)(blockIdx.x - u * a.tn) * 16;
  const Stretch s = all.find(offs, a.E, __builtin_amdgcn_readfirstlane((int)u));
  const int nleft = (int)min((int64_t)16, a.N - n0);
  // each lane's token for the copies of rows (eight lanes a row), and for those of scales
  auto token = [&](int row) -> int {
    const int o = a.order[s.row + min(row, s.rows - 1)];
    return (unsigned)o < (unsigned)a.slots ? (int)((unsigned)o / (unsigned)a.topk) : 0;
  };
  const int mine = token(lane >> 3);
  const uint8_t *G = a.B[0] + s.expert * a.next[0] + n0 * a.ldb[0], *U = a.B[1] + s.expert * a.next[1] + n0 * a.ldb[1];
  const int64_t sb = ((int64_t)s.expert * a.nb + n0 / 128) * a.kb;
  const float* scale = lane < 16 ? a.sa + (int64_t)token(l15) * a.kb : (lane < 32 ? a.sb[0] : a.sb[1]) + sb;
  auto p16_of = [&](int i) { return (((lane & 7) ^ (lane >> 4)) << 4) ^ ((i & 1) << 6); };
  uint32_t off[5];
#pragma unroll
  for (int i = 0; i < 5; ++i)
    off[i] = (i < 4 ? (uint32_t)min((i & 1) * 8 + (lane >> 3), nleft - 1) * (uint32_t)a.ldb[i / 2 & 1]
                    : (uint32_t)mine * (uint32_t)a.lda) + p16_of(i);
  const int per = (a.kb + WAVES - 1) / WAVES, kbeg = w * per, nblk = min(per, a.kb - kbeg);   // may be 0 or less
  char* ring = S + w * K::RING;
  const unsigned rbase = (unsigned)(uintptr_t)(__attribute__((address_space(3))) char*)ring;
  const int full = a.wide ? (int)(a.K / 128) : 0;
  auto copy = [&](int j) {
    const unsigned to = (unsigned)((j % K::DEPTH) * K::SLOT);
    const int64_t k = (int64_t)(kbeg + j) * 128;
    if (kbeg + j < full) {
#pragma unroll
      for (int i = 0; i < 5; ++i) lds_copy16(rbase + to + i * 1024, (i < 2 ? G : i < 4 ? U : a.A) + k, off[i]);
    } else if (a.wide && a.K % 16 == 0) {
#pragma unroll
      for (int i = 0; i < 5; ++i)
        lds_copy16(rbase + to + i * 1024, within((i < 2 ? G : i < 4 ? U : a.A) + k + off[i], k + p16_of(i) < a.K));
    } else {   // through registers; rows at any stride
      i32x4 v[5];
#pragma unroll
      for (int i = 0; i < 5; ++i) {
        const uint8_t* at = i < 4 ? (i < 2 ? G : U) + (int64_t)min((i & 1) * 8 + (lane >> 3), nleft - 1) * a.ldb[i / 2 & 1]
                                  : a.A + (int64_t)mine * a.lda;
        v[i] = piece16(at, k + p16_of(i), a.K);
      }
#pragma unroll
      for (int i = 0; i < 5; ++i) *reinterpret_cast<i32x4*>(ring + to + i * 1024 + lane * 16) = v[i];
      asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    }
    lds_copy4(rbase + to + K::SC, scale + kbeg + j);
  };
  f32x4 acc[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
  for (int j = 0; j < K::DEPTH; ++j)
    if (j < nblk) copy(j);
  const int row = l15 * 128 + (((lane >> 4) ^ ((l15 >> 1) & 7)) << 4);
  for (int j = 0; j < nblk; ++j) {
    // this block's copies have landed when no more are in flight than the later blocks'
    if (j + K::DEPTH <= nblk) asm volatile("s_waitcnt vmcnt(%0)" :: "i"((K::DEPTH - 1) * K::PER) : "memory");
    else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    const char* q = ring + (j % K::DEPTH) * K::SLOT;
    i32x4 x[3], y[3];
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      x[i] = *reinterpret_cast<const i32x4*>(q + i * 2048 + row);
      y[i] = *reinterpret_cast<const i32x4*>(q + i * 2048 + (row ^ 64));
    }
    const float* sc = reinterpret_cast<const float*>(q + K::SC);
    const float sa = sc[l15], sg = sc[16], su = sc[32];
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // read: the slot may be written again
    if (j + K::DEPTH < nblk) copy(j + K::DEPTH);
    Frag<FAST> fb[2], fa;
    fb[0].set(x[0], y[0]);
    fb[1].set(x[1], y[1]);
    fa.set(x[2], y[2]);
    f32x4 p[2];
    contract(fb, fa, p);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      acc[0][r] = __builtin_fmaf(p[0][r], sa * sg, acc[0][r]);
      acc[1][r] = __builtin_fmaf(p[1][r], sa * su, acc[1][r]);
    }
  }
  __syncthreads();   // the sums go where the rings were
  float* part = reinterpret_cast<float*>(S);
#pragma unroll
  for (int b = 0; b < 2; ++b)
#pragma unroll
    for (int r = 0; r < 4; ++r) part[((w * 2 + b) * 16 + l15) * 17 + 4 * (lane >> 4) + r] = acc[b][r];
  __syncthreads();
  const int m = t >> 4, c = t & 15;
  if (m >= s.rows || c >= nleft) return;
  float g = 0.f, h = 0.f;
#pragma unroll
  for (int v = 0; v < WAVES; ++v) {
    g += part[(v * 2 * 16 + m) * 17 + c];
    h += part[((v * 2 + 1) * 16 + m) * 17 + c];
  }
  h *= activate(g, a.act);
  const int64_t at = s.row + m;
  if constexpr (EPI == kPartial) a.P[at * a.N + n0 + c] = h;
  else put1(a.C, a.c_dt, at * a.ldc + n0 + c, h);
}

// ---------------------------------------------------------------- stream of tiles
// The tile kernel's loop (fp8_tile.hpp) over many tiles a workgroup, as one
// stream of stages: while a tile's last stages are multiplied the first ones of
// the workgroup's next tile are copied, so that a tile costs its stages and its
// stores, and not the way there (finding the expert, its rows, the first bytes)
// that a workgroup of its own would wait for.  The products of a token's slots
// back are short (8 stages for 1024 columns).
// The slots of a tile's rows come with copies of 4 bytes a lane like the scales;
// three tables of them, for the wave that still stores the tile before, this
// tile and the next.
// FLOW: that; otherwise one tile a workgroup.  A stage of a stream is slower (more
// scalars than there are registers for), so long products go without.  With a
// stream / without, to bf16, us by blocks of K:
//   experts, rows, columns   4             8             12            20            48
//   64 of 24, 2048           24.5 / 26.3   35.6 / 35.9   53.1 / 52.9   84.9 / 81.6   176 / 173
//   64 of 128, 2048          46.9 / 49.9   66.9 / 69.8   88.8 / 89.9   131 / 130     253 / 243
//   16 of 200, 4096          36.3 / 36.9   43.6 / 44.1   53.2 / 52.7   78.2 / 75.5   150 / 151
//   64 of 512, 2048          126 / 130     175 / 175     229 / 224     317 / 315     613 / 591
//   16 of 512, 4096          69.3 / 70.1   89.7 / 87.8   116 / 113     168 / 160     335 / 319
// Tiles of 32 rows, which wait for the weights, stream at any length: between 6 %
// less and 5 % more.
constexpr int kFlowBlocks = 10;
template <int BM, int BN, int WM, int WN, int NS, int EPI, bool FLOW> struct Stream {
  using T = Tile<BM, BN, WM, WN, NS>;
  static constexpr int ROWS = BM < 64 ? 64 : BM;   // of a table: a copy fills 64
  static constexpr int TOP = EPI == kCodes ? BN / WN * BM : 1;
  static constexpr int TABLES = FLOW ? 3 : 1;
  static constexpr int LDS = T::SMEM + 4 * (kMaxExperts + 1 + TABLES * ROWS + TOP) + 64;
  static constexpr int FIT = 163840 / LDS;         // workgroups a CU
  static_assert(FIT >= 1, "LDS");
  static constexpr int WPE = FIT * T::WAVES / 4 > 8 ? 8 : FIT * T::WAVES / 4;
};

template <int BM, int BN, int WM, int WN, int NS, bool FAST, int FORM, int EPI, int DT, int ROWS, bool FLOW>
__global__ __launch_bounds__((Tile<BM, BN, WM, WN, NS>::NT), (Stream<BM, BN, WM, WN, NS, EPI, FLOW>::WPE)) void stream_kernel(GArgs a) {
  using T = Tile<BM, BN, WM, WN, NS>;
  using Q = Stream<BM, BN, WM, WN, NS, EPI, FLOW>;
  constexpr bool GATED = FORM == kGated;
  constexpr int MI = T::MI, NI = T::NI, NB = GATED ? 2 : 1;
  constexpr int G = !FAST && MI * NI < 32 && NI % 2 == 0 ? 2 : 1;
  constexpr int FIRST = FAST && MI * NI == 32 ? T::PER / 2 : T::PER;
  constexpr int BC = BN / NB, WC = WN / NB;
  __shared__ __attribute__((aligned(1024))) char S[T::SMEM];
  __shared__ int offs[kMaxExperts + 1];
  __shared__ int slots_[Q::TABLES][Q::ROWS];
  __shared__ uint32_t top[Q::TOP];
  const int t = threadIdx.x, lane = t & 63;
  const int w = __builtin_amdgcn_readfirstlane(t >> 6);
  const int wm = w / (BN / WN), wn = w % (BN / WN);
  for (int e = t; e <= a.E; e += T::NT) offs[e] = offset_of(a, e);
  __syncthreads();
  const Stretches<BM> all(offs, a.E, a.slots);
  const uint32_t tiles = (uint32_t)all.total * a.tn;
  if (blockIdx.x >= tiles) return;
  struct Where { int e, m0, mleft, n0; };
  auto where = [&](uint32_t L) -> Where {
    uint32_t bm, bn;
    tile_of(L, tiles, all.total, a.tn, bm, bn);
    const Stretch s = all.find(offs, a.E, __builtin_amdgcn_readfirstlane((int)bm));
    return {s.expert, s.row, s.rows, __builtin_amdgcn_readfirstlane((int)bn * BC)};
  };
  const int nst = a.kb;
  const bool flow = FLOW && nst > NS;   // enough stages for the next tile's tables to arrive
  const unsigned sbase = (unsigned)(uintptr_t)(__attribute__((address_space(3))) char*)S;
  const unsigned tbase = (unsigned)(uintptr_t)(__attribute__((address_space(3))) int*)&slots_[0][0];
  const int last_wide = a.wide ? (a.K % 128 ? a.kb - 1 : a.kb) : 0;

  auto copy_slots = [&](const Where& p, int b) {
#pragma unroll
    for (int i = w; i < Q::ROWS / 64; i += T::WAVES)
      lds_copy4(tbase + (unsigned)(b * Q::ROWS * 4 + i * 256), a.order + p.m0 + min(i * 64 + lane, p.mleft - 1));
  };
  auto token = [&](int b, int row) -> int {   // of a tile's row; a slot that does not exist: any
    const int o = slots_[b][row];
    return (unsigned)o < (unsigned)a.slots ? (int)((unsigned)o / (unsigned)a.topk) : 0;
  };
  auto copy_scales = [&](const Where& p, int b, int g, int half) {
    int l = lane;
    asm volatile("" : "+v"(l));
    const int r = l >> 3, k = min(8 * g + (l & 7), a.kb - 1);
#pragma unroll 1
    for (int idx = w; idx < T::SCOPIES; idx += T::WAVES) {
      const float* q;
      if (idx < BM / 8) {
        const int64_t row = ROWS == kGather ? (int64_t)token(b, idx * 8 + r) : (int64_t)p.m0 + min(idx * 8 + r, p.mleft - 1);
        q = a.sa + row * a.kb;
      } else {
        const int64_t blk = (int64_t)p.e * a.nb + p.n0 / 128;
        if (GATED) q = (r == 0 ? a.sb[0] : a.sb[NB - 1]) + blk * a.kb;
        else q = a.sb[0] + (blk + min(min(r, 1), (int)a.nb - 1 - p.n0 / 128)) * a.kb;
      }
      lds_copy4(sbase + T::SCALES + (unsigned)((half & 1) * T::SCB + idx * 256), q + k);
    }
  };
  // where the copies of stages are: bases and the lanes' offsets
  const uint8_t *base_a = nullptr, *base_b = nullptr, *base_u = nullptr;
  uint32_t voff[T::PER];
  Where from{};   // the tile that is copied, and its table
  int from_tab = 0;
  auto copy_from = [&](const Where& p, int b) {
    from = p;
    from_tab = b;
    base_a = ROWS == kGather ? a.A : a.A + (int64_t)p.m0 * a.lda;
    base_b = a.B[0] + (int64_t)p.e * a.next[0] + (int64_t)p.n0 * a.ldb[0];
    if constexpr (GATED) base_u = a.B[1] + (int64_t)p.e * a.next[1] + (int64_t)p.n0 * a.ldb[1];
    const int nleft = (int)min((int64_t)BC, a.N - p.n0);
    int l = lane;
    asm volatile("" : "+v"(l));   // once a tile: not worth registers
#pragma unroll
    for (int i = 0; i < T::PER; ++i) {
      const int seg = T::seg(w, i), row = seg * 8 + (l >> 3);
      const int p16 = (((l & 7) ^ (l >> 4)) << 4) ^ ((seg & 1) << 6);
      if (seg < BM / 8) {
        voff[i] = (uint32_t)(ROWS == kGather ? token(b, row) : min(row, p.mleft - 1)) * (uint32_t)a.lda + p16;
      } else {
        const int half = GATED && seg >= (BM + BC) / 8;
        voff[i] = (uint32_t)min(row - BM - half * BC, nleft - 1) * (uint32_t)a.ldb[half] + p16;
      }
    }
  };
  auto seg_base = [&](int seg) { return seg < BM / 8 ? base_a : GATED && seg >= (BM + BC) / 8 ? base_u : base_b; };
  // copies i0 .. i1 - 1 of block st of K, into the ring's stage n
  auto copy = [&](int st, int n, int i0, int i1) {
    const unsigned buf = (unsigned)((n % NS) * T::SB);
    if (st < last_wide) {
#pragma unroll
      for (int i = i0; i < i1; ++i) {
        const int seg = T::seg(w, i);
        lds_copy16(sbase + buf + (unsigned)seg * 1024u, seg_base(seg) + (int64_t)st * 128, voff[i]);
      }
    } else if (a.wide && a.K % 16 == 0) {   // a last block that K cuts between two pieces
#pragma unroll
      for (int i = i0; i < i1; ++i) {
        const int seg = T::seg(w, i);
        int l = lane;
        asm volatile("" : "+v"(l));
        const int p16 = (((l & 7) ^ (l >> 4)) << 4) ^ ((seg & 1) << 6);
        lds_copy16(sbase + buf + (unsigned)seg * 1024u,
                   within(seg_base(seg) + voff[i] + (int64_t)st * 128, st * 128 + p16 < a.K));
      }
    } else if (i0 == 0) {   // through registers; offsets of rows at any stride, in 64 bits
#pragma unroll 1
      for (int i = 0; i < T::PER; ++i) {
        int l = lane;
        asm volatile("" : "+v"(l));
        const int seg = T::seg(w, i), row = seg * 8 + (l >> 3);
        const int p16 = (((l & 7) ^ (l >> 4)) << 4) ^ ((seg & 1) << 6);
        const uint8_t* q;
        if (seg < BM / 8) {
          const int r = ROWS == kGather ? token(from_tab, row) : min(row, from.mleft - 1);
          q = base_a + (int64_t)r * a.lda;
        } else {
          const int half = GATED && seg >= (BM + BC) / 8;
          q = (half ? base_u : base_b) + (int64_t)min(row - BM - half * BC, (int)min((int64_t)BC, a.N - from.n0) - 1) * a.ldb[half];
        }
        *reinterpret_cast<i32x4*>(S + buf + seg * 1024 + l * 16) = piece16(q, (int64_t)st * 128 + p16, a.K);
      }
      asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    }
  };

  f32x4 acc[NI][MI];
  const int l15 = lane & 15, sw = ((lane >> 4) ^ ((l15 >> 1) & 7)) << 4;
  const int arow = (wm * WM + l15) * 128 + sw;
  const int brow = (BM + wn * WC + l15) * 128 + sw;
  const int soff = T::SCALES + (wm * WM + l15) * 32;
  const int boff = T::SCALES + BM * 32 + (GATED ? 0 : wn * WC / 128 * 32);
  struct Raw { i32x4 x, y; };
  auto read_b = [&](const char* b, int j) -> Raw {
    const int off = brow + (GATED ? (j / (NI / 2)) * BC * 128 + (j % (NI / 2)) * 2048 : j * 2048);
    return {*reinterpret_cast<const i32x4*>(b + off), *reinterpret_cast<const i32x4*>(b + (off ^ 64))};
  };
  auto read_a = [&](const char* b, int i) -> Raw {
    const int off = arow + i * 2048;
    return {*reinterpret_cast<const i32x4*>(b + off), *reinterpret_cast<const i32x4*>(b + (off ^ 64))};
  };

  uint32_t L = blockIdx.x;
  Where cur = where(L), next = cur;
  int ring = 0, half = 0, tab = 0;   // stages, groups of scales and tables before this tile (mod NS, 2, 3)
  bool fresh = true, ready = false;  // no copies are under way; the first pieces are in registers
  const int groups = (nst + 7) >> 3;
  // the stage at which the next tile's first scales are asked for: when their
  // buffer is free, and with its first stage if that is later
  const int ask = max(8 * (groups - 1), nst - NS + 1);
  Frag<FAST> fb[NI], fa;
  Raw ra;
  float sb[NB], sa, sn;
  for (;;) {
    const bool last = !FLOW || L + gridDim.x >= tiles;
    if (!last) next = where(L + gridDim.x);
    const bool more = flow && !last;
    const int tab2 = tab == 2 ? 0 : tab + 1;
    if (fresh) {
      copy_slots(cur, tab);
      if constexpr (ROWS == kGather) asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
      copy_from(cur, tab);
      copy_scales(cur, tab, 0, half);
      for (int s0 = 0; s0 < NS - 1 && s0 < nst; ++s0) copy(s0, ring + s0, 0, T::PER);
      stage_barrier<T::PER>(min(nst - 1, NS - 2));
      ready = false;
    }
    if (more) copy_slots(next, tab2);
    // what stage st asks for: the first copies, scales; then the others
    auto ask_for = [&](int st) {
      const int c = st + NS - 1;
      if (c == nst && more) copy_from(next, tab2);
      if (more && st == ask) copy_scales(next, tab2, 0, half + groups);
      if (c < nst) copy(c, ring + c, 0, FIRST);
      else if (more) copy(c - nst, ring + c, 0, FIRST);
      if ((st & 7) == 0 && st + 8 < nst) copy_scales(cur, tab, (st >> 3) + 1, half + (st >> 3) + 1);
    };
    auto ask_rest = [&](int st) {
      const int c = st + NS - 1;
      if (c < nst) copy(c, ring + c, FIRST, T::PER);
      else if (more) copy(c - nst, ring + c, FIRST, T::PER);
    };
    // the copies that may be in flight behind stage st: none of those that the
    // next tile's first stage reads
    auto ahead = [&](int st) {
      if (!more) return min(nst - 1, st + NS - 1) - (st + 1);
      return st == nst - 1 && ask > nst - NS + 1 ? 0 : NS - 2;
    };
    const bool idle = wm * WM >= cur.mleft;   // none of the wave's rows exist: copies only
    if (idle) {
      for (int st = 0; st < nst; ++st) {
        ask_for(st);
        if (FIRST < T::PER) ask_rest(st);
        stage_barrier<T::PER>(ahead(st));
      }
      ready = false;
    } else {
#pragma unroll
      for (int j = 0; j < NI; ++j)
#pragma unroll
        for (int i = 0; i < MI; ++i) acc[j][i] = f32x4{0.f, 0.f, 0.f, 0.f};
      if (!ready) {
        const char* b = S + (ring % NS) * T::SB;
        const char* sc = S + (half & 1) * T::SCB;
#pragma unroll
        for (int j = 0; j < NI; ++j) { const Raw r = read_b(b, j); fb[j].set(r.x, r.y); }
        ra = read_a(b, 0);
        sn = *reinterpret_cast<const float*>(sc + soff);
#pragma unroll
        for (int q = 0; q < NB; ++q) sb[q] = *reinterpret_cast<const float*>(sc + boff + 32 * q);
      }
      for (int st = 0; st < nst; ++st) {
        ask_for(st);
        const char* sc = S + ((half + (st >> 3)) & 1) * T::SCB + (st & 7) * 4;
        const char* sc_ = st + 1 < nst ? S + ((half + ((st + 1) >> 3)) & 1) * T::SCB + ((st + 1) & 7) * 4
                                       : S + ((half + groups) & 1) * T::SCB;
        const char* b = S + ((ring + st) % NS) * T::SB;
        const char* bn_ = S + ((ring + st + 1) % NS) * T::SB;
        f32x4 p[G];
        float sp[G] = {}, s[NB];
#pragma unroll
        for (int i = 0; i < MI; ++i) {
          if (i == 1 && FIRST < T::PER) ask_rest(st);
          fa.set(ra.x, ra.y);
          sa = sn;
#pragma unroll
          for (int q = 0; q < NB; ++q) s[q] = sa * sb[q];
          if (i + 1 < MI) {
            ra = read_a(b, i + 1);
            sn = *reinterpret_cast<const float*>(sc + soff + (i + 1) * 512);
          } else {
            stage_barrier<T::PER>(ahead(st));
          }
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int j = 0; j < NI; j += G) {
            f32x4 q[G];
            contract(&fb[j], fa, q);
#pragma unroll
            for (int g = 0; g < G; ++g) {
              if (i + j > 0) asm volatile("" : "+v"(q[g]), "+v"(p[g]));
              else asm volatile("" : "+v"(q[g]));
            }
            if (i + 1 == MI) {   // the next stage's pieces (where there is none: unused bytes)
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
                asm volatile("" : "+v"(acc[pj + g][pi]));
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
      ready = more;
      const int nleft = (int)min((int64_t)BC, a.N - cur.n0);
      int l = lane;
      asm volatile("" : "+v"(l));
      const int l15 = l & 15, nl = wn * WC + 4 * (l >> 4);   // this lane's first column in the tile
      constexpr int NO = GATED ? NI / 2 : NI;
      if constexpr (EPI == kPartial || EPI == kScaled) {
        // kScaled: P is fp16 [slots][N], behind it the powers of two, one for a row
        // of the wave's columns
        constexpr int GROUP = WC;
        const int64_t nf = (a.N + GROUP - 1) / GROUP;
        _Float16* P = reinterpret_cast<_Float16*>(a.P);
        float* F = reinterpret_cast<float*>(P + align_scaled((int64_t)a.slots * a.N));
        // kPartial: sixteen rows at a time go through LDS, so that neighbouring
        // lanes store neighbouring bytes: the part of the last stage's place in the
        // ring that this wave itself fills next; nobody reads it any more.  (64
        // experts of 2048 x 1024, 512 rows: 235.6 -> 201.6 us; for kScaled, 128 bytes
        // of a row to a wave, a swap of lanes was better: 166.9 -> 153.8, with LDS 161.7.)
        constexpr int U = WN / 4, PIECE = 16 * U * 16, TURNS = 2 * PIECE <= T::PER * 1024 ? 2 : 1;
        static_assert(PIECE <= T::PER * 1024 && T::SEGS % T::WAVES == 0, "place for a piece of sums");
        char* mine = S + ((ring + nst + NS - 1) % NS) * T::SB + w * T::PER * 1024;
        // kScaled: each row's largest (columns that do not exist hold another
        // column's sums).  x + 0·x is x, and NaN where x is infinite.
        float most[EPI == kScaled ? MI : 1];
        if constexpr (EPI == kScaled) {
          bool beyond = false;
#pragma unroll
          for (int i = 0; i < MI; ++i) {
            most[i] = 0.f;
#pragma unroll
            for (int j = 0; j < NI; ++j) {
              most[i] = largest(most[i], acc[j][i][0], acc[j][i][1]);
              most[i] = largest(most[i], acc[j][i][2], acc[j][i][3]);
            }
            beyond |= most[i] == kInfinity;
          }
          if (__builtin_expect(__ballot(beyond) != 0, 0)) {
#pragma unroll
            for (int i = 0; i < MI; ++i) {
              most[i] = 0.f;
#pragma unroll
              for (int j = 0; j < NI; ++j)
#pragma unroll
                for (int r = 0; r < 4; r += 2)
                  most[i] = largest(most[i], __builtin_fmaf(acc[j][i][r], 0.f, acc[j][i][r]),
                                    __builtin_fmaf(acc[j][i][r + 1], 0.f, acc[j][i][r + 1]));
            }
          }
        }
#pragma unroll
        for (int i = 0; i < MI; ++i) {
          if constexpr (EPI == kScaled) {
            const int ml = wm * WM + i * 16 + l15;
            const int64_t row = slots_[tab][ml];
            const bool there = ml < cur.mleft && row >= 0 && row < a.slots;
            const int e = scaled_exponent(quarters_max(__builtin_bit_cast(uint32_t, most[i])));
            const float f = power_of_two(-e);
            if (there && lane < 16 && nl < nleft) F[row * nf + (cur.n0 + nl) / GROUP] = power_of_two(e);
#pragma unroll
            for (int j = 0; j < NI; ++j)
#pragma unroll
              for (int r = 0; r < 4; ++r) acc[j][i][r] *= f;
            put_row<GPTQ_F16, NI>(P, row * a.N + cur.n0 + wn * WC, there ? nleft - wn * WC : 0, acc, i, l);
          } else {
            char* buf = mine + i % TURNS * PIECE;
#pragma unroll
            for (int j = 0; j < NI; ++j)
              *reinterpret_cast<f32x4*>(buf + (l15 * U + ((4 * j + (l >> 4)) ^ (l15 & (U - 1)))) * 16) = acc[j][i];
            wave_sync();
#pragma unroll
            for (int q = 0; q < U / 4; ++q) {
              const int r = q * (64 / U) + l / U, u = l % U, ml = wm * WM + i * 16 + r;
              const f32x4 x = *reinterpret_cast<const f32x4*>(buf + (r * U + (u ^ (r & (U - 1)))) * 16);
              const int64_t row = slots_[tab][ml];
              const int n = wn * WC + u * 4;
              if (ml < cur.mleft && row >= 0 && row < a.slots)
                put4<GPTQ_F32>(a.P, row * a.N + cur.n0 + n, nleft - n, x);
            }
            wave_sync();
          }
        }
      } else {
        const Activation act(a.act);
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
          for (int j = 0; j < NO; ++j) {
            acc[j][i] = act(acc[j][i]);
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[j][i][r] *= acc[NO + j][i][r];
          }
        if constexpr (EPI == kStore) {
#pragma unroll
          for (int i = 0; i < MI; ++i) {
            const int ml = wm * WM + i * 16 + l15;
            put_row<DT, NO>(a.C, ((int64_t)cur.m0 + ml) * a.ldc + cur.n0 + wn * WC,
                            ml < cur.mleft ? nleft - wn * WC : 0, acc, i, l);
          }
        }
      }
    }
    if constexpr (EPI == kCodes) {
      // the tile's 128 columns are one block of its rows
      static_assert(EPI != kCodes || BC == 128, "a tile is one block wide");
      constexpr int NO = NI / 2;
      const int nleft = (int)min((int64_t)BC, a.N - cur.n0);
      int l = lane;
      asm volatile("" : "+v"(l));
      const int l15 = l & 15, nl = wn * WC + 4 * (l >> 4);
      if (!idle) {
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
      }
      // without waiting for the copies under way
      asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
      if (!idle) {
#pragma unroll
        for (int i = 0; i < MI; ++i) {
          const int ml = wm * WM + i * 16 + l15;
          uint32_t u = 0;
#pragma unroll
          for (int q = 0; q < BN / WN; ++q) u = max(u, top[q * BM + ml]);
          const float s = e4m3_scale((double)__builtin_bit_cast(float, u));
          const float inv = 1.f / s;
          if (ml >= cur.mleft) continue;
          const int64_t row = (int64_t)cur.m0 + ml;
          if (wn == 0 && lane < 16) a.sc[row * a.nb + cur.n0 / 128] = s;
#pragma unroll
          for (int j = 0; j < NO; ++j) {
            const uint32_t c = codes4(acc[j][i][0], acc[j][i][1], acc[j][i][2], acc[j][i][3], s, inv);
            uint8_t* o = a.codes + row * a.ld_codes + cur.n0 + nl + j * 16;
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
    if (last) break;
    L += gridDim.x;
    cur = next;
    ring = (ring + nst) % NS;
    half = (half + groups) & 1;
    tab = tab2;
    fresh = !flow;
  }
}

// ---------------------------------------------------------------- launch
template <int BM, int BN, int WM, int WN, int NS, bool FAST, int FORM, int EPI, int DT, int ROWS, bool FLOW = false>
hipError_t launch_tiles(GArgs& a, hipStream_t s) {
  a.tn = (int)ceil_div(a.N, FORM == kGated ? BN / 2 : BN);
  a.group = WN;
  const int64_t most = most_stretches<int64_t>(a.slots, a.E, BM) * a.tn;
  if (most > INT32_MAX) return hipErrorInvalidValue;
  // FLOW: as many workgroups as run at once (a multiple of 8: each stays with its XCD's tiles)
  const unsigned grid = (unsigned)(FLOW ? std::min<int64_t>(most, 256 * Stream<BM, BN, WM, WN, NS, EPI, FLOW>::FIT) : most);
  stream_kernel<BM, BN, WM, WN, NS, FAST, FORM, EPI, DT, ROWS, FLOW>
      <<<grid, Tile<BM, BN, WM, WN, NS>::NT, 0, s>>>(a);
  return hipGetLastError();
}

void finish_args(GArgs& a) {
  a.nb = ceil_div(a.N, 128);
  a.kb = (int)ceil_div(a.K, 128);
  a.kper = a.kb;
}
// Whether copies of 16 bytes can take the rows of an operand, `span` of which the
// 32-bit offsets from one base reach over.
bool wide_rows(const uint8_t* q, int64_t ld, int64_t span) {
  return (uintptr_t)q % 16 == 0 && ld % 16 == 0 && ld <= ((int64_t)1 << 31) / span;
}

// Rows of an expert, on average over those that can have any.
double rows_each(const GArgs& a) { return (double)a.slots / (double)std::min(a.slots, a.E); }

// Whether tiles of 128 columns would leave most of the card idle: their number,
// from the experts that so many tokens take if they like all alike.
bool few_gated(int64_t slots, int64_t E, int64_t k, int64_t N) {
  if (slots > 64) return false;
  const double hit = E * (1.0 - std::pow(1.0 - (double)k / E, (double)(slots / k)));
  return hit * ceil_div(N, 128) < 80;
}

// Tiles by the rows an expert has.  Up to 32 rows all of them wait for the
// weights and the smallest tile that holds most experts' rows is best: a second
// one reads the weights again, if only from the L2; above, the products count.
// Gated, codes (us; 64 experts of 1024 x 2048, top 8 / 8 of 11008 x 4096, top 2):
//   rows        2 / 1         8 / 16        32 / 64       128 / 256     512 / 1024
//   16 x 256    48.9 / 116.7  67.0 / 191.1  92.8 / 360    288 / 1199    954 / 4597
//   32 x 256    51.9 / 119.1  60.3 / 164.3  70.9 / 263    189 / 723     594 / 2727
//   64 x 256    57.2 / 131.7  58.3 / 167.0  86.1 / 239    137 / 533     424 / 1933
//   128 x 256   73.3 / 166.2  67.5 / 188.8  79.6 / 209    116 / 455     320 / 1469
//   256 x 256   127 / 279     103 / 257     99 / 259      177 / 469     326 / 1493
// Bound, from 128 rows on: issue.  The exact form converts both operands in
// every wave, two conversions for each product of a 64 x 64 wave, and adds each
// block's sums; 8 experts of 1024 rows run at 1.0 PFLOP/s.
template <int EPI, int DT> hipError_t run_gated(GArgs& a, hipStream_t s) {
  constexpr bool FAST = EPI == kStore && DT != GPTQ_F32;
  const double r = rows_each(a);
  if (few_gated(a.slots, a.E, a.topk, a.N) && (EPI != kCodes || a.P)) {
    constexpr int E = EPI == kCodes ? kPartial : kStore;
    a.tn = (int)ceil_div(a.N, 16);
    const unsigned grid = (unsigned)(most_stretches<int64_t>(a.slots, a.E, 8) * a.tn);
    if (grid <= 256) few_gated_kernel<FAST, E, 8><<<grid, 512, 0, s>>>(a);
    else few_gated_kernel<FAST, E, 4><<<grid, 256, 0, s>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || EPI != kCodes) return e;
    join_kernel<kPlain, true, kGather><<<(unsigned)ceil_div(a.M * a.nb, 16), 256, 0, s>>>(a, 1);
    return hipGetLastError();
  }
  if (r < 6) return launch_tiles<16, 256, 16, 32, 4, FAST, kGated, EPI, DT, kGather>(a, s);
  if (r < 48) return launch_tiles<32, 256, 32, 32, 4, FAST, kGated, EPI, DT, kGather>(a, s);
  return launch_tiles<128, 256, 64, 64, 2, FAST, kGated, EPI, DT, kGather>(a, s);
}
// Back, to bf16 with the sum over the slots (streams; us; 64 experts of 2048 x
// 1024, top 8 / 256 of 4096 x 512, top 8; before sums were stored 64 bytes of a row
// at a time, which took 3 to 9 % off from 64 rows on):
//   rows        8 / 2         32 / 8        128 / 32      512 / 128
//   16 x 128    34.6 / 97     48.6 / 124    122 / 204     403 / 608
//   32 x 128    32.1 / 99     38.0 / 125    86 / 177      276 / 437
//   64 x 128    35.4 / 113    46.5 / 144    89 / 200      274 / 465
//   128 x 128   35.7 / 110    42.6 / 142    68 / 185      189 / 344
//   128 x 256   33.4 / 98     40.8 / 125    63 / 172      177 / 322
//   256 x 256   39.6 / 121    45.3 / 151    87 / 200      167 / 367
// (exact 256-row tiles have no registers left).  Where a tile of 128 rows for
// each expert leaves three CUs in four idle, small tiles win for as long as those
// would be one to an expert (16 experts of 1024 x 4096, 64 tiles, 64 / 96 / 128
// rows: 32.5 / 33.2 / 48.4 against 44.9 / 47.0 / 47.6; with twice the columns
// 54.4 / 63.6 against 48.5 / 51.4).  Bound: at few rows the weights' bytes; at many
// (64 experts of 512 rows) 2.2 us a stage of a tile, as in a plain product of this
// size, and 9 us a tile for its stores, of 26, in five rounds of tiles where whole
// ones would make four.  Two ways to keep the next tile's stages from waiting for
// stores gained nothing: sums held in registers and stored a piece at a time under
// them (188 us in place of 184, 128 x 256), the copies of one stage more ahead of
// the stores (159.0 in place of 157.1).
template <bool FAST, int EPI> hipError_t run_sorted(GArgs& a, hipStream_t s) {
  const double r = rows_each(a);
  const bool few = r <= 112 && std::min(a.slots, a.E) * ceil_div(a.N, 256) <= 64;
  if (r < 48 || few) return launch_tiles<32, 128, 32, 32, 3, FAST, kPlain, EPI, GPTQ_F32, kSorted, true>(a, s);
  if (!FAST || r < 300) {
    if (a.kb > kFlowBlocks) return launch_tiles<128, 256, 64, 64, 3, FAST, kPlain, EPI, GPTQ_F32, kSorted, false>(a, s);
    return launch_tiles<128, 256, 64, 64, 3, FAST, kPlain, EPI, GPTQ_F32, kSorted, true>(a, s);
  }
  if constexpr (FAST) {
    if (a.kb > kFlowBlocks) return launch_tiles<256, 256, 128, 64, 2, FAST, kPlain, EPI, GPTQ_F32, kSorted, false>(a, s);
    return launch_tiles<256, 256, 128, 64, 2, FAST, kPlain, EPI, GPTQ_F32, kSorted, true>(a, s);
  }
  return hipErrorInvalidValue;
}

}  // namespace

size_t fp8_expert_gated_ws_bytes(int64_t T, int64_t k, int64_t E, int64_t N) {
  return few_gated(T * k, E, k, N) ? std::max<size_t>(512, align_up((size_t)(T * k) * N * 4)) : 256;
}
size_t fp8_expert_gemm_ws_bytes(int64_t T, int64_t k, int64_t N) {
  if (T <= kTokens && T * k <= kTokenSlots) return 256;
  // fp32 terms, or fp16 ones with a power of two for each 32 columns or 64
  const int64_t n = T * k * N;
  return std::max<size_t>(512, align_up((size_t)std::max(n * 4, align_scaled(n) * 2 + T * k * ceil_div(N, 32) * 4)));
}

hipError_t fp8_expert_gated_launch(const uint8_t* A, const float* sa, int64_t T, int64_t K, int64_t lda,
                                   int k, const int32_t* offsets, const int32_t* order, int E,
                                   const uint8_t* G, const float* sg, int64_t ldg, int64_t next_g,
                                   const uint8_t* U, const float* su, int64_t ldu, int64_t next_u,
                                   int64_t N, int act, void* C, int c_dt, int64_t ldc, uint8_t* codes,
                                   int64_t ld_codes, float* sc, void* ws, hipStream_t s) {
  // a row alone has no next one
  if (T == 1) lda = 0;
  if (N == 1) ldg = ldu = 0;
  GArgs a{};
  a.A = A; a.sa = sa; a.M = T * k; a.K = K; a.lda = lda;
  a.B[0] = G; a.sb[0] = sg; a.ldb[0] = ldg; a.next[0] = next_g;
  a.B[1] = U; a.sb[1] = su; a.ldb[1] = ldu; a.next[1] = next_u;
  a.N = N; a.act = act;
  a.C = C; a.ldc = ldc; a.c_dt = c_dt;
  a.codes = codes; a.ld_codes = ld_codes; a.sc = sc;
  a.offsets = offsets; a.order = order; a.E = E; a.topk = k; a.slots = (int)(T * k);
  finish_args(a);
  a.wide = wide_rows(A, lda, T) && wide_rows(G, ldg, 256) && wide_rows(U, ldu, 256) && next_g % 16 == 0 &&
           next_u % 16 == 0;
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
  if (T * k == 1) lda = 0;
  if (N == 1) ldb = 0;
  GArgs a{};
  a.A = A; a.sa = sa; a.M = T * k; a.K = K; a.lda = lda;
  a.B[0] = B; a.sb[0] = sb; a.ldb[0] = ldb; a.next[0] = next;
  a.N = N; a.P = static_cast<float*>(ws);
  a.offsets = offsets; a.order = order; a.E = E; a.topk = k; a.slots = (int)(T * k);
  finish_args(a);
  a.wide = wide_rows(A, lda, 256) && wide_rows(B, ldb, 256) && next % 16 == 0;
  hipError_t e;
  a.R = R; a.ldr = ldr; a.C = C; a.c_dt = c_dt; a.ldc = ldc;
  if (T <= kTokens && T * k <= kTokenSlots) {
    const unsigned grid = (unsigned)ceil_div(N, 16);
#define GQ_TOKEN(NA, FAST, W) token_kernel<NA, FAST, W><<<grid, W * 64, 0, s>>>(a, ids, weights, (int)T)
#define GQ_TOKENS(FAST) \
  do { \
    if (grid <= 128) { \
      if (T <= 8) GQ_TOKEN(1, FAST, 16); \
      else GQ_TOKEN(2, FAST, 16); \
    } else if (T <= 8) GQ_TOKEN(1, FAST, 8); \
    else GQ_TOKEN(2, FAST, 8); \
  } while (0)
    if (c_dt == GPTQ_F32) GQ_TOKENS(false);
    else GQ_TOKENS(true);
#undef GQ_TOKENS
#undef GQ_TOKEN
    return hipGetLastError();
  }
  if (c_dt == GPTQ_F32) e = run_sorted<false, kPartial>(a, s);
  else if (c_dt == GPTQ_BF16) e = run_sorted<true, kScaled>(a, s);
  else e = run_sorted<true, kPartial>(a, s);
  if (e != hipSuccess) return e;
  const int64_t grid = ceil_div(T * ceil_div(N, 8), 256);
  if (grid > INT32_MAX) return hipErrorInvalidValue;
#define GQ_SUM(DT, SC) combine_kernel<DT, SC><<<(unsigned)grid, 256, 0, s>>>(a.P, a.group, ids, weights, T, N, k, E, R, ldr, C, ldc)
  if (c_dt == GPTQ_F32) GQ_SUM(GPTQ_F32, false);
  else if (c_dt == GPTQ_F16) GQ_SUM(GPTQ_F16, false);
  else GQ_SUM(GPTQ_BF16, true);
#undef GQ_SUM
  return hipGetLastError();
}

}  // namespace gq
