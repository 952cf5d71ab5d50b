// Choice and launch of the products of block-scaled e4m3 matrices.
#pragma once

#include "fp8_tile.hpp"

namespace gq {
namespace {

// ---------------------------------------------------------------- choice and launch
// The kernel for a product is the one that this model says is quickest.  Its
// times are microseconds on MI355X (fp8 instructions / exact form): a stage of a
// tile with one workgroup on each of the 256 CUs, and with as many as fit; a
// round's start and epilogue.  Fitted to every kernel and split of 240 plain and
// gated products of random sizes (M to 2900, K to 10 944), of which 40 x 5760 x
// 1216 was missed by most (few rows 10.0, 32-tiles 7.3).  Small tiles win
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
// Its codes without a gate: sums go to memory 64 bytes of a row at a time, 16 rows
// and columns a store, and back (us, bytes per us).  Fitted to 176 products of 9 to
// 64 rows by 16 weights from 1024 x 4096 to 20480 x 5120 with all kernels timed
// (what is picked takes 0.7 % longer than the quickest on average, 10 % at worst;
// with the gated products' kJoin 3.0 and 28, 48 x 16384 x 2048: few rows 21.8, 64-
// tiles in two splits 17.0) and tried on 144 others, of random sizes, 1 to 64 rows
// by 512 to 20000 x 256 to 12000: 2.8 %, 38 at worst (14 x 17449 x 278: tiles of
// 128 rows 14.8, of 32 10.7); with kJoin 3.7.
constexpr double kFewJoin = 1.2, kFewJoinBytes = 7.5e5;

struct Plan { int tile; int splits, kper; };   // tile -1: few rows

// Codes of a tile that is not whole blocks wide (or of the kernel for few rows)
// go through the workspace in any case.
inline bool joins(int tile, bool gated) {
  return tile < 0 || kTiles[tile].bn / (gated ? 2 : 1) % 128 != 0;
}

// Without a workspace one split of the 256-tile
// runs for codes, any unsplit kernel otherwise.
inline Plan search_plan(int64_t M, int64_t N, int64_t K, bool gated, bool exact, bool codes, bool ws) {
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
    const double join = !codes ? 0 : gated ? kJoin : kFewJoin + (double)M * N * 8 / kFewJoinBytes;
    least = kFewLaunch + join +
            std::max((double)ceil_div(groups, 256 * here) * (kFewGroup + here * std::max(copied, issued)),
                     2.0 * groups * kb * nb / kFewWeights);
    best = {-1, 1, (int)kb};
  }
  for (int i = 0; i < kTileKinds; ++i) {
    const TileCost& c = kTiles[i];
    const bool join = codes && joins(i, gated);
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

// search_plan with the last results of each thread kept by their arguments: a
// call asks for the same few plans several times (its workspace's size and
// check, its launch), a decoding loop for the same ones at every token.
inline Plan plan_of(int64_t M, int64_t N, int64_t K, bool gated, bool exact, bool codes, bool ws) {
  struct Entry { int64_t M, N, K; int how; Plan plan; };
  static thread_local Entry kept[64] = {};
  const int how = 16 + gated + 2 * exact + 4 * codes + 8 * ws;   // never 0
  const uint64_t h = ((uint64_t)M * 0x9E3779B97F4A7C15ull + (uint64_t)N) * 0x9E3779B97F4A7C15ull + (uint64_t)K * 32 + how;
  Entry& e = kept[(h * 0x9E3779B97F4A7C15ull) >> 58];
  if (e.M != M || e.N != N || e.K != K || e.how != how)
    e = {M, N, K, how, search_plan(M, N, K, gated, exact, codes, ws)};
  return e.plan;
}

inline size_t plan_bytes(const Plan& p, int64_t M, int64_t N, bool gated, bool codes) {
  if (p.splits > 1) return (size_t)p.splits * (gated ? 2 : 1) * M * N * 4;
  return codes && joins(p.tile, gated) ? (size_t)M * N * 4 : 0;
}

template <int BM, int BN, int WM, int WN, int NS, bool FAST, int FORM, int EPI, int DT>
hipError_t launch_tile(GArgs& a, int splits, hipStream_t s) {
  using T = Tile<BM, BN, WM, WN, NS>;
  a.tm = (int)ceil_div(a.M, BM);
  a.tn = (int)ceil_div(a.N, FORM == kGated ? BN / 2 : BN);
  const int64_t grid = (int64_t)a.tm * a.tn * splits;
  if (grid > INT32_MAX) return hipErrorInvalidValue;
  tile_kernel<BM, BN, WM, WN, NS, FAST, FORM, EPI, DT><<<(unsigned)grid, T::NT, 0, s>>>(a);
  return hipGetLastError();
}

template <bool FAST, int FORM, int EPI, int DT>
hipError_t launch_kind(GArgs& a, const Plan& p, hipStream_t s) {
  switch (p.tile) {
    case 0: return launch_tile<32, 64, 16, 32, 4, FAST, FORM, EPI, DT>(a, p.splits, s);
    case 1: return launch_tile<64, 64, 32, 32, 4, FAST, FORM, EPI, DT>(a, p.splits, s);
    case 2: return launch_tile<128, 128, 64, 32, 2, FAST, FORM, EPI, DT>(a, p.splits, s);
    default: return launch_tile<256, 256, 128, 64, 2, FAST, FORM, EPI, DT>(a, p.splits, s);
  }
}

template <bool FAST, int FORM, int EPI> hipError_t launch_few(const GArgs& a, hipStream_t s) {
  const unsigned grid = (unsigned)ceil_div(a.N, 16);
#define GQ_FEW(NA) few_rows_kernel<NA, FAST, FORM, EPI><<<grid, Few<NA, FORM == kGated>::WAVES * 64, 0, s>>>(a)
  if (a.M <= 8) GQ_FEW(1);
  else if (a.M <= 16) GQ_FEW(2);
  else if (a.M <= 32) GQ_FEW(4);
  else if (a.M <= 48) GQ_FEW(6);
  else GQ_FEW(8);
#undef GQ_FEW
  return hipGetLastError();
}

// Whether copies of 16 bytes can take every row of an operand; their 32-bit
// offsets span a tile's rows.
inline bool wide_rows(const uint8_t* q, int64_t rows, int64_t ld) {
  return (uintptr_t)q % 16 == 0 && (rows == 1 || (ld % 16 == 0 && ld < ((int64_t)1 << 23)));
}

// One output form: EPI with DT (FAST goes with the 16-bit types).
template <int FORM, int EPI, int DT>
hipError_t run(GArgs& a, void* ws, hipStream_t s) {
  constexpr bool GATED = FORM == kGated, FAST = EPI == kStore && DT != GPTQ_F32, codes = EPI == kCodes;
  const Plan p = plan_of(a.M, a.N, a.K, GATED, !FAST, codes, ws != nullptr);
  a.nb = ceil_div(a.N, 128);
  a.kb = (int)ceil_div(a.K, 128);
  a.kper = p.kper;
  a.P = static_cast<float*>(ws);
  a.wide = wide_rows(a.A, a.M, a.lda) && wide_rows(a.B[0], a.N, a.ldb[0]) &&
           (!GATED || wide_rows(a.B[1], a.N, a.ldb[1]));
  const bool join = p.splits > 1 || (codes && joins(p.tile, GATED));
  hipError_t e;
  if (p.tile < 0) e = launch_few<FAST, FORM, codes ? kPartial : kStore>(a, s);
  else if (join) e = launch_kind<FAST, FORM == kLinear ? kPlain : FORM, kPartial, GPTQ_F32>(a, p, s);
  else if constexpr (codes) {
    if constexpr (!GATED)
      if (p.tile == 2) return launch_tile<128, 128, 64, 32, 2, false, FORM, kCodes, DT>(a, 1, s);
    e = launch_tile<256, 256, 128, 64, 2, false, FORM, kCodes, DT>(a, 1, s);
  } else e = launch_kind<FAST, FORM, EPI, DT>(a, p, s);
  if (e != hipSuccess || !join) return e;
  const unsigned grid = (unsigned)ceil_div(a.M * a.nb, 16);
  if (p.splits > 1) join_kernel<FORM, codes><<<grid, 256, 0, s>>>(a, p.splits);
  else join_kernel<GATED ? kPlain : FORM, codes><<<grid, 256, 0, s>>>(a, 1);   // gated: h itself
  return hipGetLastError();
}

}  // namespace
}  // namespace gq
