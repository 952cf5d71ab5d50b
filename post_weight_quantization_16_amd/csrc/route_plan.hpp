// How the tokens of a routing call are shared out: lanes a token, threads and
// blocks, LDS.  Host code alone, apart from the kernels (moe.hip), so that it can
// be checked without them.
#pragma once

#include <algorithm>
#include <cstddef>
#include <cstdint>

namespace gq {

inline int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Threads of a block of L lanes a token, V experts a lane: registers for 16 waves
// where those are few.
constexpr int route_threads(int L, int V) { return L * V <= 256 && V <= 8 ? 1024 : 256; }
constexpr int kMaxBlocks = 256;   // rows of hist: every sorting block reads them all

// How T tokens are routed.
struct RoutePlan { int lanes, v, threads, per, blocks; bool one; size_t lds; };
constexpr int64_t kFewTokens = 2048;   // up to here a token gets a wave
inline RoutePlan route_plan(int64_t T, int E, int k, int groups) {
  RoutePlan p;
  const bool one_lanes = T <= 64 && E <= 128 && groups == 1;   // one block does it all
  p.lanes = E <= 128 && T > (one_lanes ? 16 : kFewTokens) ? 16 : 64;
  p.v = 1;
  while (p.v * p.lanes < E) p.v *= 2;
  // blocks of 16 waves where one then does it all, or 256 of them fill the
  // card; with 16 lanes a token, groups' keys leave LDS for 4
  p.threads = 256;
  if (route_threads(p.lanes, p.v) == 1024 && (groups == 1 || p.lanes == 64) &&
      (T > kMaxBlocks * (256 / p.lanes) || (T > 256 / p.lanes && T <= 1024 / p.lanes)))
    p.threads = 1024;
  const int here = p.threads / p.lanes;
  p.one = T <= here;
  p.per = (int)(div_up(div_up(T, kMaxBlocks), here) * here);
  p.blocks = (int)div_up(T, std::max(p.per, 1));
  p.lds = (size_t)here * k * 12 + (groups > 1 ? (size_t)here * (E + 2 * p.lanes) * 8 : 0) + (size_t)E * 4;
  if (p.one) p.lds = std::max(p.lds, (size_t)E * (2 + p.threads / 64) * 4);
  return p;
}

}  // namespace gq
