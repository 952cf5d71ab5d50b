// Goes through the routing plan's whole range (route_plan.hpp): prints the pairs
// "lanes v one" that it can give, and exits non-zero where a plan does not cover
// its tokens, takes more LDS than a block gets by default, has more rows of
// counts than the workspace, or needs a second block where the call promises none.
#include <cstdio>
#include <set>
#include <tuple>

#include "route_plan.hpp"

using namespace gq;

int main() {
  std::set<std::tuple<int, int, int>> seen;
  const int64_t tokens[] = {1, 2, 3, 4, 5, 7, 8, 9, 15, 16, 17, 31, 32, 33, 63, 64, 65, 100, 255, 1000, 1024, 1025, 2047,
                            2048, 2049, 4095, 4096, 4097, 16384, 16385, 65537, 1000003, 1 << 24};
  for (int64_t T : tokens)
    for (int E = 1; E <= 1024; ++E)
      for (int groups = 1; groups <= 16; ++groups) {
        if (E % groups) continue;
        for (int k : {1, 8, 64}) {
          if (k > E || T * k > (int64_t(1) << 30)) continue;
          const RoutePlan p = route_plan(T, E, k, groups);
          const int here = p.threads / p.lanes;
          const char* wrong = nullptr;
          if (p.lanes * p.v < E) wrong = "experts left out";
          if ((int64_t)p.per * p.blocks < T || p.per % here) wrong = "tokens left out";
          if (p.threads > route_threads(p.lanes, p.v)) wrong = "more threads than registers";
          if (p.lds > 65536) wrong = "LDS";
          if (p.blocks > std::min<int64_t>(kMaxBlocks, div_up(T * k, 4))) wrong = "rows of counts";
          if (T <= (E <= 256 ? 16 : 4) && !p.one) wrong = "a workspace after all";
          if (p.one && p.blocks != 1) wrong = "one block";
          if (wrong) {
            std::printf("T=%lld E=%d k=%d groups=%d: %s\n", (long long)T, E, k, groups, wrong);
            return 1;
          }
          seen.insert({p.lanes, p.v, (int)p.one});
        }
      }
  for (const auto& s : seen) std::printf("%d %d %d\n", std::get<0>(s), std::get<1>(s), std::get<2>(s));
  return 0;
}
