// Routing to experts: scores, the choice among them, weights, and the slots
// sorted by expert, which the experts' products take.
//
//   p = softmax(l) or 1/(1 + e^-l);  c = p + bias (without a bias: by l)
//   groups: the top_groups best by the sum of their group_top best c
//   ids = the top_k largest c of these groups, ties to the lowest index
//   w = p[ids], over their sum where asked, times scale
//
// Whole numbers leave this file, so a choice may not depend on a rounding:
// c and the groups' sums are fp64 (fp32 sigmoids of near logits fall together
// from 12 on, and a sum with a bias rounds again).  Where the order is the
// logits' own (no bias; groups by their best), no score is formed for it at
// all: the largest cost, an fp64 exponential for every expert, falls away, and
// weights that are renormalised need those of the chosen experts alone.
//
// Bound: latency.  The logits of 16384 tokens over 128 experts are 4 MB, less
// than a microsecond of the memory's time.
#include "fp8.hpp"

namespace gq {
namespace {

struct RouteArgs {
  const void* X; int dt; int T, E; int64_t ld;
  const float* bias; const uint8_t* mask;
  int scores, k, groups, top_groups, group_top, renorm;
  double scale;
  int32_t* ids; float* weights; int32_t* offsets; int32_t* order;
  int32_t* hist;     // [blocks][E] chosen slots of each block's tokens
  int per, blocks;   // tokens of a block
};

// ---------------------------------------------------------------- slots by expert
// A stable counting sort of slot numbers by expert.  Block b's slots come
// behind those of the blocks before it (their counts in hist), wave by wave;
// within 64 slots a lane finds the others of its expert by one ballot for each
// bit of the expert's number, and its rank among them by their count below it.
// Nothing depends on the order of atomics: those count, and nothing else.
// LDS: total [E], first [E], counts [waves][E].
// What a wave's lanes wrote is read by its other lanes behind this.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

__device__ __forceinline__ void sort_slots(const int32_t* ids, int i0, int i1, int E, int slots, const int32_t* hist,
                           int blocks, int block, int32_t* offsets, int32_t* order, int* lds) {
  const int t = threadIdx.x, nt = blockDim.x, lane = t & 63, w = t >> 6, waves = nt >> 6;
  int* total = lds;
  int* first = lds + E;
  int* counts = lds + 2 * E;
  for (int e = t; e < 2 * E; e += nt) lds[e] = 0;
  for (int e = t; e < waves * E; e += nt) counts[e] = 0;
  __syncthreads();
  const int stretch = ((i1 - i0 + waves - 1) / waves + 63) / 64 * 64;
  const int b = min(i1, i0 + w * stretch), end = min(i1, b + stretch);
  for (int i = b + lane; i < end; i += 64) {
    const int e = ids[i];
    if (e >= 0 && e < E) atomicAdd(&counts[w * E + e], 1);
  }
  if (hist) {   // all blocks' counts, and those of the blocks before this one
    const int parts = max(1, nt / E);
    for (int e0 = 0; e0 < E; e0 += nt) {
      const int part = t / E, e = e0 + (E < nt ? t - part * E : t);
      if (part >= parts || e >= E) continue;
      int all = 0, before = 0;
#pragma unroll 8
      for (int q = part; q < blocks; q += parts) {
        const int h = hist[(int64_t)q * E + e];
        all += h;
        before += q < block ? h : 0;
      }
      atomicAdd(&total[e], all);
      atomicAdd(&first[e], before);
    }
  }
  __syncthreads();
  if (!hist) {
    for (int e = t; e < E; e += nt) {
      int all = 0;
      for (int v = 0; v < waves; ++v) all += counts[v * E + e];
      total[e] = all;
    }
    __syncthreads();
  }
  if (w == 0) {   // where each expert begins
    const int per = (E + 63) >> 6;
    int sum = 0;
    for (int j = 0; j < per; ++j)
      if (lane * per + j < E) sum += total[lane * per + j];
    int in = sum;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int y = __shfl_up(in, d);
      if (lane >= d) in += y;
    }
    int at = in - sum;
    for (int j = 0; j < per; ++j) {
      const int e = lane * per + j;
      if (e < E) {
        const int n = total[e];
        first[e] += at;
        if (block == 0) offsets[e] = at;
        at += n;
      }
    }
    if (lane == 63) {
      lds[0] = at;   // the slots that have an expert; total[] is not needed any more
      if (block == 0) offsets[E] = at;
    }
  }
  __syncthreads();
  for (int i = lds[0] + block * nt + t; i < slots; i += blocks * nt) order[i] = -1;
  for (int e = t; e < E; e += nt) {
    int at = first[e];
    for (int v = 0; v < waves; ++v) {
      const int n = counts[v * E + e];
      counts[v * E + e] = at;
      at += n;
    }
  }
  __syncthreads();
  const int bits = 32 - __builtin_clz(E);   // numbers 0 .. E, E for none
  for (int i = b; i < end; i += 64) {
    int e = i + lane < end ? ids[i + lane] : E;
    if (e < 0 || e > E) e = E;
    uint64_t same = ~0ull;
    for (int q = 0; q < bits; ++q) {
      const uint64_t one = __ballot((e >> q) & 1);
      same &= (e >> q) & 1 ? one : ~one;
    }
    const int rank = __builtin_popcountll(same & ((1ull << lane) - 1));
    const int at = e < E ? counts[w * E + e] : 0;
    wave_sync();
    if (e < E) {
      order[at + rank] = i + lane;
      if (rank == 0) counts[w * E + e] = at + __builtin_popcountll(same);
    }
    wave_sync();
  }
}

__global__ __launch_bounds__(512) void sort_kernel(const int32_t* ids, int per, int slots, int E,
                                                   const int32_t* hist, int blocks, int32_t* offsets,
                                                   int32_t* order) {
  extern __shared__ int lds[];
  const int i0 = (int)min((int64_t)blockIdx.x * per, (int64_t)slots), i1 = (int)min((int64_t)i0 + per, (int64_t)slots);
  sort_slots(ids, i0, i1, E, slots, hist, blocks, blockIdx.x, offsets, order, lds);
}

__global__ __launch_bounds__(512) void count_kernel(const int32_t* ids, int per, int slots, int E, int32_t* hist) {
  extern __shared__ int lds[];
  for (int e = threadIdx.x; e < E; e += blockDim.x) lds[e] = 0;
  __syncthreads();
  const int64_t i0 = (int64_t)blockIdx.x * per, i1 = min(i0 + per, (int64_t)slots);
  for (int64_t i = i0 + threadIdx.x; i < i1; i += blockDim.x) {
    const int e = ids[i];
    if (e >= 0 && e < E) atomicAdd(&lds[e], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += blockDim.x) hist[(int64_t)blockIdx.x * E + e] = lds[e];
}

// ---------------------------------------------------------------- choice
__device__ __forceinline__ float larger(float a, float b) { return fmaxf(a, b); }
__device__ __forceinline__ double larger(double a, double b) { return fmax(a, b); }
template <int CTRL> __device__ __forceinline__ float turned(float x) {
  const int b = __builtin_bit_cast(int, x);
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(b, b, CTRL, 0xF, 0xF, false));
}
template <int CTRL> __device__ __forceinline__ double turned(double x) { return dpp_d<CTRL>(x); }
// Maximum and sum over the L lanes of a token (every lane gets them).
template <int L, typename T> __device__ __forceinline__ T lanes_max(T v) {
  v = larger(v, turned<kRor8>(v));
  v = larger(v, turned<kRor4>(v));
  v = larger(v, turned<kRor2>(v));
  v = larger(v, turned<kRor1>(v));
  if constexpr (L == 64) {
    v = larger(v, __shfl_xor(v, 16));
    v = larger(v, __shfl_xor(v, 32));
  }
  return v;
}
template <int L> __device__ __forceinline__ double lanes_sum(double v) {
  v += turned<kRor8>(v);
  v += turned<kRor4>(v);
  v += turned<kRor2>(v);
  v += turned<kRor1>(v);
  if constexpr (L == 64) {
    v += __shfl_xor(v, 16);
    v += __shfl_xor(v, 32);
  }
  return v;
}
// The lowest lane of the token for which `yes` holds, or L.
template <int L> __device__ __forceinline__ int lanes_first(bool yes, int lane) {
  uint64_t m = __ballot(yes);
  if constexpr (L < 64) m = (m >> (lane & ~(L - 1))) & ((1ull << L) - 1);
  return m ? (int)__builtin_ctzll(m) : L;
}
__device__ __forceinline__ double sigmoid(double x) { return 1.0 / (1.0 + exp(-x)); }

template <bool S> struct KeyOf { typedef float type; };
template <> struct KeyOf<true> { typedef double type; };

// L lanes a token, V neighbouring experts a lane, so that the lowest lane with
// the largest key holds the lowest expert with it.  Sixteen lanes reduce by DPP
// alone; 64 where 16 would hold more than 16 experts each.
// SCORED: the choice needs p (a bias, or groups by their best two); otherwise
// the keys are the logits, in fp32, which holds them exactly.
// ONE: one block routes all tokens and sorts their slots too.
constexpr int route_threads(int L, int V) { return L == 16 && V <= 8 ? 1024 : 256; }
template <int L, int V, bool SCORED, bool ONE>
__global__ __launch_bounds__(route_threads(L, V)) void route_kernel(RouteArgs a) {
  typedef typename KeyOf<SCORED>::type Key;
  extern __shared__ double smem[];
  const int t = threadIdx.x, lane = t & 63, l = lane & (L - 1);
  const int here = blockDim.x / L, mine = t / L;   // tokens at a time, this thread's
  double* P = smem + mine * a.k;                                   // [here][k]: what was chosen
  double* rest = smem + here * a.k;
  Key* K = reinterpret_cast<Key*>(rest) + mine * a.E;              // [here][E], groups only
  if (a.groups > 1) rest += here * a.E;
  int* I = reinterpret_cast<int*>(rest) + mine * a.k;              // [here][k]
  int* hist = reinterpret_cast<int*>(rest) + here * a.k;           // [E]
  const bool count = !ONE && a.hist;
  if (count) {
    for (int e = t; e < a.E; e += blockDim.x) hist[e] = 0;
    __syncthreads();
  }
  const float none = -__builtin_inff();
  const bool soft = a.scores == 0;
  const int64_t begin = (int64_t)blockIdx.x * a.per, end = min(begin + a.per, (int64_t)a.T);
  for (int64_t tok0 = begin; tok0 < end; tok0 += here) {
    const int64_t tok = tok0 + mine;
    const bool live = tok < end;
    const bool on = live && (!a.mask || a.mask[tok]);
    float x[V];
    bool nan = false;
    float top = none;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int e = l * V + j;
      x[j] = none;
      if (on && e < a.E) x[j] = get1(a.X, a.dt, tok * a.ld + e);
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
      nan |= x[j] != x[j] || (soft && x[j] == __builtin_inff());
      top = fmaxf(top, x[j]);
    }
    double sum = 1.0, shift = 0.0;   // softmax: of all exponentials, the largest logit
    if (soft) {
      top = lanes_max<L>(top);
      shift = top > none ? top : 0.f;
      if (SCORED || !a.renorm) {
        sum = 0.0;
#pragma unroll
        for (int j = 0; j < V; ++j)
          if (x[j] > none) sum += exp((double)x[j] - shift);
        sum = lanes_sum<L>(sum);
      }
    }
    Key key[V];
    double p[SCORED ? V : 1];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      key[j] = x[j];
      if constexpr (SCORED) {
        const int e = l * V + j;
        p[j] = 0.0;
        if (x[j] > none) {
          p[j] = soft ? exp((double)x[j] - shift) / sum : sigmoid(x[j]);
          if (a.bias) {
            key[j] = p[j] + (double)a.bias[e];
            nan |= key[j] != key[j];
          }
        }
      }
    }
    nan = lanes_first<L>(nan, lane) < L;
    if (a.groups > 1) {
      const int size = a.E / a.groups;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int e = l * V + j;
        if (e >= a.E) continue;
        if constexpr (SCORED) K[e] = !a.bias && key[j] > none && a.group_top == 2 ? p[j] : key[j];
        else K[e] = key[j];
      }
      wave_sync();
      // lane g: group g, from a place of its own on, so that the lanes read different banks
      Key one = none, two = none;
      if (l < a.groups) {
        int q = l % size;
        for (int i = 0; i < size; ++i) {
          const Key v = K[l * size + q];
          two = larger(two, v < one ? v : one);
          one = larger(one, v);
          q = q + 1 < size ? q + 1 : 0;
        }
      }
      Key score = a.group_top == 2 && two > none ? one + two : one;
      uint32_t kept = 0;
      for (int r = 0; r < a.top_groups; ++r) {
        const Key best = lanes_max<L>(score);
        const int g = lanes_first<L>(best > none && score == best, lane);
        if (g < L) kept |= 1u << g;
        if (l == g) score = none;
      }
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int e = l * V + j;
        if (e < a.E && !((kept >> (e / size)) & 1)) key[j] = none;
      }
    }
    Key lead = key[0];
#pragma unroll
    for (int j = 1; j < V; ++j) lead = larger(lead, key[j]);
    for (int r = 0; r < a.k; ++r) {
      const Key best = lanes_max<L>(lead);
      const int win = lanes_first<L>(best > none && lead == best, lane);
      if (win == L) {   // nothing is left
        if (l == 0) I[r] = -1;
      } else if (l == win) {
        int at = -1;
        double value = 0.0;
        lead = none;
#pragma unroll
        for (int j = 0; j < V; ++j) {
          if (at < 0 && key[j] == best) {
            at = j;
            if constexpr (SCORED) value = p[j];
            else value = x[j];
            key[j] = none;
          }
          lead = larger(lead, key[j]);
        }
        I[r] = l * V + at;
        P[r] = value;
      }
    }
    wave_sync();
    double whole = 0.0, kept = 0.0;
    for (int r = l; r < a.k; r += L) {
      if (I[r] < 0) continue;
      double v = P[r];
      if constexpr (!SCORED) {
        v = soft ? exp(v - shift) / sum : sigmoid(v);
        P[r] = v;
      }
      whole += v;
      kept += 1.0;
    }
    if (a.renorm) {
      whole = lanes_sum<L>(whole);
      kept = lanes_sum<L>(kept);
    }
    for (int r = l; r < a.k; r += L) {
      int id = I[r];
      double v = id < 0 ? 0.0 : P[r];
      if (a.renorm && id >= 0) v = whole > 0.0 ? v / whole : 1.0 / kept;
      v *= a.scale;
      if (nan) {   // the token's output shall say so; its experts are the first ones
        id = r;
        v = __builtin_nan("");
      }
      if (live) {
        a.ids[tok * a.k + r] = id;
        a.weights[tok * a.k + r] = id < 0 ? 0.f : (float)v;
        if (count && id >= 0) atomicAdd(&hist[id], 1);
      }
    }
    wave_sync();
  }
  if constexpr (ONE) {
    __threadfence_block();
    __syncthreads();
    sort_slots(a.ids, 0, a.T * a.k, a.E, a.T * a.k, nullptr, 1, 0, a.offsets, a.order, reinterpret_cast<int*>(smem));
  } else if (count) {
    __syncthreads();
    for (int e = t; e < a.E; e += blockDim.x) a.hist[(int64_t)blockIdx.x * a.E + e] = hist[e];
  }
}

constexpr int kMaxBlocks = 256;   // rows of hist: every sorting block reads them all

// How T tokens are routed.
struct RoutePlan { int lanes, v, threads, per, blocks; bool one; size_t lds; };
RoutePlan route_plan(int64_t T, int E, int k, int groups) {
  RoutePlan p;
  p.lanes = E <= 256 ? 16 : 64;
  p.v = 1;
  while (p.v * p.lanes < E) p.v *= 2;
  // few tokens or many: blocks of 16 waves, so that one block does it all, or
  // 256 of them fill the card; groups' keys leave LDS for 4
  p.threads = route_threads(p.lanes, p.v) == 1024 && groups == 1 && (T > 4096 || T <= 64) ? 1024 : 256;
  const int here = p.threads / p.lanes;
  p.one = T <= here;
  p.per = (int)(ceil_div(ceil_div(T, kMaxBlocks), here) * here);
  p.blocks = (int)ceil_div(T, std::max(p.per, 1));
  p.lds = (size_t)here * k * 12 + (groups > 1 ? (size_t)here * E * 8 : 0) + (size_t)E * 4;
  if (p.one) p.lds = std::max(p.lds, (size_t)E * (2 + p.threads / 64) * 4);
  return p;
}

template <bool SCORED, bool ONE> hipError_t launch_route(const RouteArgs& a, const RoutePlan& p, hipStream_t s) {
#define GQ_ROUTE(L, V) \
  if (p.lanes == L && p.v == V) route_kernel<L, V, SCORED, ONE><<<ONE ? 1 : p.blocks, p.threads, p.lds, s>>>(a)
  GQ_ROUTE(16, 1); GQ_ROUTE(16, 2); GQ_ROUTE(16, 4); GQ_ROUTE(16, 8); GQ_ROUTE(16, 16);
  GQ_ROUTE(64, 8); GQ_ROUTE(64, 16);
#undef GQ_ROUTE
  return hipGetLastError();
}
template <bool ONE> hipError_t launch_route(const RouteArgs& a, const RoutePlan& p, hipStream_t s) {
  const bool scored = a.bias || (a.groups > 1 && a.group_top == 2);
  return scored ? launch_route<true, ONE>(a, p, s) : launch_route<false, ONE>(a, p, s);
}

constexpr int kSortThreads = 512, kSortAlone = 4096;   // slots that one block sorts
size_t sort_lds(int E) { return (size_t)E * (2 + kSortThreads / 64) * 4; }

}  // namespace

// counts of the blocks; 256 where one block does all of it, whatever the groups
size_t moe_ws_bytes(int64_t T, int64_t E, int64_t k) {
  if (T <= 4 && T * k <= kSortAlone) return 256;
  return std::max<size_t>(512, align_up((size_t)std::min<int64_t>(kMaxBlocks, ceil_div(T * k, 4)) * E * 4));
}

hipError_t moe_plan_launch(const int32_t* ids, int64_t T, int k, int E, int32_t* offsets, int32_t* order,
                           void* ws, hipStream_t s) {
  const int slots = (int)(T * k);
  int32_t* hist = static_cast<int32_t*>(ws);
  if (slots <= kSortAlone) {
    sort_kernel<<<1, kSortThreads, sort_lds(E), s>>>(ids, slots, slots, E, nullptr, 1, offsets, order);
    return hipGetLastError();
  }
  const int per = (int)(ceil_div(ceil_div(slots, kMaxBlocks), 512) * 512), blocks = (int)ceil_div(slots, per);
  count_kernel<<<blocks, kSortThreads, (size_t)E * 4, s>>>(ids, per, slots, E, hist);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  sort_kernel<<<blocks, kSortThreads, sort_lds(E), s>>>(ids, per, slots, E, hist, blocks, offsets, order);
  return hipGetLastError();
}

hipError_t moe_route_launch(const void* X, int dt, int64_t T, int E, int64_t ld, const float* bias,
                            const uint8_t* mask, int scores, int k, int groups, int top_groups,
                            int group_top, int renorm, double scale, int32_t* ids, float* weights,
                            int32_t* offsets, int32_t* order, void* ws, hipStream_t s) {
  const RoutePlan p = route_plan(T, E, k, groups);
  RouteArgs a{X, dt, (int)T, E, ld, bias, mask, scores, k, groups, top_groups, group_top, renorm,
              scale, ids, weights, offsets, order, nullptr, p.per, p.blocks};
  if (offsets && p.one) return launch_route<true>(a, p, s);
  if (offsets) a.hist = static_cast<int32_t*>(ws);
  hipError_t e = launch_route<false>(a, p, s);
  if (e != hipSuccess || !offsets) return e;
  sort_kernel<<<p.blocks, kSortThreads, sort_lds(E), s>>>(ids, p.per * k, (int)(T * k), E, a.hist, p.blocks,
                                                         offsets, order);
  return hipGetLastError();
}

}  // namespace gq
