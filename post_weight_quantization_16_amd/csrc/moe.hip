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
#include "route_plan.hpp"

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
// A stable counting sort of slot numbers by expert.  A block's slots come
// behind those of the rows of counts before its own in hist, wave by wave;
// within 64 slots a lane finds the others of its expert by one ballot for each
// bit of the expert's number, and its rank among them by their count below it.
// Nothing depends on the order of atomics: those count, and nothing else.
// LDS: total [E], first [E], counts [waves][E].
__device__ __forceinline__ void sort_slots(const int32_t* ids, int i0, int i1, int E, int slots,
                                           const int32_t* hist, int rows, int row, int block, int blocks,
                                           int32_t* offsets, int32_t* order, int* lds) {
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
  if (hist) {   // all rows of counts, and those before this block's
    const int parts = max(1, nt / E);
    for (int e0 = 0; e0 < E; e0 += nt) {
      const int part = t / E, e = e0 + (E < nt ? t - part * E : t);
      if (part >= parts || e >= E) continue;
      int all = 0, before = 0;
      for (int q0 = part; q0 < rows; q0 += 16 * parts) {
        int h[16];   // sixteen loads in flight
#pragma unroll
        for (int i = 0; i < 16; ++i) h[i] = hist[(int64_t)min(q0 + i * parts, rows - 1) * E + e];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int q = q0 + i * parts;
          all += q < rows ? h[i] : 0;
          before += q < row ? h[i] : 0;
        }
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

// Sixteen waves where many rows of counts are to be read (us, 256 rows of 128
// experts: 10.1 with eight, 8.4 with sixteen; 84 rows of 256: 6.4, 7.3) and LDS
// has room for each wave's own.
int sort_threads(int E, int rows) { return rows > 128 && E <= 512 ? 1024 : 512; }
// One block for `group` rows of counts, of `per` slots each.
__global__ __launch_bounds__(1024) void sort_kernel(const int32_t* ids, int per, int slots, int E,
                                                    const int32_t* hist, int rows, int group,
                                                    int32_t* offsets, int32_t* order) {
  extern __shared__ int lds[];
  const int row = blockIdx.x * group;
  const int i0 = (int)min((int64_t)row * per, (int64_t)slots), i1 = (int)min(i0 + (int64_t)group * per, (int64_t)slots);
  sort_slots(ids, i0, i1, E, slots, hist, rows, row, blockIdx.x, gridDim.x, offsets, order, lds);
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
// The two values that lanes N apart hold (N = 16, 32), in both of them.
template <int N> __device__ __forceinline__ void both(uint32_t v, uint32_t& a, uint32_t& b) {
  const auto r = N == 16 ? __builtin_amdgcn_permlane16_swap(v, v, false, false)
                         : __builtin_amdgcn_permlane32_swap(v, v, false, false);
  a = r[0];
  b = r[1];
}
template <int N> __device__ __forceinline__ void both(float v, float& a, float& b) {
  uint32_t x, y;
  both<N>(__builtin_bit_cast(uint32_t, v), x, y);
  a = __builtin_bit_cast(float, x);
  b = __builtin_bit_cast(float, y);
}
template <int N> __device__ __forceinline__ void both(double v, double& a, double& b) {
  const uint64_t q = __builtin_bit_cast(uint64_t, v);
  uint32_t x, y, z, w;
  both<N>((uint32_t)q, x, y);
  both<N>((uint32_t)(q >> 32), z, w);
  a = __builtin_bit_cast(double, (uint64_t)z << 32 | x);
  b = __builtin_bit_cast(double, (uint64_t)w << 32 | y);
}
// Maximum and sum over the L lanes of a token (every lane gets them).
template <int L, typename T> __device__ __forceinline__ T lanes_max(T v) {
  v = larger(v, turned<kRor8>(v));
  v = larger(v, turned<kRor4>(v));
  v = larger(v, turned<kRor2>(v));
  v = larger(v, turned<kRor1>(v));
  if constexpr (L == 64) {
    T a, b;
    both<16>(v, a, b);
    v = larger(a, b);
    both<32>(v, a, b);
    v = larger(a, b);
  }
  return v;
}
template <int L> __device__ __forceinline__ double lanes_sum(double v) {
  v += turned<kRor8>(v);
  v += turned<kRor4>(v);
  v += turned<kRor2>(v);
  v += turned<kRor1>(v);
  if constexpr (L == 64) {
    double a, b;
    both<16>(v, a, b);
    v = a + b;
    both<32>(v, a, b);
    v = a + b;
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

// V neighbouring logits from `at` on, those past n (0 or less: none) -inf.
template <int DT, int V> __device__ __forceinline__ void logits_of(const void* X, int64_t at, int n, float (&x)[V]) {
  typedef typename Elem<DT>::type T;
  const T* p = static_cast<const T*>(X) + at;
  if (n >= V) {
    T v[V];
    __builtin_memcpy(v, p, sizeof v);
#pragma unroll
    for (int j = 0; j < V; ++j) x[j] = Elem<DT>::up(v[j]);
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) x[j] = j < n ? Elem<DT>::up(p[j]) : -__builtin_inff();
  }
}

// L lanes a token, V neighbouring experts a lane, so that the lowest lane with
// the largest key holds the lowest expert with it.  64 lanes a token where few
// tokens wait for the chain of one (333 tokens over 256 experts in groups: 22.4
// us with 16 lanes, 10.0 with 64) or 16 lanes would hold more than 16 experts each;
// 16 where the card is full, four tokens a wave (16384 over 128: 11.6 and 23.4).
// SCORED: the choice needs p (a bias, or groups by their best two); otherwise
// the keys are the logits, in fp32, which holds them exactly.
// ONE: one block routes all tokens and sorts their slots too.
template <int L, int V, bool SCORED, bool ONE>
__global__ __launch_bounds__(route_threads(L, V)) void route_kernel(RouteArgs a) {
  typedef typename KeyOf<SCORED>::type Key;
  extern __shared__ double smem[];
  const int t = threadIdx.x, lane = t & 63, l = lane & (L - 1);
  const int here = blockDim.x / L, mine = t / L;   // tokens at a time, this thread's
  double* P = smem + mine * a.k;                                   // [here][k]: what was chosen
  double* rest = smem + here * a.k;
  Key* K = reinterpret_cast<Key*>(rest) + mine * a.E;              // [here][E], groups only
  Key* B = reinterpret_cast<Key*>(rest + here * a.E) + 2 * t;      // [here][L][2], groups only
  if (a.groups > 1) rest += here * (a.E + 2 * L);
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
    const int n = on ? a.E - l * V : 0;
    const int64_t at = tok * a.ld + l * V;
    if (a.dt == GPTQ_F32) logits_of<GPTQ_F32>(a.X, at, n, x);
    else if (a.dt == GPTQ_BF16) logits_of<GPTQ_BF16>(a.X, at, n, x);
    else logits_of<GPTQ_F16>(a.X, at, n, x);
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
      // each group's best two by L / groups lanes, then by its own
      const int parts = L / a.groups, g = l / parts, q = l - g * parts;
      Key one = none, two = none;
      if (g < a.groups)
        for (int i = q; i < size; i += parts) {
          const Key v = K[g * size + i];
          two = larger(two, v < one ? v : one);
          one = larger(one, v);
        }
      B[0] = one;
      B[1] = two;
      wave_sync();
      one = none;
      two = none;
      if (l < a.groups) {
        const Key* P2 = reinterpret_cast<Key*>(smem + here * (a.k + a.E)) + 2 * (t - l + l * parts);
        for (int i = 0; i < 2 * parts; ++i) {
          const Key v = P2[i];
          two = larger(two, v < one ? v : one);
          one = larger(one, v);
        }
      }
      Key score = a.group_top == 2 && two > none ? one + two : one;
      uint32_t kept = 0;
      for (int r = 0; r < a.top_groups; ++r) {
        const Key best = lanes_max<L>(score);
        const int first = lanes_first<L>(best > none && score == best, lane);
        if (first < L) kept |= 1u << first;
        if (l == first) score = none;
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
      if constexpr (ONE) I[r] = live ? id : -1;
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
    const int slots = a.T * a.k;
    if (slots <= 64) {   // all of them in a wave
      const int* ids = I - mine * a.k;
      for (int e = t; e <= a.E; e += blockDim.x) {
        int n = 0;
        for (int i = 0; i < slots; ++i) n += (unsigned)ids[i] < (unsigned)e;
        a.offsets[e] = n;
      }
      if (t < slots) {
        const unsigned id = (unsigned)ids[t];   // none: the largest
        int n = 0;
        for (int i = 0; i < slots; ++i) n += (unsigned)ids[i] < id || ((unsigned)ids[i] == id && i < t);
        a.order[n] = (int)id < 0 ? -1 : t;
      }
      return;
    }
    sort_slots(a.ids, 0, a.T * a.k, a.E, a.T * a.k, nullptr, 1, 0, 0, 1, a.offsets, a.order, reinterpret_cast<int*>(smem));
  } else if (count) {
    __syncthreads();
    for (int e = t; e < a.E; e += blockDim.x) a.hist[(int64_t)blockIdx.x * a.E + e] = hist[e];
  }
}

template <bool SCORED, bool ONE> hipError_t launch_route(const RouteArgs& a, const RoutePlan& p, hipStream_t s) {
#define GQ_ROUTE(L, V) \
  if (p.lanes == L && p.v == V) route_kernel<L, V, SCORED, ONE><<<ONE ? 1 : p.blocks, p.threads, p.lds, s>>>(a)
  GQ_ROUTE(16, 1); else GQ_ROUTE(16, 2); else GQ_ROUTE(16, 4); else GQ_ROUTE(16, 8);
  else GQ_ROUTE(64, 1); else GQ_ROUTE(64, 2); else GQ_ROUTE(64, 4); else GQ_ROUTE(64, 8); else GQ_ROUTE(64, 16);
  else return hipErrorInvalidValue;
#undef GQ_ROUTE
  return hipGetLastError();
}
template <bool ONE> hipError_t launch_route(const RouteArgs& a, const RoutePlan& p, hipStream_t s) {
  const bool scored = a.bias || (a.groups > 1 && a.group_top == 2);
  return scored ? launch_route<true, ONE>(a, p, s) : launch_route<false, ONE>(a, p, s);
}

constexpr int kSortAlone = 4096;   // slots that one block sorts
// Each block reads all rows of counts, 256 at most: a quarter as many blocks
// (16384 tokens, top 8 of 128: 13.3 us with one for each row, 8.4 with one for four).
constexpr int kRowsEach = 4;
hipError_t launch_sort(const int32_t* ids, int per, int slots, int E, const int32_t* hist, int rows,
                       int32_t* offsets, int32_t* order, hipStream_t s) {
  const int threads = sort_threads(E, rows);
  const size_t lds = (size_t)E * (2 + threads / 64) * 4;
  sort_kernel<<<(unsigned)ceil_div(rows, kRowsEach), threads, lds, s>>>(ids, per, slots, E, hist, rows, kRowsEach,
                                                                        offsets, order);
  return hipGetLastError();
}

}  // namespace

// counts of the blocks; 256 where one block does all of it, whatever the groups
size_t moe_ws_bytes(int64_t T, int64_t E, int64_t k) {
  if (T <= (E <= 256 ? 16 : 4)) return 256;
  return std::max<size_t>(512, align_up((size_t)std::min<int64_t>(kMaxBlocks, ceil_div(T * k, 4)) * E * 4));
}

hipError_t moe_plan_launch(const int32_t* ids, int64_t T, int k, int E, int32_t* offsets, int32_t* order,
                           void* ws, hipStream_t s) {
  const int slots = (int)(T * k);
  int32_t* hist = static_cast<int32_t*>(ws);
  if (slots <= kSortAlone) {
    return launch_sort(ids, slots, slots, E, nullptr, 1, offsets, order, s);
  }
  const int per = (int)(ceil_div(ceil_div(slots, kMaxBlocks), 512) * 512), blocks = (int)ceil_div(slots, per);
  count_kernel<<<blocks, 512, (size_t)E * 4, s>>>(ids, per, slots, E, hist);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  return launch_sort(ids, per, slots, E, hist, blocks, offsets, order, s);
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
  return launch_sort(ids, p.per * k, (int)(T * k), E, a.hist, p.blocks, offsets, order, s);
}

}  // namespace gq
