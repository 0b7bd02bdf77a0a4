// The router: each token's experts, and the choices sorted by expert.
//   s = sigmoid(l) or softmax(l) over the token's experts, v = s + bias; of num_groups runs of experts the top_groups with
//   the largest sum of their best two v; the top_k largest v there, ties to the lowest index.
// The choice is the one that 64 bits make.  Without bias and runs it is that of the logits, which are compared as they
// are.  Otherwise v is computed in FP32 first; where two neighbours among the ordered first top_k + 1 values (or the run
// values at the cut) lie closer than FP32's error, the token is done again in FP64, which this GPU has little of: some
// tokens in a hundred.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cfloat>
#include <cstdint>

#include "common.cuh"
#include "ptx.cuh"

namespace dsa {

constexpr int kRouteMaxExperts = 512;
constexpr int kRouteMaxTop = 16;
constexpr int kRouteMaxRuns = 32;
constexpr int kRouteThreads = 256;  // a warp to a token

struct RouteParams {
  const void* logits;
  const float* bias;           // [E], or null
  const int32_t* num_tokens;   // or null
  int32_t* ids;                // [T, top_k]
  float* weights;              // [T, top_k]
  int32_t* starts;             // [E + 1]
  int32_t* rows;               // [T * top_k]
  int32_t* places;             // [T, top_k]
  int64_t stride;
  int T, E, top_k, num_groups, top_groups, per;
  float scale;
  bool softmax, normalize;
};

template <typename T>
__device__ __forceinline__ float load_logit(const void* p, int64_t at) {
  const T x = static_cast<const T*>(p)[at];
  const float l = static_cast<float>(x);
  return l != l ? -INFINITY : fminf(l, FLT_MAX) + 0.0f;  // (-0 becomes 0, as which it compares)
}

// Order-preserving keys, 0 below all of them (it stands for what is not to be chosen).
__device__ __forceinline__ uint32_t order_key(float v) { return v != v ? 1u : score_key(v + 0.0f); }
__device__ __forceinline__ uint64_t order_key(double v) {
  if (v != v) return 1;
  const uint64_t u = __double_as_longlong(v + 0.0);
  return (u >> 63) ? ~u : (u | (1ull << 63));
}
__device__ __forceinline__ uint32_t warp_max(uint32_t k) { return __reduce_max_sync(0xffffffffu, k); }
__device__ __forceinline__ uint64_t warp_max(uint64_t k) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const uint64_t other = __shfl_xor_sync(0xffffffffu, k, o);
    if (other > k) k = other;
  }
  return k;
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? k ^ 0x80000000u : ~k);
}
__device__ __forceinline__ double key_value(uint64_t k) {
  return __longlong_as_double((k >> 63) ? k ^ (1ull << 63) : ~k);
}
template <typename F>
struct KeyOf;
template <>
struct KeyOf<float> { using type = uint32_t; };
template <>
struct KeyOf<double> { using type = uint64_t; };

__device__ __forceinline__ float exp_of(float x) { return expf(x); }
__device__ __forceinline__ double exp_of(double x) { return exp(x); }

// The largest of the warp's keys and its element (the lowest where several have it).
template <int V, typename K>
__device__ __forceinline__ K warp_best(const K (&key)[V], int lane, int* element) {
  K mine = key[0];
  int at = lane;
#pragma unroll
  for (int i = 1; i < V; ++i)
    if (key[i] > mine) mine = key[i], at = i * 32 + lane;
  const K best = warp_max(mine);
  *element = (int)__reduce_min_sync(0xffffffffu, mine == best ? (uint32_t)at : 0xffffffffu);
  return best;
}
template <int V, typename K>
__device__ __forceinline__ void drop(K (&key)[V], int lane, int element) {
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (element == i * 32 + lane) key[i] = 0;
}

// The choice of one token in F; lane j gets the j-th expert.  False where F cannot tell (FP32 only).
template <int V, typename F>
__device__ __forceinline__ bool choose(const RouteParams& p, const float (&l)[V], int lane, int* chosen) {
  using K = typename KeyOf<F>::type;
  K key[V];
  // The error of two values' difference in FP32 is below `close` times the larger of `size` and both.  A sigmoid is off by
  // 2^-22 at most (exponential 1 ulp, sum and quotient half of one).  A softmax probability is by 2^-19.3 of itself (its sum
  // has 16 + 5 roundings), so `size` is the largest of them.  The bias adds 2^-24 of v.
  const F close = p.softmax ? (F)0x1p-18 : (F)0x1p-20;
  F size = 1;
  if (p.softmax) {
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < V; ++i) top = fmaxf(top, l[i]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    F s[V], sum = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      s[i] = l[i] == -INFINITY ? (F)0 : exp_of((F)l[i] - (F)top);
      sum += s[i];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = i * 32 + lane;
      key[i] = e < p.E ? order_key((sum > 0 ? s[i] / sum : (F)0) + (p.bias ? (F)p.bias[e] : (F)0)) : 0;
    }
    size = 1 / sum;
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = i * 32 + lane;
      key[i] = e < p.E ? order_key((F)1 / ((F)1 + exp_of(-(F)l[i])) + (p.bias ? (F)p.bias[e] : (F)0)) : 0;
    }
  }
  bool sure = true;
  auto apart = [&](F high, F low, F bound) {
    return high - low > bound * fmax(size, fmax(fabs(high), fabs(low)));
  };
  if (p.num_groups > 1) {
    // lane g has run g's value
    F value = 0;
    for (int g = 0; g < p.num_groups; ++g) {
      K in[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int e = i * 32 + lane;
        in[i] = e >= g * p.per && e < (g + 1) * p.per ? key[i] : 0;
      }
      int at;
      F sum = key_value(warp_best<V>(in, lane, &at));
      if (p.per > 1) {
        drop<V>(in, lane, at);
        sum += key_value(warp_best<V>(in, lane, &at));
      }
      if (lane == g) value = sum;
    }
    K runs[1] = {lane < p.num_groups ? order_key(value) : (K)0};
    uint32_t kept = 0;
    K last = 0;
    for (int i = 0; i < p.top_groups; ++i) {
      int g;
      last = warp_best<1>(runs, lane, &g);
      drop<1>(runs, lane, g);
      kept |= 1u << g;
    }
    int g;
    const K next = warp_best<1>(runs, lane, &g);
    if (sizeof(F) == 4 && p.top_groups < p.num_groups) sure = apart(key_value(last), key_value(next), 4 * close);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = i * 32 + lane;
      if (e < p.E && !((kept >> (e / p.per)) & 1)) key[i] = 0;
    }
  }
  F before = 0;
  for (int j = 0; j <= p.top_k; ++j) {
    if (j == p.top_k && sizeof(F) == 8) break;
    int e;
    const K best = warp_best<V>(key, lane, &e);
    if (best == 0) break;  // (no value is left beyond the last one)
    const F v = key_value(best);
    if (sizeof(F) == 4 && j > 0) sure = sure && apart(before, v, close);
    before = v;
    if (j < p.top_k && lane == j) *chosen = e;
    drop<V>(key, lane, e);
  }
  return sure;
}

// Scores of the chosen, an expert to a lane, from its logit and the row's softmax statistics.
template <int V, typename T>
__global__ void __launch_bounds__(kRouteThreads) route_choose_kernel(const __grid_constant__ RouteParams p) {
  const int lane = threadIdx.x & 31;
  const int t = (int)((blockIdx.x * (unsigned)kRouteThreads + threadIdx.x) >> 5);
  if (t >= p.T) return;
  const int64_t out = (int64_t)t * p.top_k + lane;
  if (p.num_tokens && t >= *p.num_tokens) {
    if (lane < p.top_k) {
      p.ids[out] = -1;
      p.weights[out] = 0.f;
      p.places[out] = -1;
    }
    return;
  }
  float l[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = i * 32 + lane;
    l[i] = e < p.E ? load_logit<T>(p.logits, (int64_t)t * p.stride + e) : -INFINITY;
  }
  int chosen = 0;
  if (!p.bias && p.num_groups == 1) {
    uint32_t key[V];
#pragma unroll
    for (int i = 0; i < V; ++i) key[i] = i * 32 + lane < p.E ? order_key(l[i]) : 0;
    for (int j = 0; j < p.top_k; ++j) {
      int e;
      warp_best<V>(key, lane, &e);
      if (lane == j) chosen = e;
      drop<V>(key, lane, e);
    }
  } else if (!choose<V, float>(p, l, lane, &chosen)) {
    choose<V, double>(p, l, lane, &chosen);
  }
  // weights: in FP32, but for rows all of whose scores are next to nothing
  const bool mine = lane < p.top_k;
  const float lc = load_logit<T>(p.logits, (int64_t)t * p.stride + chosen);
  float top = 0.f, sum = 1.f, score;
  if (p.softmax) {
    top = -INFINITY;
#pragma unroll
    for (int i = 0; i < V; ++i) top = fmaxf(top, l[i]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) sum += l[i] == -INFINITY ? 0.f : expf(l[i] - top);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    score = lc == -INFINITY ? 0.f : expf(lc - top) / sum;
  } else {
    score = 1.f / (1.f + expf(-lc));
  }
  if (!mine) score = 0.f;
  if (p.normalize) {
    float all = score;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
    if (all < 1e-30f) {
      double d = 0;
      if (mine && lc != -INFINITY) d = p.softmax ? exp((double)lc - (double)top) : 1.0 / (1.0 + exp(-(double)lc));
      double each = d;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) each += __shfl_xor_sync(0xffffffffu, each, o);
      score = each > 0 ? (float)(d / each) : 0.f;
    } else {
      score /= all;
    }
  }
  if (mine) {
    p.ids[out] = chosen;
    p.weights[out] = score * p.scale;
  }
}

// The stable counting sort of the choices by expert, in one CTA: each warp counts a run of them, every expert's counts are
// summed over the warps and the experts, and each warp goes over its run again.
constexpr int kPlaceThreads = 1024;
__global__ void __launch_bounds__(kPlaceThreads) route_place_kernel(const __grid_constant__ RouteParams p) {
  extern __shared__ int counts[];  // [32][E], then [E]
  constexpr int kWarps = kPlaceThreads / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int* const mine = counts + warp * p.E;
  int* const base = counts + kWarps * p.E;
  for (int i = lane; i < p.E; i += 32) mine[i] = 0;
  __syncwarp();
  const int64_t n = (int64_t)p.T * p.top_k;
  const int64_t run = (n + kWarps * 32 - 1) / (kWarps * 32) * 32;
  const int64_t first = warp * run, last = min(n, first + run);
  for (int64_t i = first + lane; i - lane < last; i += 32) {
    const int e = i < last ? p.ids[i] : -1;
    const uint32_t same = __match_any_sync(0xffffffffu, e);
    if (e >= 0 && lane == __ffs(same) - 1) mine[e] += __popc(same);
    __syncwarp();
  }
  __syncthreads();
  for (int e = tid; e < p.E; e += kPlaceThreads) {
    int sum = 0;
    for (int w = 0; w < kWarps; ++w) {
      const int c = counts[w * p.E + e];
      counts[w * p.E + e] = sum;
      sum += c;
    }
    base[e] = sum;
  }
  __syncthreads();
  if (warp == 0) {
    int sum = 0;
    for (int at = 0; at < p.E; at += 32) {
      const int c = at + lane < p.E ? base[at + lane] : 0;
      int up = c;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, up, o);
        if (lane >= o) up += v;
      }
      if (at + lane < p.E) {
        base[at + lane] = sum + up - c;
        p.starts[at + lane] = sum + up - c;
      }
      sum += __shfl_sync(0xffffffffu, up, 31);
    }
    if (lane == 0) p.starts[p.E] = sum;
  }
  __syncthreads();
  for (int64_t i = first + lane; i - lane < last; i += 32) {
    const int e = i < last ? p.ids[i] : -1;
    const uint32_t same = __match_any_sync(0xffffffffu, e);
    if (e >= 0) {
      const int place = base[e] + mine[e] + __popc(same & ((1u << lane) - 1));
      p.places[i] = place;
      p.rows[place] = (int32_t)(i / p.top_k);
    }
    __syncwarp();
    if (e >= 0 && lane == __ffs(same) - 1) mine[e] += __popc(same);
    __syncwarp();
  }
}

}  // namespace dsa
