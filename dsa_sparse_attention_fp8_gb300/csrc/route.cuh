// The router: each token's experts, and the choices sorted by expert.
//   s = sigmoid(l) or softmax(l) over the token's experts, v = s + bias; of num_groups runs of experts the top_groups with
//   the largest sum of their best two v; the top_k largest v there, ties to the lowest index.
// The choice is the one that 64 bits make.  Without bias and runs it is that of the logits, which are compared as they
// are.  Otherwise v is computed in FP32 first; where two neighbours among the ordered first top_k + 1 values (or the run
// values at the cut) lie closer than FP32's error, what is close is done again in FP64, which this GPU has little of.
// Bound by instructions: a token of 256 experts, 8 runs and 8 choices takes a warp some 1080 (a first form, which searched
// every run with a whole warp and all keys for each choice, 2550).  8192 tokens: 23 us, the choice 15 and the places 8 (one
// CTA, matching choices across a warp, 131); 64 tokens, in one launch, 5.8.
// How many tokens are done again hangs on the values, since the error that is allowed for is that of a score of 1 (of a softmax,
// of its largest): of sigmoids of logits of deviation 1.5 around 0 one in a thousand, but most of those that crowd near 0 or 1
// and have no bias to tell them apart.  8192 such tokens without a bias: around -10 26 us, -12 31, 8 49, 14 115 (then all their
// values are done again), of deviation 6 around 0 41; softmax of deviation 1.5 34, 8 79, 12 138.  With a bias of deviation
// 0.05 17 to 25, softmax 35.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cfloat>
#include <cstdint>

#include "common.cuh"
#include "ptx_matmul.cuh"

namespace dsa {

constexpr int kRouteMaxExperts = 512;
constexpr int kRouteMaxTop = 16;
constexpr int kRouteMaxRuns = 32;
constexpr int kRouteThreads = 256;  // a warp to a token
constexpr int kFewThreads = 512, kPlaceThreads = 1024;
constexpr int kFewCtas = 8, kPlaceCtas = 16;  // of a cluster, at most

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
  int T, E, top_k, num_groups, top_groups;
  int per, lanes, wide;        // experts of a run, lanes that share a run, experts of a lane
  float scale;
  bool softmax, normalize;
};

template <typename T>
__device__ __forceinline__ float load_logit(const void* p, int64_t at) {
  const T x = static_cast<const T*>(p)[at];
  const float l = static_cast<float>(x);
  return l != l ? -INFINITY : fminf(l, FLT_MAX) + 0.0f;  // (-0 becomes 0, as which it compares)
}

// Order-preserving keys, 0 below all of them (it stands for what is not to be chosen).  NaN counts as -inf; there is no -0.
__device__ __forceinline__ uint32_t order_key(float v) { return score_key(fmaxf(v, -INFINITY)); }
__device__ __forceinline__ uint64_t order_key(double v) {
  const uint64_t u = __double_as_longlong(v == v ? v : -INFINITY);
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
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return max(a, b); }
__device__ __forceinline__ uint64_t larger(uint64_t a, uint64_t b) { return a > b ? a : b; }
__device__ __forceinline__ uint32_t smaller(uint32_t a, uint32_t b) { return min(a, b); }
__device__ __forceinline__ uint64_t smaller(uint64_t a, uint64_t b) { return a < b ? a : b; }
__device__ __forceinline__ float exp_of(float x) { return expf(x); }
__device__ __forceinline__ double exp_of(double x) { return exp(x); }

// Where a lane's experts lie: `lanes` lanes share a run (a power of two; all 32 the one run of an ungrouped choice), each
// has `wide` <= V neighbours.  So the order of lanes, and of a lane's own, is that of the experts, and a run's best are found
// among few lanes.
struct Own {
  int first, count;
  // the place of the i-th, of expert 0 where there is none (loads without branches)
  __device__ __forceinline__ int at(int i) const { return i < count ? first + i : 0; }
};
__device__ __forceinline__ Own own_experts(const RouteParams& p, int lane) {
  const int run = lane / p.lanes, sub = lane - run * p.lanes;
  const int count = run < p.num_groups ? min(p.wide, p.per - sub * p.wide) : 0;
  return {run * p.per + sub * p.wide, max(0, count)};
}

// A lane's largest key and its place.
template <int V, typename K>
__device__ __forceinline__ K lane_best(const K (&key)[V], int* at) {
  K best = key[0];
  *at = 0;
#pragma unroll
  for (int i = 1; i < V; ++i) {
    *at = key[i] > best ? i : *at;
    best = larger(best, key[i]);
  }
  return best;
}

// The first `n` keys of the warp in order, each taken out: take(j, key, expert) for each of them, the expert as the lane that
// had it knows it; stops early where no key is left.
template <int V, typename K, typename Take>
__device__ __forceinline__ void in_order(K (&key)[V], int first, int n, int lane, Take take) {
  int at;
  K mine = lane_best<V>(key, &at);
  for (int j = 0; j < n; ++j) {
    const K best = warp_max(mine);
    if (best == 0) return;
    const int who = __ffs(__ballot_sync(0xffffffffu, mine == best)) - 1;  // (ties: the lowest lane, and there the first)
    take(j, best, __shfl_sync(0xffffffffu, first + at, who));
    const int gone = lane == who ? at : -1;
#pragma unroll
    for (int i = 0; i < V; ++i) key[i] = i == gone ? 0 : key[i];
    mine = lane_best<V>(key, &at);
  }
}

// The first `n` keys of the warp in order: lane j gets the j-th and its expert, lanes from the number returned on nothing.
// The n-th of the lanes' own largest is no more than the n-th of all, so whatever is not below it (seldom many more than n)
// goes to a lane each, and every lane counts what comes before its own; rounds of taking the largest out, with a lane's keys
// searched again each time, take twice the instructions.
template <int V>
__device__ __forceinline__ int first_in_order(const uint32_t (&key)[V], int first, int n, int lane, uint2* list, uint32_t* its, int* expert) {
  uint32_t rest = key[0], least = 1;
#pragma unroll
  for (int i = 1; i < V; ++i) rest = max(rest, key[i]);
  for (int j = 0; j < n; ++j) {
    const uint32_t best = warp_max(rest);
    least = max(best, 1u);
    rest = rest == best ? 0 : rest;
  }
  int total = 0;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const bool want = key[i] >= least;
    const uint32_t who = __ballot_sync(0xffffffffu, want);
    const int at = total + __popc(who & ((1u << lane) - 1));
    if (want && at < 32) list[at] = make_uint2(key[i], first + i);
    total += __popc(who);
  }
  __syncwarp();
  if (total > 32) {
    uint32_t left[V];
#pragma unroll
    for (int i = 0; i < V; ++i) left[i] = key[i];
    int found = 0;
    in_order<V>(left, first, n, lane, [&](int j, uint32_t best, int e) {
      if (lane == j) *its = best, *expert = e;
      found = j + 1;
    });
    __syncwarp();
    return found;
  }
  const uint2 mine = lane < total ? list[lane] : make_uint2(0, 0);
  __syncwarp();
  int rank = 0;
  for (int j = 0; j < total; ++j) {
    const uint32_t k = __shfl_sync(0xffffffffu, mine.x, j), e = __shfl_sync(0xffffffffu, mine.y, j);
    rank += k > mine.x || (k == mine.x && e < mine.y);
  }
  if (lane < total) list[rank] = mine;
  __syncwarp();
  *its = list[lane].x;
  *expert = (int)list[lane].y;
  __syncwarp();
  return min(total, n);
}

// The values v of a lane's experts in F, as keys, and the largest score there can be.
template <int V, typename F, typename K>
__device__ __forceinline__ F value_keys(const RouteParams& p, const float (&l)[V], const Own& own, K (&key)[V]) {
  F s[V], inv = 1;
  if (p.softmax) {
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < V; ++i) top = fmaxf(top, l[i]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    F sum = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      s[i] = l[i] == -INFINITY ? (F)0 : exp_of((F)l[i] - (F)top);
      sum += s[i];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (sum > 0) inv = 1 / sum;
#pragma unroll
    for (int i = 0; i < V; ++i) s[i] = sizeof(F) == 4 ? s[i] * inv : sum > 0 ? s[i] / sum : (F)0;
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) s[i] = sizeof(F) == 4 ? (F)rcp_approx(1.0f + __expf(-l[i])) : (F)1 / ((F)1 + exp_of(-(F)l[i]));
  }
  if (p.bias) {
#pragma unroll
    for (int i = 0; i < V; ++i) s[i] += (F)p.bias[own.at(i)];
  }
#pragma unroll
  for (int i = 0; i < V; ++i) key[i] = i < own.count ? order_key(s[i]) : 0;
  return inv;
}

// The run's best two keys, in all of its lanes.
template <int V, typename K>
__device__ __forceinline__ void best_two(const RouteParams& p, const K (&key)[V], K* best, K* second) {
  K b = 0, s = 0;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    s = larger(s, smaller(b, key[i]));
    b = larger(b, key[i]);
  }
  for (int o = 1; o < p.lanes; o <<= 1) {
    const K b2 = __shfl_xor_sync(0xffffffffu, b, o), s2 = __shfl_xor_sync(0xffffffffu, s, o);
    s = larger(larger(s, s2), smaller(b, b2));
    b = larger(b, b2);
  }
  *best = b;
  *second = s;
}

// How many runs come before this lane's, by their values' keys.
template <typename K>
__device__ __forceinline__ int runs_ahead(const RouteParams& p, K mine, int run) {
  int ahead = 0;
  for (int g = 0; g < p.num_groups; ++g) {
    const K other = __shfl_sync(0xffffffffu, mine, g * p.lanes);
    ahead += other > mine || (other == mine && g < run);
  }
  return ahead;
}

template <int V, typename T>
__device__ __forceinline__ void load_logits(const RouteParams& p, int64_t row, const Own& own, float (&l)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) l[i] = load_logit<T>(p.logits, row + own.at(i));
#pragma unroll
  for (int i = 0; i < V; ++i) l[i] = i < own.count ? l[i] : -INFINITY;
}

// The choice of one token with all values in 64 bits; lane j gets the j-th expert.
template <int V, typename T>
__device__ __noinline__ int choose64(const RouteParams& p, int64_t row, int lane) {
  const Own own = own_experts(p, lane);
  float l[V];
  load_logits<V, T>(p, row, own, l);
  uint64_t key[V];
  value_keys<V, double>(p, l, own, key);
  if (p.num_groups > 1) {
    uint64_t best, second;
    best_two<V>(p, key, &best, &second);
    const int run = lane / p.lanes;
    const double value = key_value(best) + (p.per > 1 ? key_value(second) : 0.0);
    if (runs_ahead(p, run < p.num_groups ? order_key(value) : (uint64_t)0, run) >= p.top_groups) {
#pragma unroll
      for (int i = 0; i < V; ++i) key[i] = 0;
    }
  }
  int chosen = 0;
  in_order<V>(key, own.first, p.top_k, lane, [&](int j, uint64_t, int e) {
    if (lane == j) chosen = e;
  });
  return chosen;
}

// Experts whose key is `least` or more, one to a lane (-1 past them); how many there are.
template <int V>
__device__ __forceinline__ int candidates(const uint32_t (&key)[V], uint32_t least, int first, int lane, int* list, int* mine) {
  int total = 0;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const bool want = key[i] != 0 && key[i] >= least;
    const uint32_t who = __ballot_sync(0xffffffffu, want);
    const int at = total + __popc(who & ((1u << lane) - 1));
    if (want && at < 32) list[at] = first + i;
    total += __popc(who);
  }
  __syncwarp();
  *mine = lane < total ? list[lane] : -1;
  __syncwarp();
  return total;
}
// A candidate's value in 64 bits (of sigmoids), 0 of none.
template <typename T>
__device__ __forceinline__ uint64_t value64(const RouteParams& p, int64_t row, int e) {
  if (e < 0) return 0;
  const double s = 1.0 / (1.0 + exp(-(double)load_logit<T>(p.logits, row + e)));
  return order_key(s + (p.bias ? (double)p.bias[e] : 0.0));
}

// The choice of one token; lane j gets the j-th expert.  Values in FP32, whose difference is off by less than `close` times
// the larger of `size` and both: a sigmoid by 2^-21.9 at most (the exponential's 2 + 1.17 |l| ulp count s (1 - s) times, below
// 0.63 of 2^-23; sum 2^-24, reciprocal 2^-23), a softmax probability by 2^-19 of itself (its sum has 32 + 5 roundings), so `size`
// is the largest of them; the bias adds 2^-24 of v.  What lies closer is done again in 64 bits: of sigmoids the candidates alone, one to a lane, otherwise all.
// (A value takes some 30 instructions of the 64-bit unit, 64 cycles each, and a call waits for its last token: with all
// values again, 8192 tokens took 28 us, of which 14 were for ten of them.)
template <int V, typename T>
__device__ __forceinline__ int choose(const RouteParams& p, const float (&l)[V], const Own& own, int64_t row, int lane, int* list) {
  const float close = p.softmax ? 0x1p-17f : 0x1p-20f;
  uint32_t key[V];
  const float size = value_keys<V, float>(p, l, own, key);
  const auto bound = [&](float a, float b) { return close * fmaxf(size, fmaxf(fabsf(a), fabsf(b))); };
  if (p.num_groups > 1) {
    const int run = lane / p.lanes;
    const bool is = run < p.num_groups;
    uint32_t best, second;
    best_two<V>(p, key, &best, &second);
    const float value = key_value(best) + (p.per > 1 ? key_value(second) : 0.0f);
    const uint32_t mine = is ? order_key(value) : 0;
    int ahead = runs_ahead(p, mine, run);
    if (p.top_groups < p.num_groups) {
      const bool kept = ahead < p.top_groups;
      // a run's value is off by what its two are off by, however small their sum: the least of the kept runs' and the largest of
      // the others' as they may be
      const float off = 2 * bound(key_value(best), key_value(second));
      const float least = key_value(~warp_max(is && kept ? ~order_key(value - off) : 0u));
      const float next = key_value(warp_max(is && !kept ? order_key(value + off) : 0u));
      if (!(least > next)) {
        const float low = p.per > 1 ? key_value(second) : key_value(best);
        int e;
        const int n = candidates<V>(key, is ? order_key(low - 2 * bound(low, low)) : ~0u, own.first, lane, list, &e);
        if (p.softmax || n > 32) return choose64<V, T>(p, row, lane);
        const uint64_t v = value64<T>(p, row, e);
        const int its = e < 0 ? -1 : e / p.per;
        uint64_t exactly = 0;
        for (int g = 0; g < p.num_groups; ++g) {
          const uint64_t one = warp_max(its == g ? v : (uint64_t)0);
          const int owner = __ffs(__ballot_sync(0xffffffffu, its == g && v == one)) - 1;
          const uint64_t two = warp_max(its == g && lane != owner ? v : (uint64_t)0);
          if (run == g) exactly = order_key(key_value(one) + (p.per > 1 ? key_value(two) : 0.0));
        }
        ahead = runs_ahead(p, exactly, run);
      }
    }
    if (ahead >= p.top_groups) {
#pragma unroll
      for (int i = 0; i < V; ++i) key[i] = 0;
    }
  }
  uint32_t its;
  int chosen;
  const int found = first_in_order<V>(key, own.first, p.top_k + 1, lane, reinterpret_cast<uint2*>(list), &its, &chosen);
  const float mine = key_value(its), next = __shfl_down_sync(0xffffffffu, mine, 1);
  const bool sure = __all_sync(0xffffffffu, lane >= p.top_k || lane + 1 >= found || mine - next > bound(mine, next));
  const float last = __shfl_sync(0xffffffffu, mine, p.top_k - 1);
  if (lane >= p.top_k) chosen = 0;
  if (sure) return chosen;
  int e;
  const int n = candidates<V>(key, order_key(last - 2 * bound(last, last)), own.first, lane, list, &e);
  if (p.softmax || n > 32) return choose64<V, T>(p, row, lane);
  const uint64_t v = value64<T>(p, row, e);
  int rank = 0;
  for (int j = 0; j < n; ++j) {
    const uint64_t other = __shfl_sync(0xffffffffu, v, j);
    const int o = __shfl_sync(0xffffffffu, e, j);
    rank += other > v || (other == v && o < e);
  }
  for (int j = 0; j < p.top_k; ++j) {
    const int who = __ffs(__ballot_sync(0xffffffffu, lane < n && rank == j)) - 1;
    const int o = __shfl_sync(0xffffffffu, e, who);
    if (lane == j) chosen = o;
  }
  return chosen;
}

// The experts of token t and their weights, written; lane j < top_k returns the j-th expert, or -1 for a row that is none.
template <int V, typename T>
__device__ __forceinline__ int choose_token(const RouteParams& p, int t, int real, int lane, int* list) {
  const int64_t out = (int64_t)t * p.top_k + lane;
  if (t >= real) {
    if (lane < p.top_k) {
      p.ids[out] = -1;
      p.weights[out] = 0.f;
      p.places[out] = -1;
    }
    return -1;
  }
  const Own own = own_experts(p, lane);
  const int64_t row = (int64_t)t * p.stride;
  float l[V];
  load_logits<V, T>(p, row, own, l);
  int chosen = 0;
  if (!p.bias && p.num_groups == 1) {
    uint32_t key[V];
#pragma unroll
    for (int i = 0; i < V; ++i) key[i] = i < own.count ? order_key(l[i]) : 0;
    uint32_t its;
    first_in_order<V>(key, own.first, p.top_k, lane, reinterpret_cast<uint2*>(list), &its, &chosen);
    if (lane >= p.top_k) chosen = 0;
  } else {
    chosen = choose<V, T>(p, l, own, row, lane, list);
  }
  // weights: an exponential (a unit in the last place), IEEE quotients and sums in FP32; of sigmoids 7.5 units at most, of a
  // softmax 14 and half a unit for each 1 that a logit lies below the largest
  const bool mine = lane < p.top_k;
  const float lc = load_logit<T>(p.logits, row + chosen);
  float top = 0.f, score;
  if (p.softmax) {
    top = -INFINITY;
#pragma unroll
    for (int i = 0; i < V; ++i) top = fmaxf(top, l[i]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) sum += l[i] == -INFINITY ? 0.f : expf(l[i] - top);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    score = lc == -INFINITY ? 0.f : __fdiv_rn(expf(lc - top), sum);
  } else {
    const float e = expf(-fabsf(lc));  // (at most 1: small scores are not lost to an overflow)
    score = __fdiv_rn(lc < 0.f ? e : 1.f, 1.f + e);
  }
  if (!mine) score = 0.f;
  if (p.normalize) {
    float all = score;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
    // scores near FP32's smallest numbers have no 24 bits: then in 64
    if (__any_sync(0xffffffffu, mine && lc != -INFINITY && (p.softmax ? lc - top : lc) < -80.0f)) {
      double d = 0;
      if (mine && lc != -INFINITY) d = p.softmax ? exp((double)lc - (double)top) : 1.0 / (1.0 + exp(-(double)lc));
      double each = d;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) each += __shfl_xor_sync(0xffffffffu, each, o);
      score = each > 0 ? (float)(d / each) : 0.f;
    } else {
      score = all > 0.0f ? __fdiv_rn(score, all) : 0.f;
    }
  }
  if (mine) {
    p.ids[out] = chosen;
    p.weights[out] = score * p.scale;
  }
  return mine ? chosen : -1;
}

__device__ __forceinline__ int real_tokens(const RouteParams& p) { return p.num_tokens ? *p.num_tokens : p.T; }

template <int V, typename T>
__global__ void __launch_bounds__(kRouteThreads) route_choose_kernel(const __grid_constant__ RouteParams p) {
  const int t = (int)(blockIdx.x * (kRouteThreads / 32) + (threadIdx.x >> 5));
  __shared__ alignas(8) int list[kRouteThreads / 32][64];
  pdl_launch_dependents();
  pdl_wait();
  if (t < p.T) choose_token<V, T>(p, t, real_tokens(p), threadIdx.x & 31, list[threadIdx.x >> 5]);
}

// ---------------------------------------------------------------- places
// The stable counting sort of the choices by expert, by a cluster: each warp has a run of the tokens and counts their
// experts, the counts are summed over a CTA's warps, the cluster's CTAs (each writes its sums to all) and the experts, and
// each choice gets its place.  (A token's experts differ, so a token's choices can be counted at once: matching 32 choices
// across a warp instead took 1400 cycles.)
struct Counts {
  int* warp;   // [warps][E]: of each warp, then those of the warps before it
  int* cta;    // [kPlaceCtas][E]: sums of each CTA of the cluster
  int* base;   // [E]: the first place of this CTA's choices of an expert
  int* carry;  // [warps]
};
template <int W>
__device__ __forceinline__ Counts counts_of(int* smem, int E) {
  return {smem, smem + W * E, smem + (W + kPlaceCtas) * E, smem + (W + kPlaceCtas + 1) * E};
}
inline int counts_bytes(int warps, int E) { return ((warps + kPlaceCtas + 1) * E + warps) * 4; }

// From every warp's counts to the places' bases.  All threads, which have arrived at the cluster's barrier (cluster_arrive):
// no CTA writes to another that has not started.  Nothing touches another CTA after the barrier inside.
template <int W>
__device__ __forceinline__ void sum_counts(const RouteParams& p, const Counts& c, uint32_t rank, uint32_t ctas) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  __syncthreads();
  if (ctas > 1) cluster_wait();
  static_assert(W * 32 >= kRouteMaxExperts, "a thread to an expert");
  const int e = tid;
  if (e < p.E) {
    int n[W], sum = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) n[w] = c.warp[w * p.E + e];
#pragma unroll
    for (int w = 0; w < W; ++w) {
      c.warp[w * p.E + e] = sum;
      sum += n[w];
    }
    const uint32_t at = smem_u32(c.cta + rank * p.E + e);
    for (uint32_t r = 0; r < ctas; ++r) st_cluster_u32(map_to(at, r), (uint32_t)sum);
  }
  if (ctas > 1) cluster_sync(); else __syncthreads();
  int all = 0, before = 0;
  if (e < p.E) {
    for (uint32_t r = 0; r < ctas; ++r) {
      const int n = c.cta[r * p.E + e];
      before += r < rank ? n : 0;
      all += n;
    }
  }
  int up = all;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, up, o);
    if (lane >= o) up += v;
  }
  if (lane == 31) c.carry[warp] = up;
  __syncthreads();
  int sum = 0;
#pragma unroll
  for (int w = 0; w < W; ++w) sum += w < warp ? c.carry[w] : 0;
  sum += up - all;  // choices of the experts before
  if (e < p.E) c.base[e] = sum + before;
  if (rank == 0 && e < p.E) {
    p.starts[e] = sum;
    if (e == p.E - 1) p.starts[p.E] = sum + all;
  }
  __syncthreads();
}

// Choices that another kernel made.
__global__ void __launch_bounds__(kPlaceThreads) route_place_kernel(const __grid_constant__ RouteParams p) {
  extern __shared__ int smem[];
  constexpr int W = kPlaceThreads / 32;
  const uint32_t rank = cluster_rank(), ctas = cluster_size();
  if (ctas > 1) cluster_arrive();
  const Counts c = counts_of<W>(smem, p.E);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int* const mine = c.warp + warp * p.E;
  for (int i = lane; i < p.E; i += 32) mine[i] = 0;
  __syncwarp();
  pdl_launch_dependents();
  pdl_wait();
  // a lane's choice among the warp's tokens, several tokens loaded at a time
  constexpr int kAhead = 16;
  const int warps = (int)ctas * W, run = (p.T + warps - 1) / warps;
  const int first = min(p.T, ((int)rank * W + warp) * run), last = min(p.T, first + run);
  for (int t = first; t < last; t += kAhead) {
    int e[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) e[j] = t + j < last && lane < p.top_k ? p.ids[(int64_t)(t + j) * p.top_k + lane] : -1;
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (e[j] >= 0) p.places[(int64_t)(t + j) * p.top_k + lane] = mine[e[j]]++;
      __syncwarp();
    }
  }
  sum_counts<W>(p, c, rank, ctas);
  const int64_t end = (int64_t)last * p.top_k;
  for (int64_t i = (int64_t)first * p.top_k + lane; i < end; i += 32 * 8) {
    int e[8], at[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const bool is = i + 32 * j < end;
      e[j] = is ? p.ids[i + 32 * j] : -1;
      at[j] = is ? p.places[i + 32 * j] : 0;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (e[j] < 0) continue;
      const int place = c.base[e[j]] + mine[e[j]] + at[j];
      p.places[i + 32 * j] = place;
      p.rows[place] = (int32_t)((uint32_t)(i + 32 * j) / (uint32_t)p.top_k);
    }
  }
}

// Few tokens: the choice and the places in one launch, a warp's tokens one after the other.
template <int V, typename T>
__global__ void __launch_bounds__(kFewThreads) route_few_kernel(const __grid_constant__ RouteParams p) {
  extern __shared__ int smem[];
  constexpr int W = kFewThreads / 32;
  __shared__ alignas(8) int list[W][64];
  const uint32_t rank = cluster_rank(), ctas = cluster_size();
  if (ctas > 1) cluster_arrive();
  const Counts c = counts_of<W>(smem, p.E);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int* const mine = c.warp + warp * p.E;
  for (int i = lane; i < p.E; i += 32) mine[i] = 0;
  __syncwarp();
  pdl_launch_dependents();
  pdl_wait();
  const int warps = (int)ctas * W, each = (p.T + warps - 1) / warps;
  const int first = ((int)rank * W + warp) * each, last = min(p.T, first + each);
  const int real = real_tokens(p);
  for (int t = first; t < last; ++t) {
    const int e = choose_token<V, T>(p, t, real, lane, list[warp]);
    if (e >= 0) p.places[(int64_t)t * p.top_k + lane] = mine[e]++;
    __syncwarp();
  }
  sum_counts<W>(p, c, rank, ctas);
  for (int t = first; t < min(last, real); ++t) {
    if (lane >= p.top_k) continue;
    const int64_t i = (int64_t)t * p.top_k + lane;
    const int e = p.ids[i], place = c.base[e] + mine[e] + p.places[i];
    p.places[i] = place;
    p.rows[place] = t;
  }
}

}  // namespace dsa
