// The experts' rows back to their tokens: out[t] = add[t] + sum_j w[t, j] y[places[t, j]], in FP32, one rounding.
#pragma once

#include <cstdint>

#include "common.cuh"
#include "norm.cuh"
#include "ptx.cuh"

namespace dsa {

constexpr int kCombineMaxTop = 16;

struct CombineParams {
  const void* y;
  const int32_t* places;   // [T, top_k]
  const float* weights;    // [T, top_k]
  const void* add;         // or null
  void* out;
  int32_t* status;
  int64_t y_stride, add_stride, out_stride;  // elements
  int M, T, top_k, N;
};

// A thread has 8 elements of a token; blockIdx.y is the slice of the row.  All of a token's rows are asked for before the
// first is added.  `add` may be `out` itself: ordinary loads.  Bound by HBM: 8192 tokens of eight rows of 7168 bf16
// elements, 1.17 GB in 199 us (5.9 TB/s, 87 % of the copy rate); 64 tokens 3.8 us, two latencies and the launch (a CTA to a
// token, row after row, 10).
constexpr int kCombineThreads = 128;
template <typename T, bool VEC>
__global__ void __launch_bounds__(kCombineThreads) combine_kernel(const __grid_constant__ CombineParams p) {
  constexpr int kAhead = 8;
  const int t = blockIdx.x;
  const int32_t* const places = p.places + (int64_t)t * p.top_k;
  const float* const weights = p.weights + (int64_t)t * p.top_k;
  pdl_launch_dependents();
  pdl_wait();
  for (int at = (blockIdx.y * kCombineThreads + threadIdx.x) * 8; at < p.N; at += gridDim.y * kCombineThreads * 8) {
    float sum[8] = {};
    Norm8<T> own;
    if (p.add) own = load8<T, VEC>(static_cast<const T*>(p.add) + (int64_t)t * p.add_stride, at, p.N);
    for (int j0 = 0; j0 < p.top_k; j0 += kAhead) {
      int place[kAhead];
      float w[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const bool is = j0 + j < p.top_k;
        place[j] = is ? places[j0 + j] : -1;
        w[j] = is ? weights[j0 + j] : 0.f;
      }
      Norm8<T> v[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        if (place[j] >= p.M) {
          if (at == 0) raise_status(p.status, kStatusBadMetadata);
          place[j] = -1;
        }
        if (place[j] >= 0) v[j] = load8<T, VEC>(static_cast<const T*>(p.y) + (int64_t)place[j] * p.y_stride, at, p.N);
      }
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        if (place[j] < 0) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = widen(v[j], i);
          sum[2 * i] = fmaf(w[j], f.x, sum[2 * i]);
          sum[2 * i + 1] = fmaf(w[j], f.y, sum[2 * i + 1]);
        }
      }
    }
    Norm8<T> out;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float2 f = make_float2(sum[2 * i], sum[2 * i + 1]);
      if (p.add) {
        const float2 a = widen(own, i);
        f.x += a.x, f.y += a.y;
      }
      round2(out, i, f);
    }
    store8<T, VEC>(static_cast<T*>(p.out) + (int64_t)t * p.out_stride, at, p.N, out);
  }
}

}  // namespace dsa
