// The experts' rows back to their tokens: out[t] = add[t] + sum_j w[t, j] y[places[t, j]], in FP32, one rounding.
#pragma once

#include <cstdint>

#include "common.cuh"
#include "norm.cuh"

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

// A CTA per token.  `add` may be `out` itself: ordinary loads.
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) combine_kernel(const __grid_constant__ CombineParams p) {
  const int t = blockIdx.x;
  const int32_t* places = p.places + (int64_t)t * p.top_k;
  const float* weights = p.weights + (int64_t)t * p.top_k;
  for (int at = threadIdx.x * 8; at < p.N; at += blockDim.x * 8) {
    float sum[8] = {};
    for (int j = 0; j < p.top_k; ++j) {
      const int place = places[j];
      if (place >= p.M) {
        if (at == 0) raise_status(p.status, kStatusBadMetadata);
        continue;
      }
      if (place < 0) continue;
      const Norm8<T> v = load8<T, VEC>(static_cast<const T*>(p.y) + (int64_t)place * p.y_stride, at, p.N);
      const float w = weights[j];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = widen(v, i);
        sum[2 * i] = fmaf(w, f.x, sum[2 * i]);
        sum[2 * i + 1] = fmaf(w, f.y, sum[2 * i + 1]);
      }
    }
    if (p.add) {
      const Norm8<T> v = load8<T, VEC>(static_cast<const T*>(p.add) + (int64_t)t * p.add_stride, at, p.N);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = widen(v, i);
        sum[2 * i] += f.x;
        sum[2 * i + 1] += f.y;
      }
    }
    Norm8<T> out;
#pragma unroll
    for (int i = 0; i < 4; ++i) round2(out, i, make_float2(sum[2 * i], sum[2 * i + 1]));
    store8<T, VEC>(static_cast<T*>(p.out) + (int64_t)t * p.out_stride, at, p.N, out);
  }
}

}  // namespace dsa
