// Residual addition, root-mean-square norm and block quantisation in one pass
// over a row:
//   h = round(x + r)            (to the stored type; h = x without a residual)
//   y = h * rsqrt(mean(h^2) + eps) * w
//   codes = E4M3(y / s), s = amax / 448 over each 128 elements of y (the rule
//   of the indexer cache), and / or y rounded to the stored type.
// The norm is that of the stored sum, so that whoever reads the residual
// stream back gets the same row.  Sums are held in FP32.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cstdint>

#include "common.cuh"

namespace dsa {

constexpr int kNormGroup = 128;
constexpr int kNormMaxWidth = 32768;

struct NormParams {
  const void* x;
  const void* residual;      // or null
  const void* weight;        // [N]
  void* sum;                 // h, or null
  void* out;                 // y rounded, or null
  uint8_t* codes;            // [T, N], or null
  float* scales;             // [T, ceil(N / 128)]
  int64_t x_stride, residual_stride, sum_stride, out_stride;  // elements between rows
  int T, N;
  float eps;
};

// The stored types: 8 consecutive elements of a row as FP32, and back.
template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f32(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32(float v) { return __float2bfloat16_rn(v); }

// 8 elements of a row as they lie in memory.  16-byte accesses where every row
// starts on a 16-byte boundary and is a multiple of 8 elements long; single
// elements otherwise.
template <typename T>
union Norm8 {
  uint4 u[sizeof(T) / 2];
  T e[8];
};
template <typename T, bool VEC>
__device__ __forceinline__ Norm8<T> load8(const T* row, int at, int n) {
  Norm8<T> v;
  if (VEC) {
#pragma unroll
    for (int j = 0; j < (int)sizeof(T) / 2; ++j)
      v.u[j] = at < n ? __ldg(reinterpret_cast<const uint4*>(row + at) + j) : make_uint4(0, 0, 0, 0);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v.e[j] = at + j < n ? row[at + j] : from_f32<T>(0.f);
  }
  return v;
}
template <typename T, bool VEC>
__device__ __forceinline__ void store8(T* row, int at, int n, const float* f) {
  if (VEC) {
    Norm8<T> v;
#pragma unroll
    for (int j = 0; j < 8; ++j) v.e[j] = from_f32<T>(f[j]);
#pragma unroll
    for (int j = 0; j < (int)sizeof(T) / 2; ++j) reinterpret_cast<uint4*>(row + at)[j] = v.u[j];
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (at + j < n) row[at + j] = from_f32<T>(f[j]);
  }
}

// A CTA per row; thread i owns elements [8 i, 8 i + 8) and every 8 * blockDim
// further on, VPT times, in registers from the load to the store, so a row is
// read once.  The 16 lanes of half a warp share a 128-element group.
template <typename T, bool VEC, int VPT>
__global__ void __launch_bounds__(VPT == 1 ? 1024 : 512) add_rms_norm_kernel(const __grid_constant__ NormParams p) {
  __shared__ float warp_sum[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, step = blockDim.x * 8, row = blockIdx.x;
  const T* x = static_cast<const T*>(p.x) + (int64_t)row * p.x_stride;
  const T* res = p.residual ? static_cast<const T*>(p.residual) + (int64_t)row * p.residual_stride : nullptr;
  Norm8<T> v[VPT], rv[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int at = threadIdx.x * 8 + i * step;
    v[i] = load8<T, VEC>(x, at, p.N);
    if (res) rv[i] = load8<T, VEC>(res, at, p.N);
  }
  float sq = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int at = threadIdx.x * 8 + i * step;
    float h[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (res) v[i].e[j] = from_f32<T>(to_f32(v[i].e[j]) + to_f32(rv[i].e[j]));
      h[j] = to_f32(v[i].e[j]);
      sq += h[j] * h[j];
    }
    if (p.sum && at < p.N) store8<T, VEC>(static_cast<T*>(p.sum) + (int64_t)row * p.sum_stride, at, p.N, h);
  }
  // (the weights' loads fall into the sum's)
  Norm8<T> wv[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) wv[i] = load8<T, VEC>(static_cast<const T*>(p.weight), threadIdx.x * 8 + i * step, p.N);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
  if (lane == 0) warp_sum[warp] = sq;
  __syncthreads();
  float total = lane < (int)(blockDim.x >> 5) ? warp_sum[lane] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  const float rstd = 1.0f / sqrtf(total / (float)p.N + p.eps);
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int at = threadIdx.x * 8 + i * step;
    float y[8];
    float amax = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      y[j] = to_f32(v[i].e[j]) * rstd * to_f32(wv[i].e[j]);
      amax = fmaxf(amax, fabsf(y[j]));
    }
    if (p.out && at < p.N)
      store8<T, VEC>(static_cast<T*>(p.out) + (int64_t)row * p.out_stride, at, p.N, y);
    if (!p.codes) continue;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const float s = amax == 0.f ? 1.0f : __fdiv_rn(amax, 448.0f);
    uint32_t c[4];
    quantize8(y, s, c);
    if (at < p.N) {
      uint8_t* dst = p.codes + (int64_t)row * p.N + at;
      if (VEC) {
        *reinterpret_cast<uint2*>(dst) = make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (at + j < p.N) dst[j] = (uint8_t)(c[j >> 1] >> (8 * (j & 1)));
      }
      if ((lane & 15) == 0) p.scales[(int64_t)row * ((p.N + kNormGroup - 1) / kNormGroup) + at / kNormGroup] = s;
    }
  }
}

}  // namespace dsa
