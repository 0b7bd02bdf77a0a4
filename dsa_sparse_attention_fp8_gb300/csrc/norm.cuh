// Residual addition, root-mean-square norm and block quantisation in one pass
// over a row:
//   h = round(x + r)            (to the stored type; h = x without a residual)
//   y = h * rsqrt(mean(h^2) + eps) * w
//   codes = E4M3(y / s), s = amax / 448 over each 128 elements of y, 1 where
//   that is 0 (the rule of the indexer cache), and / or y rounded to the stored
//   type.
// The norm is that of the stored sum, so that whoever reads the residual
// stream back gets the same row.  Sums are held in FP32.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cstdint>
#include <type_traits>

#include "common.cuh"
#include "quantize.cuh"

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

// 8 elements of a row as they lie in memory, and as four pairs in FP32.
// 16-byte accesses where every row starts on a 16-byte boundary and is a
// multiple of 8 elements long; single elements otherwise.  Ordinary loads: the
// sum may be written over x or the residual, and what a kernel writes it may
// not read by way of the read-only path.
template <typename T>
union Norm8 {
  uint4 u[sizeof(T) / 2];
  uint32_t w[2 * sizeof(T)];
  T e[8];
};
template <typename T, bool VEC>
__device__ __forceinline__ Norm8<T> load8(const T* row, int at, int n) {
  Norm8<T> v;
#pragma unroll
  for (int j = 0; j < (int)sizeof(T) / 2; ++j) v.u[j] = make_uint4(0, 0, 0, 0);
  if (VEC) {
#pragma unroll
    for (int j = 0; j < (int)sizeof(T) / 2; ++j)
      if (at < n) v.u[j] = reinterpret_cast<const uint4*>(row + at)[j];
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (at + j < n) v.e[j] = row[at + j];
  }
  return v;
}
template <typename T, bool VEC>
__device__ __forceinline__ void store8(T* row, int at, int n, const Norm8<T>& v) {
  if (VEC) {
#pragma unroll
    for (int j = 0; j < (int)sizeof(T) / 2; ++j)
      if (at < n) reinterpret_cast<uint4*>(row + at)[j] = v.u[j];
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (at + j < n) row[at + j] = v.e[j];
  }
}
template <typename T>
__device__ __forceinline__ float2 widen(const Norm8<T>& v, int i) {
  if constexpr (sizeof(T) == 4)
    return make_float2(v.e[2 * i], v.e[2 * i + 1]);
  else if constexpr (std::is_same_v<T, __nv_bfloat16>)
    return make_float2(__uint_as_float(v.w[i] << 16), __uint_as_float(v.w[i] & 0xFFFF0000u));
  else
    return __half22float2(*reinterpret_cast<const __half2*>(&v.w[i]));
}
template <typename T>
__device__ __forceinline__ void round2(Norm8<T>& v, int i, float2 f) {
  if constexpr (sizeof(T) == 4) {
    v.e[2 * i] = f.x;
    v.e[2 * i + 1] = f.y;
  } else if constexpr (std::is_same_v<T, __nv_bfloat16>) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(f.x, f.y);
    v.w[i] = *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __half2 h = __floats2half2_rn(f.x, f.y);
    v.w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
}

// A CTA per row.  Thread i owns elements [8 i, 8 i + 8) and every 8 * blockDim
// further on, VPT times, in registers from the load to the store, so a row is
// read once; the 16 lanes of half a warp share a 128-element group.  Arithmetic
// is in pairs (packed FP32).  Bound by HBM where rows are many: 8192 rows of
// 7168 bf16 elements, 411 MB read and written, in 74.2 us (5.6 TB/s; with one
// value at a time and VPT = 1, 50 instructions an element, 107 us; with a
// persistent grid that copies two rows ahead into shared memory 85).  Of 64
// rows, 6 us: launch and the latencies of two loads, a barrier and a store.
// Rows that are not a multiple of 8 long, or not aligned, go element by element:
// 8192 rows of 7169 198 us, by their accesses.
template <typename T, bool VEC, int VPT>
__global__ void __launch_bounds__(VPT == 1 ? 1024 : 512) add_rms_norm_kernel(const __grid_constant__ NormParams p) {
  __shared__ float warp_sum[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, step = blockDim.x * 8, row = blockIdx.x;
  const T* x = static_cast<const T*>(p.x) + (int64_t)row * p.x_stride;
  const T* res = static_cast<const T*>(p.residual) + (int64_t)row * p.residual_stride;
  Norm8<T> v[VPT], rv[VPT], wv[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int at = threadIdx.x * 8 + i * step;
    v[i] = load8<T, VEC>(x, at, p.N);
    if (p.residual) rv[i] = load8<T, VEC>(res, at, p.N);
  }
  uint64_t sq2 = 0;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (p.residual) {
        const float2 a = widen(v[i], j), b = widen(rv[i], j);
        round2(v[i], j, unpack2(add2(pack2(a.x, a.y), pack2(b.x, b.y))));
      }
      const float2 h = widen(v[i], j);
      sq2 = fma2(pack2(h.x, h.y), pack2(h.x, h.y), sq2);
    }
    if (p.sum)
      store8<T, VEC>(static_cast<T*>(p.sum) + (int64_t)row * p.sum_stride, threadIdx.x * 8 + i * step, p.N, v[i]);
  }
  // (the weights' loads fall into the sum's)
#pragma unroll
  for (int i = 0; i < VPT; ++i) wv[i] = load8<T, VEC>(static_cast<const T*>(p.weight), threadIdx.x * 8 + i * step, p.N);
  float sq = unpack2(sq2).x + unpack2(sq2).y;
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
    Norm8<T> out;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 h = widen(v[i], j), w = widen(wv[i], j);
      const float2 f = unpack2(mul2(mul2(pack2(h.x, h.y), pack2(rstd, rstd)), pack2(w.x, w.y)));
      y[2 * j] = f.x;
      y[2 * j + 1] = f.y;
      amax = max3(amax, fabsf(f.x), fabsf(f.y));
      if (p.out) round2(out, j, f);
    }
    if (p.out) store8<T, VEC>(static_cast<T*>(p.out) + (int64_t)row * p.out_stride, at, p.N, out);
    if (!p.codes) continue;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    // 1 for a group of zeros, and for one of FP32's smallest numbers, whose
    // scale would be 0 (and 0 / 0 no code)
    const float step = __fdiv_rn(amax, 448.0f), s = step == 0.f ? 1.0f : step;
    const uint2 c = quantize8(y, s);
    if (at < p.N) {
      uint8_t* dst = p.codes + (int64_t)row * p.N + at;
      if (VEC) {
        *reinterpret_cast<uint2*>(dst) = c;
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (at + j < p.N) dst[j] = (uint8_t)((j < 4 ? c.x : c.y) >> (8 * (j & 3)));
      }
      if ((lane & 15) == 0) p.scales[(int64_t)row * ((p.N + kNormGroup - 1) / kNormGroup) + at / kNormGroup] = s;
    }
  }
}

}  // namespace dsa
