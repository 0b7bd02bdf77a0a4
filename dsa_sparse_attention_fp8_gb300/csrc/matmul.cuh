// Products of rows and weights, in one group or grouped by expert:
//   y[i, n] = sum_b xs[r, b] ws[n / 128, b] sum_{k in block b} x[r, k] w[n, k]
// with r = rows[i] or i, w and ws those of i's group; blocks of 128 along K (E4M3), or one sum without scales (16 bits).
// Gated: silu(y[i, n]) * y[i, N/2 + n].  Written rounded, or as E4M3 with a scale per 128 elements.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cstdint>

#include "common.cuh"
#include "quantize.cuh"

namespace dsa {

constexpr int kMatmulMaxGroups = 1024;
constexpr int kMatmulBlock = 128;  // elements of K and weight rows that share a scale

struct MatmulParams {
  const void* x;
  const float* x_scales;     // [x_rows, kb], E4M3 only
  const int32_t* rows;       // [M], or null
  const void* w;
  const float* w_scales;     // [E, nb, kb], E4M3 only
  const int32_t* starts;     // [E + 1], or null: one group of all M rows
  void* out;                 // or null: codes and scales
  uint8_t* codes;
  float* scales;
  int32_t* status;
  int64_t x_stride, w_stride, w_group, out_stride;  // elements
  int x_rows, M, N, K, E, width, kb, nb;            // width: N, or N / 2 where gated
  int x_type, out_type;
  bool gated;
};

__device__ __forceinline__ float load_element(const void* p, int64_t at, int type) {
  if (type == 0) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[at]);
  if (type == 1) return __half2float(static_cast<const __half*>(p)[at]);
  if (type == 2) return static_cast<const float*>(p)[at];
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(static_cast<const uint8_t*>(p)[at], __NV_E4M3)));
}
__device__ __forceinline__ void store_element(void* p, int64_t at, int type, float v) {
  if (type == 0) static_cast<__nv_bfloat16*>(p)[at] = __float2bfloat16_rn(v);
  else if (type == 1) static_cast<__half*>(p)[at] = __float2half_rn(v);
  else static_cast<float*>(p)[at] = v;
}

// A thread has a column of 16 rows.
constexpr int kSimpleRows = 16;
__global__ void __launch_bounds__(128) matmul_kernel(const __grid_constant__ MatmulParams p) {
  __shared__ float xt[kSimpleRows][128];
  __shared__ float most[kSimpleRows][4];
  __shared__ int src[kSimpleRows];
  const int tid = threadIdx.x;
  // the group and first row of this tile
  int e = 0, begin = 0, end = p.M, tile = blockIdx.x;
  if (p.starts) {
    for (e = 0; e < p.E; ++e) {
      begin = p.starts[e], end = p.starts[e + 1];
      if (begin < 0 || end > p.M || end < begin) {
        if (blockIdx.x == 0 && blockIdx.y == 0 && tid == 0) raise_status(p.status, kStatusBadMetadata);
        continue;
      }
      const int tiles = (end - begin + kSimpleRows - 1) / kSimpleRows;
      if (tile < tiles) break;
      tile -= tiles;
    }
    if (e == p.E) return;
  }
  begin += tile * kSimpleRows;
  const int count = min(kSimpleRows, end - begin);
  if (count <= 0) return;
  if (tid < kSimpleRows) {
    int r = -1;
    if (tid < count) {
      r = p.rows ? p.rows[begin + tid] : begin + tid;
      if (r < 0 || r >= p.x_rows) {
        raise_status(p.status, kStatusBadMetadata);
        r = -1;
      }
    }
    src[tid] = r;
  }
  const int c = blockIdx.y * 128 + tid;
  const bool real = c < p.width;
  float acc[2][kSimpleRows] = {};
  for (int b = 0; b < p.kb; ++b) {
    __syncthreads();
    const int k0 = b * 128, n = min(128, p.K - k0);
    for (int i = 0; i < kSimpleRows; ++i)
      xt[i][tid] = src[i] >= 0 && tid < n ? load_element(p.x, (int64_t)src[i] * p.x_stride + k0 + tid, p.x_type) : 0.f;
    __syncthreads();
    if (!real) continue;
    for (int h = 0; h < (p.gated ? 2 : 1); ++h) {
      const int row = c + h * p.width;
      const int64_t at = (int64_t)e * p.w_group + (int64_t)row * p.w_stride + k0;
      float part[kSimpleRows] = {};
      for (int k = 0; k < n; ++k) {
        const float w = load_element(p.w, at + k, p.x_type);
        for (int i = 0; i < kSimpleRows; ++i) part[i] = fmaf(xt[i][k], w, part[i]);
      }
      const float ws = p.w_scales ? p.w_scales[((int64_t)e * p.nb + row / 128) * p.kb + b] : 1.f;
      for (int i = 0; i < kSimpleRows; ++i) {
        const float xs = p.x_scales && src[i] >= 0 ? p.x_scales[(int64_t)src[i] * p.kb + b] : 1.f;
        if (src[i] >= 0) acc[h][i] = fmaf(part[i], xs * ws, acc[h][i]);
      }
    }
  }
  for (int i = 0; i < count; ++i) {
    float y = acc[0][i];
    if (p.gated) y = y / (1.f + __expf(-y)) * acc[1][i];
    if (!real) y = 0.f;
    if (p.out) {
      if (real) store_element(p.out, (int64_t)(begin + i) * p.out_stride + c, p.out_type, y);
      continue;
    }
    float amax = fabsf(y);
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if ((tid & 31) == 0) most[i][tid >> 5] = amax;
    __syncthreads();
    amax = fmaxf(fmaxf(most[i][0], most[i][1]), fmaxf(most[i][2], most[i][3]));
    const float step = __fdiv_rn(amax, 448.0f), s = step == 0.f ? 1.0f : step;
    if (!real) continue;
    p.codes[(int64_t)(begin + i) * p.width + c] = __nv_cvt_float_to_fp8(__fdiv_rn(y, s), __NV_SATFINITE, __NV_E4M3);
    if (tid == 0) p.scales[(int64_t)(begin + i) * ((p.width + 127) / 128) + blockIdx.y] = s;
  }
}

}  // namespace dsa
