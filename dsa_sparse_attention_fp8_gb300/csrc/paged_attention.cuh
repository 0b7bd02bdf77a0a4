// Attention of a chunk of new tokens over a paged K/V cache.
//
// Row t of request r sits at position p = seq - q + (t - start[r]); head h
// reads key head h / (Hq / Hkv).  With z_s = scale * q . k_s over the visible
// tokens s (s <= p, and with a window s > p - window or s < sinks):
//   lse = ln sum_s exp(z_s),  out = sum_s exp(z_s - lse) v_s.
// A row that sees nothing gives out = 0, lse = -inf.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cstdint>

#include "common.cuh"

namespace dsa {

struct AttnParams {
  const uint16_t* q;           // [T, Hq, D], element strides
  int64_t q_token, q_head;
  uint16_t* out;               // [T, Hq, D], element strides
  int64_t out_token, out_head;
  float* lse;                  // [T, Hq] or null
  const uint8_t* cache[2];     // [num_pages, 64, Hkv, D], byte strides
  int64_t page_stride[2], token_stride[2], head_stride[2];
  const float* scale[2];       // [num_pages, Hkv, 64], element strides (E4M3 caches)
  int64_t scale_page[2], scale_head[2];
  int64_t num_pages;
  const int32_t* start;        // [R + 1]
  const int32_t* seq_lens;     // [R]
  const int32_t* block_table;  // [R, max_blocks]
  int R, max_blocks, T, Hq, Hkv, D;
  int window, sinks;
  float scale_log2;            // softmax scale * log2(e)
  int32_t* status;
};

template <bool BF16>
__device__ __forceinline__ float widen1(uint16_t v) {
  return BF16 ? __uint_as_float((uint32_t)v << 16) : __half2float(__ushort_as_half(v));
}

// One warp per (row, head), lane l owning elements l, l + 32, ...: a plain
// online softmax over the row's keys.
template <bool BF16, bool FP8>
__global__ void __launch_bounds__(256) paged_attention_simple_kernel(const __grid_constant__ AttnParams p) {
  const int64_t warp = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  if (warp >= (int64_t)p.T * p.Hq) return;
  const int t = (int)(warp / p.Hq), hq = (int)(warp % p.Hq), h = hq / (p.Hq / p.Hkv);
  const int r = find_request(p.start, p.R, t);
  const int s0 = __ldg(p.start + r), s1 = __ldg(p.start + r + 1), seq = __ldg(p.seq_lens + r);
  float acc[4] = {0.f, 0.f, 0.f, 0.f}, q[4] = {0.f, 0.f, 0.f, 0.f};
  float m = -INFINITY, l = 0.f;
  const bool mine = t >= s0 && t < s1;  // rows past the last request belong to none
  const bool ok = mine && s0 >= 0 && s1 <= p.T && seq >= s1 - s0 && (int64_t)seq <= (int64_t)p.max_blocks * kPageTokens;
  if (mine && !ok && lane == 0) raise_status(p.status, kStatusBadMetadata);
  if (ok) {
    const int pos = seq - (s1 - s0) + (t - s0);
    for (int i = 0; i < 4; ++i)
      if (lane + 32 * i < p.D) q[i] = widen1<BF16>(p.q[t * p.q_token + hq * p.q_head + lane + 32 * i]);
    const int far = p.window > 0 && pos >= p.window ? pos - p.window + 1 : 0;
    for (int s = 0; s <= pos; ++s) {
      if (s < far && s >= p.sinks) { s = far - 1; continue; }
      const int64_t page = __ldg(p.block_table + (int64_t)r * p.max_blocks + s / kPageTokens);
      if (page < 0 || page >= p.num_pages) {
        if (lane == 0) raise_status(p.status, kStatusBadPage);
        continue;
      }
      const int off = s % kPageTokens;
      const uint8_t* row[2];
      float sc[2] = {1.f, 1.f};
      for (int w = 0; w < 2; ++w) {
        row[w] = p.cache[w] + page * p.page_stride[w] + off * p.token_stride[w] + h * p.head_stride[w];
        if (FP8) sc[w] = __ldg(p.scale[w] + page * p.scale_page[w] + h * p.scale_head[w] + off);
      }
      auto at = [&](int w, int j) -> float {
        if (FP8) {
          const __half_raw x = __nv_cvt_fp8_to_halfraw(row[w][j], __NV_E4M3);
          return __half2float(*reinterpret_cast<const __half*>(&x)) * sc[w];
        }
        return widen1<BF16>(reinterpret_cast<const uint16_t*>(row[w])[j]);
      };
      float z = 0.f;
      for (int i = 0; i < 4; ++i)
        if (lane + 32 * i < p.D) z += q[i] * at(0, lane + 32 * i);
      for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
      z *= p.scale_log2;
      const float mn = fmaxf(m, z), a = m == -INFINITY ? 0.f : exp2f(m - mn);
      const float e = mn == -INFINITY ? 0.f : exp2f(z - mn);
      l = l * a + e;
      for (int i = 0; i < 4; ++i)
        if (lane + 32 * i < p.D) acc[i] = acc[i] * a + e * at(1, lane + 32 * i);
      m = mn;
    }
  }
  for (int i = 0; i < 4; ++i)
    if (lane + 32 * i < p.D) {
      const float o = l > 0.f ? acc[i] / l : 0.f;
      p.out[t * p.out_token + hq * p.out_head + lane + 32 * i] =
          BF16 ? __bfloat16_as_ushort(__float2bfloat16_rn(o)) : __half_as_ushort(__float2half_rn(o));
    }
  if (p.lse && lane == 0)
    p.lse[(int64_t)t * p.Hq + hq] = l > 0.f ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
}

}  // namespace dsa
