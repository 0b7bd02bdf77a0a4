// K/V cache write: each new token's key and value heads into a paged cache at
// its slot (page * 64 + offset), as they are (16-bit caches) or as E4M3 codes
// with one FP32 scale per (token, head) by the rule of the indexer cache
// (s = amax / 448 in IEEE FP32, s = 1 for an all-zero row, codes E4M3(x / s),
// nearest even, saturating).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cstdint>

#include "common.cuh"
#include "quantize.cuh"

namespace dsa {

struct KvWriteParams {
  const uint16_t* src[2];       // k, v: [T, Hkv, D], element strides below
  int64_t src_token[2], src_head[2];
  const int64_t* slots;         // [T]
  int T, heads, dim;
  int tokens;                   // of a CTA
  uint32_t per_token;           // pair * this >> 16 is the pair's token: ceil(2^16 / heads), 0 for one token
  uint8_t* cache[2];            // [num_pages, 64, Hkv, D], byte strides below
  int64_t page_stride[2], token_stride[2], head_stride[2];
  float* scale[2];              // [num_pages, Hkv, 64], element strides below (E4M3 caches)
  int64_t scale_page[2], scale_head[2];
  int64_t num_pages;
  int32_t* status;
};

template <bool BF16>
__device__ __forceinline__ float2 widen2(uint32_t w) {
  if (BF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

// A pair is one head of one token, its key and its value.  16 lanes own a pair,
// 8 elements (16 bytes) of each each, so a warp reads two rows of up to 256
// bytes with one instruction, and a row's maximum takes four shuffles.  A CTA
// has the pairs of `tokens` tokens.  8192 tokens of 8 heads of 128 bf16 elements:
// into a cache of the same type, 67 MB read and written, 11.9 us (5.6 TB/s,
// bound by HBM and L2); into an E4M3 cache, 51 MB, 16.5 to 19.3 us (3.0 to 2.6
// TB/s), bound by the instructions of the quantisation (with four rows a lane,
// each with its own address arithmetic and divisions, 24.7).  64 tokens: 2.7 us,
// a launch (4.0 with four rows a lane).
constexpr int kKvThreads = 128;

template <bool BF16, bool FP8>
__global__ void __launch_bounds__(kKvThreads) kv_write_kernel(const __grid_constant__ KvWriteParams p) {
  const int lane = threadIdx.x & 15, d = lane * 8;
  const int64_t t0 = (int64_t)blockIdx.x * p.tokens;
  const int pairs = (int)min((int64_t)p.tokens, p.T - t0) * p.heads;
  for (int first = threadIdx.x >> 4 & ~1; first < pairs; first += kKvThreads / 16) {  // (a warp's two pairs together)
    const int pair = first + (threadIdx.x >> 4 & 1);
    const int t = (int)((uint32_t)pair * p.per_token >> 16), head = pair - t * p.heads;
    const bool in = pair < pairs;
    const int64_t slot = in ? __ldg(p.slots + t0 + t) : -1;
    uint4 x[2];
#pragma unroll
    for (int w = 0; w < 2; ++w)
      x[w] = in && d < p.dim ? __ldg(reinterpret_cast<const uint4*>(p.src[w] + (t0 + t) * p.src_token[w] +
                                                                    head * p.src_head[w] + d))
                             : make_uint4(0, 0, 0, 0);
    const int64_t page = slot >> 6;  // (64 tokens)
    const int off = (int)(slot & 63);
    const bool live = slot >= 0 && page < p.num_pages;
    if (slot >= 0 && !live && lane == 0) raise_status(p.status, kStatusBadPage);
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      uint8_t* dst = p.cache[w] + page * p.page_stride[w] + off * p.token_stride[w] + head * p.head_stride[w];
      if (!FP8) {
        if (live && d < p.dim) *reinterpret_cast<uint4*>(dst + lane * 16) = x[w];
        continue;
      }
      const uint32_t u[4] = {x[w].x, x[w].y, x[w].z, x[w].w};
      float f[8];
      float amax = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 w2 = widen2<BF16>(u[j]);
        f[2 * j] = w2.x;
        f[2 * j + 1] = w2.y;
        amax = max3(amax, fabsf(w2.x), fabsf(w2.y));
      }
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      const float s = amax == 0.f ? 1.0f : __fdiv_rn(amax, 448.0f);
      const uint2 c = quantize8(f, s);
      if (live) {
        if (d < p.dim) *reinterpret_cast<uint2*>(dst + d) = c;
        if (lane == 0) p.scale[w][page * p.scale_page[w] + head * p.scale_head[w] + off] = s;
      }
    }
  }
}

}  // namespace dsa
