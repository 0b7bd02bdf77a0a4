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

namespace dsa {

struct KvWriteParams {
  const uint16_t* src[2];       // k, v: [T, Hkv, D], element strides below
  int64_t src_token[2], src_head[2];
  const int64_t* slots;         // [T]
  int T, heads, dim;
  int tokens;                   // of a CTA
  uint32_t per_token;           // ceil(2^16 / rows of a token): row * this >> 16 is the row's token, for rows < 64
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

// A row is one head of one token's key or value.  16 lanes own a row, 8
// elements (16 bytes) each, so a warp reads two rows of up to 256 bytes with
// one instruction, and a row's maximum takes four shuffles.  kRows rows per
// lane are in flight at once; a CTA has the rows of `tokens` tokens.  8192
// tokens of 8 + 8 heads of 128 bf16 elements into an E4M3 cache, 51 MB read and
// written, take 24.7 us (2.1 TB/s; from L2, where the rows of a step are, and
// bound by its scattered writes of 128 bytes and of a scale's 4), 64 tokens 4 to
// 5 us, a launch.
constexpr int kKvThreads = 256;
constexpr int kKvRows = 4;

template <bool BF16, bool FP8>
__global__ void __launch_bounds__(kKvThreads) kv_write_kernel(const __grid_constant__ KvWriteParams p) {
  constexpr int kRows = kKvRows;
  const int lane = threadIdx.x & 15;
  const int64_t t0 = (int64_t)blockIdx.x * p.tokens;
  const int rows = (int)min((int64_t)p.tokens, p.T - t0) * 2 * p.heads;  // (token, k or v, head)
  for (int first = threadIdx.x >> 4; first - (int)(threadIdx.x >> 4) < rows; first += kKvThreads / 16 * kRows) {
    uint4 x[kRows];
    int64_t slot[kRows];
    int which[kRows], head[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int row = first + i * (kKvThreads / 16);
      x[i] = make_uint4(0, 0, 0, 0);
      slot[i] = -1;
      which[i] = head[i] = 0;
      if (row < rows) {
        const int t = (int)((uint32_t)row * p.per_token >> 16), rest = row - t * (2 * p.heads);
        which[i] = rest >= p.heads;
        head[i] = rest - which[i] * p.heads;
        slot[i] = __ldg(p.slots + t0 + t);
        if (lane * 8 < p.dim)
          x[i] = __ldg(reinterpret_cast<const uint4*>(p.src[which[i]] + (t0 + t) * p.src_token[which[i]] +
                                                      head[i] * p.src_head[which[i]] + lane * 8));
      }
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int w = which[i];
      const int64_t page = slot[i] >> 6;  // (64 tokens)
      const int off = (int)(slot[i] & 63);
      const bool live = slot[i] >= 0 && page < p.num_pages;
      if (slot[i] >= 0 && !live && lane == 0) raise_status(p.status, kStatusBadPage);
      uint8_t* dst = p.cache[w] + page * p.page_stride[w] + off * p.token_stride[w] + head[i] * p.head_stride[w];
      if (!FP8) {
        if (live && lane * 8 < p.dim) *reinterpret_cast<uint4*>(dst + lane * 16) = x[i];
        continue;
      }
      const uint32_t u[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
      float f[8];
      float amax = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 w2 = widen2<BF16>(u[j]);
        f[2 * j] = w2.x;
        f[2 * j + 1] = w2.y;
        amax = fmaxf(amax, fmaxf(fabsf(w2.x), fabsf(w2.y)));
      }
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      const float s = amax == 0.f ? 1.0f : __fdiv_rn(amax, 448.0f);
      const uint2 c = quantize8(f, s);
      if (live) {
        if (lane * 8 < p.dim)
          *reinterpret_cast<uint2*>(dst + lane * 8) = c;
        if (lane == 0) p.scale[w][page * p.scale_page[w] + head[i] * p.scale_head[w] + off] = s;
      }
    }
  }
}

}  // namespace dsa
