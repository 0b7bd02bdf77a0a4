// Device-side pieces shared by every kernel of the library: the page size, the
// status bits and the request search.
#pragma once

#include <cuda_fp8.h>
#include <cstdint>

namespace dsa {

constexpr int kPageTokens = 64;

constexpr int kStatusBadPage = 0x1;
constexpr int kStatusBadMetadata = 0x2;
constexpr int kStatusTimeout = 0x4;
constexpr int kStatusNoPages = 0x8;

__device__ __forceinline__ void raise_status(int32_t* status, int bits) {
  if (status) atomicOr(status, bits);
}

// Request that owns query row t: the last r with query_start_loc[r] <= t.
__device__ __forceinline__ int find_request(const int32_t* __restrict__ qsl, int R, int t) {
  int lo = 0, hi = R - 1;
  while (lo < hi) {
    int mid = (lo + hi + 1) >> 1;
    if (__ldg(qsl + mid) <= t) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// E4M3 codes of 8 values over a common scale, E4M3(x / s) with IEEE FP32
// division, nearest even, saturating; two codes to a word's lower half.  The
// quotient is taken as x * (1 / s), at most 2 units in the last place off,
// which changes no code unless it lies that near to a border between two
// codes: in the normal range those are the values whose lower 20 bits are
// 0x80000.  There, and in E4M3's subnormal range, the division is done.
__device__ __forceinline__ void quantize8(const float* x, float s, uint32_t* codes) {
  const float inv = __fdiv_rn(1.0f, s);
  float q[8];
  bool near = s < 1e-30f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    q[i] = x[i] * inv;
    near |= ((__float_as_uint(q[i]) - 0x7FFFCu) & 0xFFFFFu) <= 8u || fabsf(q[i]) < 0.015625f;
  }
  if (near) {
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = __fdiv_rn(x[i], s);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    codes[i] = __nv_cvt_float2_to_fp8x2(make_float2(q[2 * i], q[2 * i + 1]), __NV_SATFINITE, __NV_E4M3) & 0xFFFFu;
}

}  // namespace dsa
