// E4M3 codes by the rule of the indexer cache, for rows that a thread holds in
// eights.
#pragma once

#include <cuda_fp8.h>
#include <cstdint>

#include "ptx_serving.cuh"

namespace dsa {

// E4M3 codes of 8 values over a common scale, E4M3(x / s) with IEEE FP32
// division, nearest even, saturating; four codes to a word.  The quotient lies
// between x * (1 / s) a little too small and a little too large (1 / s is off by
// 2^-23 at most, the factor, the product and the division by 2^-24 each, and the
// factors are 2^-21 apart from 1): where both round to the same code, that is
// the quotient's, and only where they do not, some 1 in 10^5 values, is the
// division done.  (Below 1e-30 and above 1e37 the reciprocal may leave the
// normal numbers.)
__device__ __forceinline__ uint2 quantize8(const float* x, float s) {
  const float inv = rcp_approx(s);
  const uint64_t lo = pack2(inv * (1.0f - 0x1p-21f), inv * (1.0f - 0x1p-21f));
  const uint64_t hi = pack2(inv * (1.0f + 0x1p-21f), inv * (1.0f + 0x1p-21f));
  uint32_t c[4], differ = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint64_t v = pack2(x[2 * i], x[2 * i + 1]);
    c[i] = __nv_cvt_float2_to_fp8x2(unpack2(mul2(v, lo)), __NV_SATFINITE, __NV_E4M3);
    differ |= c[i] ^ __nv_cvt_float2_to_fp8x2(unpack2(mul2(v, hi)), __NV_SATFINITE, __NV_E4M3);
  }
  if (differ || s < 1e-30f || s > 1e37f) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      c[i] = __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(x[2 * i], s), __fdiv_rn(x[2 * i + 1], s)), __NV_SATFINITE,
                                      __NV_E4M3);
  }
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

}  // namespace dsa
