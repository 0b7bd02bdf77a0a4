// Device-side pieces shared by every kernel of the library: the page size, the
// status bits and the request search.
#pragma once

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

}  // namespace dsa
