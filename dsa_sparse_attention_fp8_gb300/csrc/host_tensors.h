// Host-side checks of tensors and their tensor maps, shared by the entry points'
// translation units.
#pragma once

#include <cuda.h>

#include <cstdint>

#include "dsa_indexer.h"
#include "host.h"

namespace dsa_host {

inline int element_bytes(int type) { return type == DSA_TYPE_FP32 ? 4 : type == DSA_TYPE_E4M3 ? 1 : 2; }

// Whether a stride over n elements is neither negative nor off a multiple of
// `unit` (one element may have any stride: nothing is ever a stride away).
inline bool stride_ok(int64_t stride, int64_t n, int unit) { return n <= 1 || (stride >= 0 && stride % unit == 0); }

// Whether a stride over n elements keeps them apart, as what is written, or read
// by way of a tensor map, has to be.
inline bool apart(int64_t stride, int64_t n) { return n <= 1 || stride != 0; }

// A map over up to four dimensions, innermost first; strides in bytes (of
// dimensions 1 on).  A dimension of one element may have any stride: it gets
// one that the encoder takes.
inline int make_map(CUtensorMap* m, const char* what, CUtensorMapDataType type, int size, const void* base, int rank,
             const int64_t* dims, const int64_t* strides, const int* box, bool swizzle) {
  auto fn = encode_fn();
  if (!fn) return fail(DSA_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
  cuuint64_t d[4], st[3];
  cuuint32_t b[4], e[4];
  for (int i = 0; i < rank; ++i) {
    d[i] = (cuuint64_t)dims[i];
    b[i] = (cuuint32_t)box[i];
    e[i] = 1;
    if (i > 0) st[i - 1] = dims[i] > 1 ? (cuuint64_t)strides[i - 1] : (cuuint64_t)((dims[0] * size + 15) / 16 * 16);
  }
  const CUresult r = fn(m, type, (cuuint32_t)rank, const_cast<void*>(base), d, st, b, e, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(DSA_ERR_CUDA, "cuTensorMapEncodeTiled(%s) failed (%d)", what, (int)r);
  return DSA_OK;
}

}  // namespace dsa_host
