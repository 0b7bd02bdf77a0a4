// Inline PTX of the kernels around the paged caches, beside what ptx.cuh has.
// (A header of its own: the scoring kernel's committed counters are valid for
// the sources that it is built from.)
#pragma once

#include <cuda_runtime.h>
#include <cstdint>

#include "ptx.cuh"

namespace dsa {

// TMA loads of tiles of three and four dimensions.
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void* tmap, int32_t x, int32_t y,
                                            int32_t z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void* tmap, int32_t x, int32_t y,
                                            int32_t z, int32_t w, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
      : "memory");
}

// D[tmem] (+)= A[smem] * B[smem]^T over the first `steps` (at most 4) K steps of
// 16, kind::f16 (A and B of one 16-bit type), one CTA: both operands K-major
// in the 128-byte swizzle layout.  Issued by one thread, as one block of
// assembly: the descriptors of all steps, computed ahead by the compiler,
// would take registers.
__device__ __forceinline__ void umma_f16_k64(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                             uint32_t idesc, uint32_t accumulate, uint32_t steps) {
  asm volatile(
      "{\n\t.reg .pred on, acc, all;\n\t.reg .b64 a, b;\n\t"
      "setp.eq.u32 all, 0, 0;\n\tsetp.ne.u32 acc, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, acc;\n\t"
      "setp.gt.u32 on, %5, 1;\n\tadd.s64 a, %1, 2;\n\tadd.s64 b, %2, 2;\n\t"
      "@on tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, all;\n\t"
      "setp.gt.u32 on, %5, 2;\n\tadd.s64 a, %1, 4;\n\tadd.s64 b, %2, 4;\n\t"
      "@on tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, all;\n\t"
      "setp.gt.u32 on, %5, 3;\n\tadd.s64 a, %1, 6;\n\tadd.s64 b, %2, 6;\n\t"
      "@on tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, all;\n\t"
      "}" ::"r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(steps)
      : "memory");
}

// The same for 8-bit operands (kind::f8f6f4), K steps of 32.
__device__ __forceinline__ void umma_f8_k128(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                             uint32_t idesc, uint32_t accumulate, uint32_t steps) {
  asm volatile(
      "{\n\t.reg .pred on, acc, all;\n\t.reg .b64 a, b;\n\t"
      "setp.eq.u32 all, 0, 0;\n\tsetp.ne.u32 acc, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, acc;\n\t"
      "setp.gt.u32 on, %5, 1;\n\tadd.s64 a, %1, 2;\n\tadd.s64 b, %2, 2;\n\t"
      "@on tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, all;\n\t"
      "setp.gt.u32 on, %5, 2;\n\tadd.s64 a, %1, 4;\n\tadd.s64 b, %2, 4;\n\t"
      "@on tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, all;\n\t"
      "setp.gt.u32 on, %5, 3;\n\tadd.s64 a, %1, 6;\n\tadd.s64 b, %2, 6;\n\t"
      "@on tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, all;\n\t"
      "}" ::"r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(steps)
      : "memory");
}

// D[tmem] (+)= A[tmem] * B[smem] over 8 K steps of 16 (A's first 64 elements in
// columns 0 to 31, the others in 64 to 95), B MN-major in the 128-byte swizzle
// layout.
__device__ __forceinline__ void umma_f16_ta_k128(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc,
                                                 uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred acc, all;\n\t.reg .b64 b;\n\t.reg .b32 a;\n\t"
      "setp.eq.u32 all, 0, 0;\n\t"
      "setp.ne.u32 acc, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, acc;\n\t"
      "add.s32 a, %1, 8;\n\tadd.s64 b, %2, 128;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, all;\n\t"
      "add.s32 a, %1, 16;\n\tadd.s64 b, %2, 256;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, all;\n\t"
      "add.s32 a, %1, 24;\n\tadd.s64 b, %2, 384;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, all;\n\t"
      "add.s32 a, %1, 64;\n\tadd.s64 b, %2, 512;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, all;\n\t"
      "add.s32 a, %1, 72;\n\tadd.s64 b, %2, 640;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, all;\n\t"
      "add.s32 a, %1, 80;\n\tadd.s64 b, %2, 768;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, all;\n\t"
      "add.s32 a, %1, 88;\n\tadd.s64 b, %2, 896;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, all;\n\t"
      "}" ::"r"(d_tmem), "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Instruction descriptor of 16-bit operands with FP32 accumulators, for either
// type (BF16, or FP16 whose format code is 0).
__device__ __forceinline__ uint32_t idesc_16_f32(bool bf16, uint32_t M, uint32_t N, bool b_mn_major) {
  const uint32_t d = idesc_bf16_f32(M, N, b_mn_major);
  return bf16 ? d : d & ~((1u << 7) | (1u << 10));
}

// A wait for tensor-memory loads, bound to the registers of one: their uses
// cannot be moved ahead of the wait, whatever other loads are in flight.
__device__ __forceinline__ void tmem_ld_wait16(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]));
}
__device__ __forceinline__ void tmem_ld_wait32(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31]));
}

// Moves registers between the warpgroups of a block; every warp of the calling
// warpgroup executes it.  The block's warpgroups together never hold more
// than the block was launched with.
template <int N>
__device__ __forceinline__ void regs_grow() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_shrink() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// 2^x by the hardware's approximation (2 ulp), subnormal results flushed.
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 1 / x to within a unit in the last place; subnormal x and results are zeros.
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Packed pairs of FP32 (one instruction for two, each rounded as usual).
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
  return v;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

}  // namespace dsa
