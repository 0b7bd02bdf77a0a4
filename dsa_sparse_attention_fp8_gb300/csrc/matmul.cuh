// Products of rows and weights, in one group or grouped by expert:
//   y[i, n] = sum_b xs[r, b] ws[n / 128, b] sum_{k in block b} x[r, k] w[n, k]
// with r = rows[i] or i, w and ws those of i's group; blocks of 128 along K (E4M3), or one sum without scales (16 bits).
// Gated: silu(y[i, n]) * y[i, N/2 + n].  Written rounded, or as E4M3 with a scale per 128 elements.
//
// Rows are the accumulator's lanes (M), weight rows its columns (N).  Scales are FP32 numbers, not powers of two, so no
// tensor-core instruction applies them: each block of K makes an accumulator of its own in tensor memory, which the
// epilogue warps multiply by xs * ws and add up in registers while the next block's products run.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cstdint>

#include "common.cuh"
#include "ptx_matmul.cuh"
#include "quantize.cuh"

namespace dsa {

constexpr int kMatmulMaxGroups = 1024;
constexpr int kMatmulBlock = 128;    // elements of K and weight rows that share a scale
constexpr int kMatmulThreads = 384;  // eight epilogue warps; one that loads, one that issues products, one that sets up

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
  bool gated, give_up;
};

// ---------------------------------------------------------------- tiles
// The groups as every CTA lays them out for itself: tiles of BM rows before each, its first row and its end.  A tile number
// runs over a group's row tiles first, so that CTAs that run together read the same weights.
struct Groups {
  int* first;  // [E + 1]
  int* begin;  // [E]
  int* end;    // [E]
};
struct Tile {
  int e, row, count, column;  // its group, first row, rows, first column of the result
};

// All threads; a barrier before the result is used.
template <int BM>
__device__ __forceinline__ void load_groups(const MatmulParams& p, const Groups& g) {
  for (int e = threadIdx.x; e < p.E; e += kMatmulThreads) {
    int b = 0, n = p.M;
    if (p.starts) {
      b = __ldg(p.starts + e), n = __ldg(p.starts + e + 1);
      if (b < 0 || n > p.M || n < b) {
        if (blockIdx.x == 0) raise_status(p.status, kStatusBadMetadata);
        b = n = 0;
      }
    }
    g.begin[e] = b;
    g.end[e] = n;
  }
}
// One warp.
template <int BM>
__device__ __forceinline__ void count_tiles(int E, const Groups& g) {
  const int lane = threadIdx.x & 31;
  int sum = 0;
  for (int at = 0; at < E; at += 32) {
    const int e = at + lane;
    const int c = e < E ? (int)(((int64_t)g.end[e] - g.begin[e] + BM - 1) / BM) : 0;
    int up = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, up, o);
      if (lane >= o) up += v;
    }
    if (e < E) g.first[e] = sum + up - c;
    sum += __shfl_sync(0xffffffffu, up, 31);
  }
  if (lane == 0) g.first[E] = sum;
}

// Walks the tiles of one CTA or cluster: t, t + step, ...
template <int BM, int OUT>
struct Walk {
  Groups g;
  int64_t t, step, total;
  int E, e = 0, columns;
  __device__ Walk(const MatmulParams& p, const Groups& groups, int64_t from, int64_t by)
      : g(groups), t(from), step(by), E(p.E), columns((p.width + OUT - 1) / OUT) {
    total = (int64_t)g.first[E] * columns;
  }
  __device__ bool next(Tile* tile) {
    if (t >= total) return false;
    if ((int64_t)g.first[e + 1] * columns <= t) {
      int lo = e + 1, hi = E - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if ((int64_t)g.first[mid] * columns <= t) lo = mid; else hi = mid - 1;
      }
      e = lo;
    }
    const int tiles = g.first[e + 1] - g.first[e];
    const int64_t j = t - (int64_t)g.first[e] * columns;
    const int column = tiles == 1 ? (int)j : (int)(j / tiles);
    const int m = (int)(j - (int64_t)column * tiles);
    tile->e = e;
    tile->row = g.begin[e] + m * BM;
    tile->count = min(BM, g.end[e] - tile->row);
    tile->column = column * OUT;
    t += step;
    return true;
  }
};

// ---------------------------------------------------------------- results
__device__ __forceinline__ float gate(float g, float u) { return __fdividef(g, 1.0f + __expf(-g)) * u; }

__device__ __forceinline__ uint32_t round_pair(float a, float b, bool bf16) {
  if (bf16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Four neighbouring results of a row to out.
__device__ __forceinline__ void store4(const MatmulParams& p, int64_t row, int n, const float (&y)[4], bool vec) {
  const int64_t at = row * p.out_stride + n;
  if (vec && n + 4 <= p.width) {
    if (p.out_type == 2) {
      *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at) = make_float4(y[0], y[1], y[2], y[3]);
    } else {
      const bool bf16 = p.out_type == 0;
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + at) = make_uint2(round_pair(y[0], y[1], bf16), round_pair(y[2], y[3], bf16));
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (n + i >= p.width) break;
    if (p.out_type == 2) static_cast<float*>(p.out)[at + i] = y[i];
    else if (p.out_type == 0) static_cast<__nv_bfloat16*>(p.out)[at + i] = __float2bfloat16_rn(y[i]);
    else static_cast<__half*>(p.out)[at + i] = __float2half_rn(y[i]);
  }
}

// ---------------------------------------------------------------- few rows to a group
// Tiles of BM rows and 128 results.  A cluster's CTAs share a tile's K in equal parts, each part a stream of its own from
// HBM, and join their sums through each other's shared memory in rank order.
template <bool FP8, bool GATED, int BM>
struct FewCfg {
  static constexpr int kOut = 128;               // results of a tile
  static constexpr int BN = GATED ? 256 : 128;   // its weight rows: gated 64 gates, their 64 partners, and so again
  static constexpr int kBox = GATED ? 64 : 128;  // weight rows of a load
  static constexpr int kHalf = BN / 2;           // columns of an epilogue warpgroup
  static constexpr int kK = FP8 ? 128 : 64;      // elements of K in a stage: 128 bytes
  static constexpr int kStageA = BM * 128, kStageB = BN * 128, kStage = kStageA + kStageB;
  static constexpr int kRound = GATED ? 32 : 64;     // rows joined at a time
  static constexpr int kStride = (BN + 4) * 4;       // bytes between their sums; the fifth float from the end tells a bad row
  static constexpr int kJoin = kRound * kStride;
  static constexpr int kTable = (3 * kMatmulMaxGroups + 4) * 4;
  static constexpr int kRest = kJoin + kTable + 512 + 1024;  // barriers, alignment
  static constexpr int kStages = (232448 - kRest) / kStage < 8 ? (232448 - kRest) / kStage : 8;
  static constexpr int kBuffers = 512 / BN;  // accumulators
  static constexpr int kSmem = kRest + kStages * kStage;
  static_assert(kStages >= 3 && kSmem <= 232448);
};

template <bool FP8, bool GATED, int BM>
__global__ void __launch_bounds__(kMatmulThreads, 1)
few_rows_kernel(const __grid_constant__ CUtensorMap tx, const __grid_constant__ CUtensorMap tw, const __grid_constant__ MatmulParams p) {
  using C = FewCfg<FP8, GATED, BM>;
  extern __shared__ uint8_t raw[];
  const uint32_t stages = (smem_u32(raw) + 1023u) & ~1023u;
  uint8_t* const base = raw + (stages - smem_u32(raw));
  const uint32_t join = stages + C::kStages * C::kStage;
  int* const table = reinterpret_cast<int*>(base + C::kStages * C::kStage + C::kJoin);
  const Groups groups{table, table + kMatmulMaxGroups + 1, table + 2 * kMatmulMaxGroups + 1};
  const uint32_t bars = join + C::kJoin + C::kTable;
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(base + (bars - stages) + 496);
  const uint32_t tmem_holder = bars + 500;
  const auto full = [&](int s) { return bars + 8 * s; };
  const auto empty = [&](int s) { return bars + 64 + 8 * s; };
  const auto acc_full = [&](int b) { return bars + 128 + 8 * b; };
  const auto acc_empty = [&](int b) { return bars + 160 + 8 * b; };
  const uint32_t join_full = bars + 192, join_free = bars + 200;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t S = cluster_size(), rank = cluster_rank();
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) mbar_init(full(s), 1), mbar_init(empty(s), 1);
    for (int b = 0; b < C::kBuffers; ++b) mbar_init(acc_full(b), 1), mbar_init(acc_empty(b), 8);
    mbar_init(join_full, 8 * S);
    mbar_init(join_free, 8 * S);
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tx);
    tma_prefetch_desc(&tw);
  }
  load_groups<BM>(p, groups);
  if (warp == 9) {
    tmem_alloc(tmem_holder, 512);
    tmem_relinquish();
  }
  __syncthreads();
  if (warp == 8) count_tiles<BM>(p.E, groups);
  tc_fence_before();
  if (S > 1) cluster_sync(); else __syncthreads();
  tc_fence_after();
  const uint32_t tmem = lds_u32(tmem_holder);
  const auto quit = [&] {
    *abort_flag = 1;
    raise_status(p.status, kStatusTimeout);
  };

  // this CTA's part of K, in stages
  const int blocks = (p.K + C::kK - 1) / C::kK;
  const int k0 = (int)((int64_t)blocks * rank / S), k1 = (int)((int64_t)blocks * (rank + 1) / S);
  Walk<BM, C::kOut> walk(p, groups, blockIdx.x / S, gridDim.x / S);
  Tile tile;

  if (warp < 8) {
    // ------------------------------------------------ sums and results
    regs_grow<216>();  // (2 x 216 + 72 = 3 x 168)
    const int half = warp >> 2, q = warp & 3;
    const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16) + half * C::kHalf;
    const bool vec = p.out && (reinterpret_cast<uintptr_t>(p.out) | (uintptr_t)(p.out_stride * (p.out_type == 2 ? 4 : 2))) % (p.out_type == 2 ? 16 : 8) == 0;
    const bool vec_codes = p.codes && (reinterpret_cast<uintptr_t>(p.codes) | (uintptr_t)p.width) % 4 == 0;
    int buffer = 0, turn = 0, joined = 0;
    bool on = true;
    while (on && walk.next(&tile)) {
      const int row = q * 32 + lane;
      const bool busy = q * 32 < tile.count;  // the warp has rows
      int src = 0;
      bool bad = false;
      if (row < tile.count) {
        src = p.rows ? __ldg(p.rows + tile.row + row) : tile.row + row;
        bad = src < 0 || src >= p.x_rows;
        if (bad) src = 0;
        if (bad && half == 0 && rank == 0) raise_status(p.status, kStatusBadMetadata);
      }
      uint64_t acc[C::kHalf / 2];
#pragma unroll
      for (int i = 0; i < C::kHalf / 2; ++i) acc[i] = 0;
      if (FP8) {
        const float* const xs = p.x_scales + (int64_t)src * p.kb;
        const int n0 = GATED ? tile.column + 64 * half : tile.column;
        const float* const ws = p.w_scales + ((int64_t)tile.e * p.nb + n0 / kMatmulBlock) * p.kb;
        const float* const wu = p.w_scales + ((int64_t)tile.e * p.nb + min(p.nb - 1, (p.width + n0) / kMatmulBlock)) * p.kb;
        // the scales of four blocks are loaded while the four before are summed
        float s_next[4], g_next[4], u_next[4];
        const auto ahead = [&](int k) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int at = min(k + j, k1 - 1);
            s_next[j] = __ldg(xs + at);
            g_next[j] = __ldg(ws + at);
            u_next[j] = GATED ? __ldg(wu + at) : 0.f;
          }
        };
        ahead(k0);
        for (int k = k0; k < k1 && on; k += 4) {
          float gs[4], us[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) gs[j] = s_next[j] * g_next[j], us[j] = s_next[j] * u_next[j];
          if (k + 4 < k1) ahead(k + 4);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (k + j >= k1) break;
            on = __all_sync(~0u, mbar_wait(acc_full(buffer), turn, abort_flag));
            if (!on) break;
            tc_fence_after();
            if (busy) {
              uint32_t d[2][32];
              const uint32_t from = lanes + buffer * C::BN;
              tmem_ld<32>(from, d[0]);
              tmem_ld_wait32(d[0]);
#pragma unroll
              for (int c = 0; c < C::kHalf / 32; ++c) {
                if (c + 1 < C::kHalf / 32) tmem_ld<32>(from + 32 * (c + 1), d[(c + 1) & 1]);
                const float f = GATED && c >= 2 ? us[j] : gs[j];
                const uint64_t f2 = pack2(f, f);
                const uint32_t* v = d[c & 1];
#pragma unroll
                for (int i = 0; i < 16; ++i)
                  acc[16 * c + i] = fma2(pack2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])), f2, acc[16 * c + i]);
                if (c + 1 < C::kHalf / 32) tmem_ld_wait32(d[(c + 1) & 1]);
              }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(acc_empty(buffer));
            if (++buffer == C::kBuffers) buffer = 0, turn ^= 1;
          }
        }
      } else {
        on = __all_sync(~0u, mbar_wait(acc_full(buffer), turn, abort_flag));
        if (on) {
          tc_fence_after();
          if (busy) {
#pragma unroll
            for (int c = 0; c < C::kHalf / 32; ++c) {
              uint32_t d[32];
              tmem_ld<32>(lanes + buffer * C::BN + 32 * c, d);
              tmem_ld_wait32(d);
#pragma unroll
              for (int i = 0; i < 16; ++i) acc[16 * c + i] = pack2(__uint_as_float(d[2 * i]), __uint_as_float(d[2 * i + 1]));
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(acc_empty(buffer));
          if (++buffer == C::kBuffers) buffer = 0, turn ^= 1;
        }
      }
      if (!on) break;

      // rounds of kRound rows: every CTA lays its sums out, then each warp of the cluster takes rows
      for (int r0 = 0; r0 < tile.count && on; r0 += C::kRound) {
        if (joined) on = __all_sync(~0u, mbar_wait_cluster(join_free, (joined - 1) & 1, abort_flag));  // what lies there was read
        if (!on) break;
        if (busy && q * 32 >= r0 && q * 32 < r0 + C::kRound) {
          const uint32_t to = join + (row - r0) * C::kStride;
#pragma unroll
          for (int c = 0; c < C::kHalf; c += 4) {
            const float2 lo = unpack2(acc[c / 2]), hi = unpack2(acc[c / 2 + 1]);
            const int column = GATED ? (c < 64 ? 64 * half + c : 64 + 64 * half + c) : half * C::kHalf + c;
            sts_v4(to + 4 * column, make_uint4(__float_as_uint(lo.x), __float_as_uint(lo.y), __float_as_uint(hi.x), __float_as_uint(hi.y)));
          }
          if (half == 0) sts_u32(to + 4 * C::BN, bad);
        }
        __syncwarp();
        if (lane < S) mbar_arrive_cluster(map_to(join_full, lane));
        on = __all_sync(~0u, mbar_wait_cluster(join_full, joined & 1, abort_flag));
        if (!on) break;
        const int rows = min(C::kRound, tile.count - r0);
        for (int r = (int)rank * 8 + warp; r < rows; r += 8 * S) {
          const uint32_t at = join + r * C::kStride + 16 * lane;
          float4 a = make_float4(0.f, 0.f, 0.f, 0.f), u = a;
          for (uint32_t o = 0; o < S; ++o) {
            const uint32_t there = S > 1 ? map_to(at, o) : at;
            const float4 v = ld_cluster_v4(there);
            a.x += v.x, a.y += v.y, a.z += v.z, a.w += v.w;
            if (GATED) {
              const float4 w = ld_cluster_v4(there + 512);
              u.x += w.x, u.y += w.y, u.z += w.z, u.w += w.w;
            }
          }
          float y[4] = {a.x, a.y, a.z, a.w};
          if (GATED) y[0] = gate(a.x, u.x), y[1] = gate(a.y, u.y), y[2] = gate(a.z, u.z), y[3] = gate(a.w, u.w);
          const int64_t to = (int64_t)tile.row + r0 + r;
          const int n = tile.column + 4 * lane;
          const bool no_row = lds_u32(join + r * C::kStride + 4 * C::BN) != 0;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (no_row || n + i >= p.width) y[i] = 0.f;
          if (p.out) {
            store4(p, to, n, y, vec);
            continue;
          }
          float amax = fmaxf(fmaxf(fabsf(y[0]), fabsf(y[1])), fmaxf(fabsf(y[2]), fabsf(y[3])));
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
          const float step = __fdiv_rn(amax, 448.0f), s = step == 0.f ? 1.0f : step;
          uint32_t codes = __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(y[0], s), __fdiv_rn(y[1], s)), __NV_SATFINITE, __NV_E4M3);
          codes |= (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(y[2], s), __fdiv_rn(y[3], s)), __NV_SATFINITE, __NV_E4M3) << 16;
          uint8_t* const dst = p.codes + to * p.width + n;
          if (vec_codes && n + 4 <= p.width) {
            *reinterpret_cast<uint32_t*>(dst) = codes;
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (n + i < p.width) dst[i] = (uint8_t)(codes >> (8 * i));
          }
          if (lane == 0) p.scales[to * ((p.width + 127) / 128) + tile.column / 128] = s;
        }
        __syncwarp();
        if (lane < S) mbar_arrive_cluster(map_to(join_free, lane));
        ++joined;
      }
    }
    if (!on) quit();
  } else {
    regs_shrink<72>();
    if (warp == 8) {
      // ------------------------------------------------ loads
      int s = 0, phase = 0;
      uint32_t used = 0;  // stages that were ever filled
      bool on = !p.give_up;
      if (!on) quit();
      while (on && walk.next(&tile)) {
        int4 from = make_int4(0, 0, 0, 0);
        const int boxes = p.rows ? (tile.count + 3) / 4 : (tile.count + 31) / 32;
        if (p.rows) {
          int r[4];
  #pragma unroll
          for (int i = 0; i < 4; ++i) {
            r[i] = __ldg(p.rows + tile.row + min(4 * lane + i, tile.count - 1));
            if (r[i] < 0 || r[i] >= p.x_rows) r[i] = 0;
          }
          from = make_int4(r[0], r[1], r[2], r[3]);
        }
        const uint32_t bytes = C::kStageB + boxes * (p.rows ? 512 : 4096);
        for (int k = k0; k < k1; ++k) {
          if (!__all_sync(~0u, mbar_wait(empty(s), phase ^ 1, abort_flag))) {
            on = false;
            break;
          }
          const uint32_t a = stages + s * C::kStage, b = a + C::kStageA;
          const int x = k * C::kK;
          if (lane == 0) {
            mbar_arrive_expect_tx(full(s), bytes);
  #pragma unroll
            for (int i = 0; i < C::BN / C::kBox; ++i) {
              const int n = GATED ? tile.column + 64 * (i >> 1) + (i & 1) * p.width : tile.column;
              tma_load_3d(b + i * C::kBox * 128, &tw, x, n, tile.e, full(s));
            }
          }
          __syncwarp();
          if (lane < boxes) {
            if (p.rows) tma_gather4(a + lane * 512, &tx, x, from, full(s));
            else tma_load_2d(a + lane * 4096, &tx, x, tile.row + 32 * lane, full(s));
          }
          used |= 1u << s;
          if (++s == C::kStages) s = 0, phase ^= 1;
        }
      }
      if (!on) {
        // the copies under way end before the CTA does
        quit();
        for (int i = 0; i < C::kStages; ++i)
          if (used >> i & 1) mbar_wait(full(i), (i < s ? phase : phase ^ 1), nullptr);
      }
    } else if (warp == 9) {
      // ------------------------------------------------ products
      if (lane == 0) {
        const uint32_t idesc = FP8 ? idesc_e4m3_f32(128, C::BN) : idesc_16_f32(p.x_type == 0, 128, C::BN, false);
        int s = 0, phase = 0, buffer = 0, turn = 0;
        bool on = true;
        while (on && walk.next(&tile)) {
          for (int k = k0; k < k1; ++k) {
            if (FP8 || k == k0) on = mbar_wait(acc_empty(buffer), turn ^ 1, abort_flag);
            on = on && mbar_wait(full(s), phase, abort_flag);
            if (!on) break;
            tc_fence_after();
            const uint32_t a = stages + s * C::kStage, d = tmem + buffer * C::BN;
            if (FP8) umma_f8_k128(d, sw128_desc(a), sw128_desc(a + C::kStageA), idesc, 0, 4);
            else umma_f16_k64(d, sw128_desc(a), sw128_desc(a + C::kStageA), idesc, k > k0, 4);
            umma_commit(empty(s));
            if (FP8 || k + 1 == k1) {
              umma_commit(acc_full(buffer));
              if (++buffer == C::kBuffers) buffer = 0, turn ^= 1;
            }
            if (++s == C::kStages) s = 0, phase ^= 1;
          }
        }
        if (!on) {
          quit();
          // products under way end before the CTA does: their last commit is that of the stage before
          const int last = s == 0 ? C::kStages - 1 : s - 1;
          mbar_wait(empty(last), s == 0 ? phase ^ 1 : phase, nullptr);
        }
      }
      __syncwarp();
    }
  }
  __syncwarp();
  tc_fence_before();
  if (S > 1) cluster_sync(); else __syncthreads();
  tc_fence_after();
  if (warp == 9) tmem_dealloc(tmem, 512);
}

}  // namespace dsa
