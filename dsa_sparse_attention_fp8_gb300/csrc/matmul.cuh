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
  int x_type, out_type, most_tiles, box;            // row tiles whose numbers fit, rows of a load
  int load_stages;  // after so many stages loading warps give up (tests of the unwinding); -1: never
  bool gated;
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
      b = ld_early(p.starts + e), n = ld_early(p.starts + e + 1);
      if (b < 0 || n > p.M || n < b) {
        if (blockIdx.x == 0) raise_status(p.status, kStatusBadMetadata);
        b = n = 0;
      }
    }
    g.begin[e] = b;
    g.end[e] = n;
  }
}
// One warp.  Groups that overlap, which only starts that go back make, may together have many times the rows that there are:
// all their tiles count, up to the `most` whose numbers fit 31 bits.
template <int BM>
__device__ __forceinline__ void count_tiles(int E, int most, const Groups& g) {
  const int lane = threadIdx.x & 31;
  int64_t sum = 0;
  for (int at = 0; at < E; at += 32) {
    const int e = at + lane;
    const int c = e < E ? (int)(((int64_t)g.end[e] - g.begin[e] + BM - 1) / BM) : 0;
    int64_t up = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(0xffffffffu, up, o);
      if (lane >= o) up += v;
    }
    if (e < E) g.first[e] = (int)min((int64_t)most, sum + up - c);
    sum += __shfl_sync(0xffffffffu, up, 31);
  }
  if (lane == 0) g.first[E] = (int)min((int64_t)most, sum);
}

// The t-th tile, in kOut columns of the result and BM rows; false past the last.
template <int BM, int OUT>
__device__ __forceinline__ bool find_tile(const MatmulParams& p, const Groups& g, int t, Tile* tile) {
  const int columns = (p.width + OUT - 1) / OUT;
  if (t >= g.first[p.E] * columns) return false;
  int e = 0, hi = p.E - 1;
  while (e < hi) {
    const int mid = (e + hi + 1) >> 1;
    if (g.first[mid] * columns <= t) e = mid; else hi = mid - 1;
  }
  const int tiles = g.first[e + 1] - g.first[e], j = t - g.first[e] * columns;
  const int column = j / tiles;
  tile->e = e;
  tile->row = g.begin[e] + (j - column * tiles) * BM;
  tile->count = min(BM, g.end[e] - tile->row);
  tile->column = column * OUT;
  return true;
}

// Adds a block's accumulator, COLS columns of this warp's lanes, to acc: the first half times f, the rest times u.
template <int COLS>
__device__ __forceinline__ void add_block(uint32_t from, uint64_t (&acc)[COLS / 2], float f, float u) {
#pragma unroll
  for (int c = 0; c < COLS / 64; ++c) {
    uint32_t d[64];
    tmem_ld<64>(from + 64 * c, d);
    tmem_ld_wait();
    const uint64_t f0 = COLS == 64 || c == 0 ? pack2(f, f) : pack2(u, u);
#pragma unroll
    for (int i = 0; i < 32; ++i) fma2_here(acc[32 * c + i], d[2 * i], d[2 * i + 1], f0);
  }
}
template <int COLS>
__device__ __forceinline__ void take_block(uint32_t from, uint64_t (&acc)[COLS / 2]) {
#pragma unroll
  for (int c = 0; c < COLS / 32; ++c) {
    uint32_t d[32];
    tmem_ld<32>(from + 32 * c, d);
    tmem_ld_wait32(d);
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[16 * c + i] = pack2(__uint_as_float(d[2 * i]), __uint_as_float(d[2 * i + 1]));
  }
}

// ---------------------------------------------------------------- unwinding
// Every wait is bounded.  A role whose wait runs out raises the flag of each CTA that works on the tile and leaves; so do the
// others when they see it.  Copies and products under way then end before the CTA does: the loading and the product warp
// leave word of where they stopped, which is read once every role has left.  A barrier that copies alone arrive at tells
// of their end (gathered rows, whose warps wait for their own copies, have barriers of their own).  Roles give up in one place,
// behind all of them: four copies of that code took 0.4 us more of each call with 64 gated rows.
__device__ __forceinline__ void give_up(const MatmulParams& p, uint32_t abort_flag, uint32_t ctas) {
  for (uint32_t r = 0; r < ctas; ++r) st_cluster_u32(map_to(abort_flag, r), 1);
  raise_status(p.status, kStatusTimeout);
}
struct Stopped {
  int s, phase;   // the stage that would have come next, and its pass
  uint32_t used;  // stages that were ever filled
};
__device__ __forceinline__ void tell_stop(uint32_t at, int s, int phase, uint32_t used) {
  if ((threadIdx.x & 31) == 0) sts_u32(at, (uint32_t)s | (uint32_t)phase << 7 | used << 8);
}
__device__ __forceinline__ Stopped where_stopped(uint32_t at) {
  const uint32_t v = lds_u32(at);
  return {(int)(v & 127), (int)(v >> 7 & 1), v >> 8};
}
__device__ __forceinline__ void end_loads(const Stopped& l, uint32_t full, int stages) {
  for (int i = 0; i < stages; ++i)
    if (l.used >> i & 1) mbar_wait(full + 8 * i, i < l.s ? l.phase : l.phase ^ 1, nullptr);
}
// (the last products' commit is that of the stage before; of none the barrier is as it was made)
__device__ __forceinline__ void end_products(const Stopped& m, uint32_t empty, int stages) {
  mbar_wait(empty + 8 * (m.s == 0 ? stages - 1 : m.s - 1), m.s == 0 ? m.phase ^ 1 : m.phase, nullptr);
}
// How many stages a loading warp may fill, -1 for all of them; CTAs of odd rank one more or less, so that a pair's stop apart.
__device__ __forceinline__ int stages_to_fill(const MatmulParams& p, uint32_t rank) {
  return p.load_stages > 0 ? p.load_stages ^ (int)(rank & 1) : p.load_stages;
}

// ---------------------------------------------------------------- gathered rows
// Two warps copy a tile's rows x[rows[i]] into the stages, 16 bytes a lane, in the layout that the tensor core reads (and
// TMA writes): 128-byte rows whose 16-byte pieces change places within eight rows.  Every lane's copies arrive at the
// stage's barrier by themselves; whoever waits there fences them for the tensor core (a fence in these warps would wait for
// all their copies, also those of later stages: experts of a chunk took 4773 us by it).  The tensor-copy unit gathers too,
// four rows an instruction, but at 19 cycles a row (4041 us; 1506 from rows that lie in order).
constexpr int kGatherLanes = 64;
template <int STAGES, int STAGE, int BM, int OUT>
__device__ __forceinline__ bool gather_rows(const MatmulParams& p, const Groups& groups, int t, int step, int offset, int most, int size,
                                            int k0, int k1, uint32_t stages, int g, const volatile int* abort_flag,
                                            uint32_t empty, uint32_t landed) {
  const int lane = threadIdx.x & 31, piece = lane & 7;
  const uint32_t row_pieces = (uint32_t)(p.x_stride * size / 16);
  const int end = p.K * size;  // of a row's bytes
  int s = 0, phase = 0;
  Tile tile;
  bool on = true;
  for (; on && find_tile<BM, OUT>(p, groups, t, &tile); t += step) {
    const int mine = max(0, min(most, tile.count - offset));
    // this lane's rows are 8 i + 4 g + lane / 8
    const int own = 4 * g + (lane >> 3);
    uint32_t from[16];  // and start these many pieces into x
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int r = 8 * i + own < mine ? ld_early(p.rows + tile.row + offset + 8 * i + own) : 0;
      from[i] = r < 0 || r >= p.x_rows ? 0 : (uint32_t)r * row_pieces;
    }
    const uint8_t* const x = static_cast<const uint8_t*>(p.x) + piece * 16;
    for (int k = k0; k < k1; ++k) {
      on = __all_sync(~0u, mbar_wait(empty + 8 * s, phase ^ 1, abort_flag));
      if (!on) break;
      const int at = k * 128;
      const uint32_t bytes = (uint32_t)min(16, max(0, end - at - piece * 16));
      const uint32_t to = stages + s * STAGE + own * 128 + ((piece ^ own) * 16);
      const uint8_t* const src = bytes ? x + at : x;
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (8 * i + own < mine) copy16_async(to + i * 1024, src + (uint64_t)from[i] * 16, bytes);
      copies_arrive(landed + 8 * s);
      if (++s == STAGES) s = 0, phase ^= 1;
    }
  }
  copies_wait_all();
  return on;
}

// ---------------------------------------------------------------- results
// silu(g) u = g / (1 + e) u, or g e / (1 + e) u of a negative g, with e = exp(-|g|) <= 1: nothing overflows, so that small
// results are right down to where e is subnormal (g below -87.3).  e is off by a unit in the last place, the quotient by two,
// the sum and the products by half of one each: five units in all, whatever g.
__device__ __forceinline__ float gate(float g, float u) {
  const float e = expf(-fabsf(g));
  return __fdividef(g < 0.f ? g * e : g, 1.0f + e) * u;
}

__device__ __forceinline__ uint32_t round_pair(float a, float b, bool bf16) {
  if (bf16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ void store_element(void* p, int64_t at, int type, float v) {
  if (type == 0) static_cast<__nv_bfloat16*>(p)[at] = __float2bfloat16_rn(v);
  else if (type == 1) static_cast<__half*>(p)[at] = __float2half_rn(v);
  else static_cast<float*>(p)[at] = v;
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
    store_element(p.out, at + i, p.out_type, y[i]);
  }
}

// ---------------------------------------------------------------- few rows to a group
// Tiles of BM rows and 128 results (WIDE: 256), a CTA or a cluster to a tile, one after the other.  A cluster's CTAs have equal
// parts of K, and join their sums through each other's shared memory in rank order.
//
// Bound, of one tile, by what one SM draws from L2, some 100 GB/s, and so by how many SMs share the weights (a tile of 64 rows,
// 128 weight rows and 7168 elements of K, already in L2: 21.0 us by one CTA, 9.4 by four, 7.7 by eight).  How many clusters run
// at once decides where there are more tiles: 15 of eight or seven CTAs, 23 of six, 28 of five, 36 of four as one device
// tells (64 rows, K 7168, gated N 4096, 16 tiles, from L2: 19.2 us by eight, 12.7 by six, 13.0 by four).  From HBM that
// takes 14.6 us, of which launch and set-up are 4, the stream of a sixth of K 4 and the join of 64 rows 4.  Bound, of many
// tiles, by HBM: 64 groups of eight rows with such weights, 1.76 GB in 275 to 281 us, 93 to 95 % of the copy rate.
// A stage holds BM rows though the instruction reads 128: those past BM are weights, in lanes that nobody reads.
template <bool FP8, bool GATED, bool WIDE, int BM, int ROUND>
struct FewCfg {
  static_assert(!(GATED && WIDE));
  static constexpr int kOut = WIDE ? 256 : 128;         // results of a tile
  static constexpr int BN = GATED || WIDE ? 256 : 128;  // its weight rows: gated 64 gates, their 64 partners, and so again
  static constexpr int kBox = GATED ? 64 : 128;         // weight rows of a load
  static constexpr int kHalf = BN / 2;                  // columns of an epilogue warpgroup
  static constexpr int kK = FP8 ? 128 : 64;             // elements of K in a stage: 128 bytes
  static constexpr int kStageA = BM * 128, kStageB = BN * 128, kStage = kStageA + kStageB;
  static constexpr int kRound = ROUND;                  // rows joined at a time
  static constexpr int kStride = (BN + 4) * 4;          // bytes between their sums; the float behind them tells a bad row
  static constexpr int kJoin = kRound * kStride;
  static constexpr int kTable = (3 * kMatmulMaxGroups + 4) * 4;
  static constexpr int kRest = kJoin + kTable + 512 + 1024;  // barriers, alignment
  static constexpr int kStages = (232448 - kRest) / kStage < 8 ? (232448 - kRest) / kStage : 8;
  static constexpr int kBuffers = 512 / BN;  // accumulators
  static constexpr int kSmem = kRest + kStages * kStage;
  static_assert(kStages >= 3 && kSmem <= 232448);
};

template <bool FP8, bool GATED, bool WIDE, int BM, int ROUND>
__global__ void __launch_bounds__(kMatmulThreads, 1)
few_rows_kernel(const __grid_constant__ CUtensorMap tx, const __grid_constant__ CUtensorMap tw, const __grid_constant__ MatmulParams p) {
  using C = FewCfg<FP8, GATED, WIDE, BM, ROUND>;
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
  const auto landed = [&](int s) { return bars + 208 + 8 * s; };  // gathered rows
  const uint32_t loads_stopped = bars + 484, products_stopped = bars + 488;

  const int warp = __shfl_sync(~0u, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t S = cluster_size(), rank = cluster_rank();
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) mbar_init(full(s), 1), mbar_init(empty(s), 1);
    for (int s = 0; p.rows && s < C::kStages; ++s) mbar_init(landed(s), kGatherLanes);
    for (int b = 0; b < C::kBuffers; ++b) mbar_init(acc_full(b), 1), mbar_init(acc_empty(b), 8);
    mbar_init(join_full, 8 * S);
    mbar_init(join_free, 8 * S);
    *abort_flag = 0;
    fence_barrier_init();
    if (!p.rows) tma_prefetch_desc(&tx);
    tma_prefetch_desc(&tw);
  }
  if (warp == 9) {
    tmem_alloc(tmem_holder, 512);
    tmem_relinquish();
  }
  pdl_launch_dependents();
  pdl_wait();
  load_groups<BM>(p, groups);
  __syncthreads();
  if (warp == 8) count_tiles<BM>(p.E, p.most_tiles, groups);
  tc_fence_before();
  if (S > 1) cluster_sync(); else __syncthreads();
  tc_fence_after();
  const uint32_t tmem = lds_u32(tmem_holder);
  bool on = true;  // this warp's waits have not run out

  // this CTA's part of K, in stages
  const int blocks = (p.K + C::kK - 1) / C::kK;
  const int k0 = (int)((int64_t)blocks * rank / S), k1 = (int)((int64_t)blocks * (rank + 1) / S);
  const int step = gridDim.x / S;
  Tile tile;

  if (warp < 8) {
    // ------------------------------------------------ sums and results
    regs_grow<216>();  // (2 x 216 + 72 = 3 x 168)
    const int half = warp >> 2, q = warp & 3;
    const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16) + half * C::kHalf;
    const bool vec = p.out && (reinterpret_cast<uintptr_t>(p.out) | (uintptr_t)(p.out_stride * (p.out_type == 2 ? 4 : 2))) % (p.out_type == 2 ? 16 : 8) == 0;
    const bool vec_codes = p.codes && (reinterpret_cast<uintptr_t>(p.codes) | (uintptr_t)p.width) % 4 == 0;
    int buffer = 0, turn = 0, joined = 0;
    // A tile's rows and first scales are asked for a tile ahead: where it is and this lane's row of x before the products of the
    // tile before are summed, the scales before its results are written (experts of a batch of 64, 290 us without it, 279.5).
    Tile ahead;
    const auto row_of = [&](const Tile& of) {
      const int row = q * 32 + lane;
      return row >= of.count ? 0 : p.rows ? ld_early(p.rows + of.row + row) : of.row + row;
    };
    const auto scales_of = [&](const Tile& of, int src, const float** xs, const float** ws, const float** wu) {
      const int n0 = GATED ? of.column + 64 * half : WIDE ? of.column + 128 * half : of.column;
      *xs = p.x_scales + (int64_t)(src < 0 || src >= p.x_rows ? 0 : src) * p.kb;
      *ws = p.w_scales + ((int64_t)of.e * p.nb + min(p.nb - 1, n0 / kMatmulBlock)) * p.kb;
      *wu = p.w_scales + ((int64_t)of.e * p.nb + min(p.nb - 1, (p.width + n0) / kMatmulBlock)) * p.kb;
    };
    float s_next = 0.f, g_next = 0.f, u_next = 0.f;
    const auto first_scales = [&](const Tile& of, int src) {
      const float *xs, *ws, *wu;
      scales_of(of, src, &xs, &ws, &wu);
      s_next = ld_early(xs + k0), g_next = ld_early(ws + k0), u_next = GATED ? ld_early(wu + k0) : 0.f;
    };
    int t = blockIdx.x / S;
    bool more = find_tile<BM, C::kOut>(p, groups, t, &ahead);
    int src_ahead = more ? row_of(ahead) : 0;
    if (FP8 && more) first_scales(ahead, src_ahead);
    while (on && more) {
      tile = ahead;
      const int row = q * 32 + lane, src = src_ahead;
      t += step;
      more = find_tile<BM, C::kOut>(p, groups, t, &ahead);
      if (more) src_ahead = row_of(ahead);
      const bool busy = q * 32 < tile.count;  // the warp has rows
      const bool bad = row < tile.count && (src < 0 || src >= p.x_rows);
      if (bad && half == 0 && rank == 0) raise_status(p.status, kStatusBadMetadata);
      uint64_t acc[C::kHalf / 2];
#pragma unroll
      for (int i = 0; i < C::kHalf / 2; ++i) acc[i] = 0;
      if (FP8) {
        const float *xs, *ws, *wu;
        scales_of(tile, src, &xs, &ws, &wu);
        // (a block's scales are loaded while the block before is summed)
        for (int k = k0; k < k1; ++k) {
          const float f = s_next * g_next, u = GATED ? s_next * u_next : f;
          const int at = min(k + 1, k1 - 1);
          s_next = ld_early(xs + at), g_next = ld_early(ws + at);
          if (GATED) u_next = ld_early(wu + at);
          on = __all_sync(~0u, mbar_wait(acc_full(buffer), turn, abort_flag));
          if (!on) break;
          tc_fence_after();
          if (busy) add_block<C::kHalf>(lanes + buffer * C::BN, acc, f, u);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(acc_empty(buffer));
          if (++buffer == C::kBuffers) buffer = 0, turn ^= 1;
        }
      } else {
        on = __all_sync(~0u, mbar_wait(acc_full(buffer), turn, abort_flag));
        if (on) {
          tc_fence_after();
          if (busy) take_block<C::kHalf>(lanes + buffer * C::BN, acc);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(acc_empty(buffer));
          if (++buffer == C::kBuffers) buffer = 0, turn ^= 1;
        }
      }
      if (!on) break;
      if (FP8 && more) first_scales(ahead, src_ahead);

      // rounds of kRound rows: every CTA lays its sums out, then each warp of the cluster takes rows
      for (int r0 = 0; r0 < tile.count && on; r0 += C::kRound) {
        const bool again = more || r0 + C::kRound < tile.count;  // another round follows, in every CTA of the cluster
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
        // a row's 128 results, four to a lane, from its sums (upper: those of what they gate, or the next 128 results)
        const auto finish = [&](int r, float4 a, float4 u) {
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
            if (WIDE) {
              float z[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (no_row) z[i] = 0.f;
              store4(p, to, n + 128, z, vec);
            }
            return;
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
        };
        if (S == 1) {
          // (four rows are read before the first is finished)
          for (int r = warp; r < rows; r += 32) {
            float4 a[4], u[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint32_t at = join + min(r + 8 * j, C::kRound - 1) * C::kStride + 16 * lane;
              const uint4 v = lds_v4(at), w = C::BN == 256 ? lds_v4(at + 512) : make_uint4(0, 0, 0, 0);
              a[j] = make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w));
              u[j] = make_float4(__uint_as_float(w.x), __uint_as_float(w.y), __uint_as_float(w.z), __uint_as_float(w.w));
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (r + 8 * j < rows) finish(r + 8 * j, a[j], u[j]);
          }
        } else {
          for (int r = (int)rank * 8 + warp; r < rows; r += 8 * S) {
            const uint32_t at = join + r * C::kStride + 16 * lane;
            float4 part[8], upper[8];  // (all parts are asked for before the first is added)
#pragma unroll
            for (uint32_t o = 0; o < 8; ++o) {
              part[o] = upper[o] = make_float4(0.f, 0.f, 0.f, 0.f);
              if (o < S) {
                const uint32_t there = map_to(at, o);
                part[o] = ld_cluster_v4(there);
                if (C::BN == 256) upper[o] = ld_cluster_v4(there + 512);
              }
            }
            float4 a = part[0], u = upper[0];
#pragma unroll
            for (uint32_t o = 1; o < 8; ++o) {
              a.x += part[o].x, a.y += part[o].y, a.z += part[o].z, a.w += part[o].w;
              u.x += upper[o].x, u.y += upper[o].y, u.z += upper[o].z, u.w += upper[o].w;
            }
            finish(r, a, u);
          }
        }
        __syncwarp();
        // (given back with the cluster's scope, since other CTAs' sums were read; after the last round nobody waits)
        if (again && lane < S) S > 1 ? mbar_arrive_cluster(map_to(join_free, lane)) : mbar_arrive(join_free);
        ++joined;
      }
    }
  } else {
    regs_shrink<72>();
    if (warp == 8) {
      // ------------------------------------------------ loads
      int s = 0, phase = 0, left = stages_to_fill(p, rank);
      uint32_t used = 0;
      for (int t = blockIdx.x / S; on && find_tile<BM, C::kOut>(p, groups, t, &tile); t += step) {
        const int boxes = p.rows ? 0 : (tile.count + p.box - 1) / p.box;
        const uint32_t bytes = C::kStageB + boxes * p.box * 128;
        for (int k = k0; k < k1; ++k) {
          if (left == 0 || !__all_sync(~0u, mbar_wait(empty(s), phase ^ 1, abort_flag))) {
            on = false;
            break;
          }
          left -= left > 0;
          const uint32_t a = stages + s * C::kStage, b = a + C::kStageA;
          const int x = k * C::kK;
          if (elect_one()) {
            mbar_arrive_expect_tx(full(s), bytes);
#pragma unroll
            for (int i = 0; i < C::BN / C::kBox; ++i) {
              const int n = GATED ? tile.column + 64 * (i >> 1) + (i & 1) * p.width : tile.column + 128 * i;
              tma_load_3d(b + i * C::kBox * 128, &tw, x, n, tile.e, full(s));
            }
            for (int i = 0; i < boxes; ++i) tma_load_2d(a + i * p.box * 128, &tx, x, tile.row + p.box * i, full(s));
          }
          __syncwarp();
          used |= 1u << s;
          if (++s == C::kStages) s = 0, phase ^= 1;
        }
      }
      tell_stop(loads_stopped, s, phase, used);
    } else if (warp == 9) {
      // ------------------------------------------------ products
      const uint32_t idesc = FP8 ? idesc_e4m3_f32(128, C::BN) : idesc_16_f32(p.x_type == 0, 128, C::BN, false);
      int s = 0, phase = 0, buffer = 0, turn = 0;
      for (int t = blockIdx.x / S; on && find_tile<BM, C::kOut>(p, groups, t, &tile); t += step) {
        for (int k = k0; k < k1; ++k) {
          if (FP8 || k == k0) on = __all_sync(~0u, mbar_wait(acc_empty(buffer), turn ^ 1, abort_flag));
          on = on && __all_sync(~0u, mbar_wait(full(s), phase, abort_flag));
          if (on && p.rows) on = __all_sync(~0u, mbar_wait(landed(s), phase, abort_flag));
          if (!on) break;
          if (p.rows) fence_proxy_async_smem();
          tc_fence_after();
          const uint32_t a = stages + s * C::kStage, d = tmem + buffer * C::BN;
          if (elect_one()) {
            if (FP8) umma_f8_k128_all(d, sw128_desc(a), sw128_desc(a + C::kStageA), idesc, 0);
            else umma_f16_k64_all(d, sw128_desc(a), sw128_desc(a + C::kStageA), idesc, k > k0);
            umma_commit(empty(s));
            if (FP8 || k + 1 == k1) umma_commit(acc_full(buffer));
          }
          __syncwarp();
          if (FP8 || k + 1 == k1) {
            if (++buffer == C::kBuffers) buffer = 0, turn ^= 1;
          }
          if (++s == C::kStages) s = 0, phase ^= 1;
        }
      }
      tell_stop(products_stopped, s, phase, 0);
    } else if (p.rows) {
      // ------------------------------------------------ gathered rows
      const int g = warp - 10;
      on = gather_rows<C::kStages, C::kStage, BM, C::kOut>(p, groups, blockIdx.x / S, step, 0, BM, FP8 ? 1 : 2, k0, k1, stages, g, abort_flag,
                                                           empty(0), landed(0));
    }
  }
  if (!on) give_up(p, bars + 496, S);
  __syncwarp();
  tc_fence_before();
  if (S > 1) cluster_sync(); else __syncthreads();
  tc_fence_after();
  if (*abort_flag) {
    if (warp == 8) end_loads(where_stopped(loads_stopped), full(0), C::kStages);
    if (warp == 9) end_products(where_stopped(products_stopped), empty(0), C::kStages);
    __syncwarp();
  }
  if (warp == 9) tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------- many rows to a group
// Tiles of 256 rows and 256 weight rows, each shared by a pair of CTAs (cta_group::2): a CTA loads half of the rows and half
// of the weights, and has half of the rows' sums.
//
// 8192 rows, K = N = 7168: 317 us, 2.7 PFLOP/s, 69 % of twice the measured BF16 rate (16 bits: 1.6 PFLOP/s, 82 % of it).  Two
// things bound it about alike.  The way from L2: a pair takes 64 KB for a block of K, and with a quarter of the products, and
// no sums, the same loads take 242 us.  And the hand-over of an accumulator, of which tensor memory holds two (products,
// the sums' reads of 256 columns, and back): without the sums 260 us.  Halves of an accumulator handed over
// one by one, products of 128 weight rows each, read the rows twice from shared memory: 447 us.  The sums need 128 registers
// a thread and a load's 64; where other values live across the loop the compiler copies each loaded register (one more load
// in flight 565 us, scales four blocks at a time 366, a tile ahead as for few rows 353, a loop given 224 registers 337).
template <bool FP8, bool GATED>
struct ManyCfg {
  static constexpr int BM = 256, BN = 256, kOut = GATED ? 128 : 256;
  static constexpr int kBox = GATED ? 64 : 128;  // weight rows of a load
  static constexpr int kK = FP8 ? 128 : 64;      // elements of K in a stage: 128 bytes
  static constexpr int kStageA = 128 * 128, kStageB = 128 * 128, kStage = kStageA + kStageB;
  static constexpr int kRow = 80;                // bytes of a row's staged piece, 64, its largest value, and room against bank conflicts
  static constexpr int kPieces = 8 * 32 * kRow;
  static constexpr int kTable = (3 * kMatmulMaxGroups + 4) * 4;
  static constexpr int kRest = kPieces + kTable + 512 + 1024;  // barriers, alignment
  static constexpr int kStages = (232448 - kRest) / kStage;
  static constexpr int kSmem = kRest + kStages * kStage;
  static_assert(kStages >= 6 && kStages <= 8);
};

// 64 bytes of each of a warp's 32 rows, a row to a lane, out by way of shared memory so that neighbouring lanes write a row's
// piece: `rows` rows at `to`, `stride` bytes apart, of which the first `bytes` are wanted.  VEC: both multiples of 16, four
// lanes a row; otherwise elements of SIZE bytes.
template <bool VEC, int SIZE>
__device__ __forceinline__ void store_piece(uint32_t stage, uint8_t* to, int64_t stride, int rows, int bytes, const uint32_t* v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < 4; ++i) sts_v4(stage + lane * 80 + 16 * i, make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]));
  __syncwarp();
  if constexpr (VEC) {
    const int at = (lane & 3) * 16;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 8 * i + (lane >> 2);
      const uint4 w = lds_v4(stage + r * 80 + at);
      if (r < rows && at < bytes) *reinterpret_cast<uint4*>(to + r * stride + at) = w;
    }
  } else {
    const int at = (lane & 15) * 4;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int r = 2 * i + (lane >> 4);
      const uint32_t w = lds_u32(stage + r * 80 + at);
      if (r >= rows) continue;
      uint8_t* const dst = to + r * stride + at;
#pragma unroll
      for (int j = 0; j < 4 / SIZE; ++j) {
        if (at + j * SIZE >= bytes) break;
        if constexpr (SIZE == 4) *reinterpret_cast<uint32_t*>(dst) = w;
        else if constexpr (SIZE == 2) *reinterpret_cast<uint16_t*>(dst + 2 * j) = (uint16_t)(w >> (16 * j));
        else dst[j] = (uint8_t)(w >> (8 * j));
      }
    }
  }
  __syncwarp();
}

template <bool FP8, bool GATED>
__global__ void __launch_bounds__(kMatmulThreads, 1)
many_rows_kernel(const __grid_constant__ CUtensorMap tx, const __grid_constant__ CUtensorMap tw, const __grid_constant__ MatmulParams p) {
  using C = ManyCfg<FP8, GATED>;
  extern __shared__ uint8_t raw[];
  const uint32_t stages = (smem_u32(raw) + 1023u) & ~1023u;
  uint8_t* const base = raw + (stages - smem_u32(raw));
  const uint32_t pieces = stages + C::kStages * C::kStage;
  int* const table = reinterpret_cast<int*>(base + C::kStages * C::kStage + C::kPieces);
  const Groups groups{table, table + kMatmulMaxGroups + 1, table + 2 * kMatmulMaxGroups + 1};
  const uint32_t bars = pieces + C::kPieces + C::kTable;
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(base + (bars - stages) + 496);
  const uint32_t tmem_holder = bars + 500;
  const auto full = [&](int s) { return bars + 8 * s; };    // (the first CTA's are used)
  const auto empty = [&](int s) { return bars + 64 + 8 * s; };
  const auto acc_full = [&](int b) { return bars + 128 + 8 * b; };
  const auto acc_empty = [&](int b) { return bars + 144 + 8 * b; };  // (the first CTA's)
  const auto landed = [&](int s) { return bars + 200 + 8 * s; };     // each CTA's gathered rows, in the first's the second's too
  const auto both = [&](int q) { return bars + 160 + 8 * q; };       // a row's two warps
  const uint32_t loads_stopped = bars + 484, products_stopped = bars + 488;
  const uint32_t fills = bars + 464;  // this CTA's: how many, and of the last 32 whether the second CTA had rows; then the other's

  const int warp = __shfl_sync(~0u, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  cluster_arrive();
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) mbar_init(full(s), 1), mbar_init(empty(s), 1);
    for (int s = 0; p.rows && s < C::kStages; ++s) mbar_init(landed(s), rank == 0 ? kGatherLanes + 1 : kGatherLanes);
    for (int b = 0; b < 2; ++b) mbar_init(acc_full(b), 1), mbar_init(acc_empty(b), 16);
    for (int q = 0; q < 4; ++q) mbar_init(both(q), 2);
    *abort_flag = 0;
    fence_barrier_init();
    if (!p.rows) tma_prefetch_desc(&tx);
    tma_prefetch_desc(&tw);
  }
  __syncwarp();
  cluster_wait();  // (tensor memory of a pair is asked for by both)
  if (warp == 9) {
    tmem_alloc_pair(tmem_holder, 512);
    tmem_relinquish_pair();
  }
  pdl_launch_dependents();
  pdl_wait();
  load_groups<C::BM>(p, groups);
  __syncthreads();
  if (warp == 8) count_tiles<C::BM>(p.E, p.most_tiles, groups);
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = lds_u32(tmem_holder);
  bool on = true;  // this warp's waits have not run out
  const int blocks = (p.K + C::kK - 1) / C::kK;
  const int step = gridDim.x / 2;
  Tile tile;

  if (warp < 8) {
    // ------------------------------------------------ sums and results
    regs_grow<216>();  // (2 x 216 + 72 = 3 x 168)
    const int half = warp >> 2, q = warp & 3;
    const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16) + half * 128;
    const uint32_t stage = pieces + warp * 32 * C::kRow;
    const int size = p.out_type == 2 ? 4 : 2;
    const bool vec = p.out ? (reinterpret_cast<uintptr_t>(p.out) | (uintptr_t)(p.out_stride * size)) % 16 == 0
                           : (reinterpret_cast<uintptr_t>(p.codes) | (uintptr_t)p.width) % 16 == 0;
    int buffer = 0, turn = 0, tiles = 0;
    for (int t = blockIdx.x / 2; on && find_tile<C::BM, C::kOut>(p, groups, t, &tile); t += step) {
      const int64_t row0 = tile.row + 128 * (int)rank + q * 32;   // the warp's first row
      const int rows = tile.count - 128 * (int)rank - q * 32;      // and how many it has
      int src = 0;
      bool bad = false;
      if (lane < rows) {
        src = p.rows ? ld_early(p.rows + row0 + lane) : (int)row0 + lane;
        bad = src < 0 || src >= p.x_rows;
        if (bad) src = 0;
        if (bad && half == 0) raise_status(p.status, kStatusBadMetadata);
      }
      uint64_t acc[64];
#pragma unroll
      for (int i = 0; i < 64; ++i) acc[i] = 0;
      if (FP8) {
        const float* const xs = p.x_scales + (int64_t)src * p.kb;
        const int n0 = GATED ? tile.column + 64 * half : tile.column + 128 * half;
        const float* const ws = p.w_scales + ((int64_t)tile.e * p.nb + min(p.nb - 1, n0 / kMatmulBlock)) * p.kb;
        const float* const wu = p.w_scales + ((int64_t)tile.e * p.nb + min(p.nb - 1, (p.width + n0) / kMatmulBlock)) * p.kb;
        // (a block's scales are loaded while the block before is summed)
        float s_next = ld_early(xs + 0), g_next = ld_early(ws + 0), u_next = GATED ? ld_early(wu + 0) : 0.f;
        for (int k = 0; k < blocks; ++k) {
          const float f = s_next * g_next, u = GATED ? s_next * u_next : f;
          const int at = min(k + 1, blocks - 1);
          s_next = ld_early(xs + at), g_next = ld_early(ws + at);
          if (GATED) u_next = ld_early(wu + at);
          on = __all_sync(~0u, mbar_wait(acc_full(buffer), turn, abort_flag));
          if (!on) break;
          tc_fence_after();
          if (rows > 0) add_block<128>(lanes + buffer * 256, acc, f, u);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster_relaxed(map_to(acc_empty(buffer), 0));
          if (++buffer == 2) buffer = 0, turn ^= 1;
        }
      } else {
        on = __all_sync(~0u, mbar_wait(acc_full(buffer), turn, abort_flag));
        if (on) {
          tc_fence_after();
          if (rows > 0) take_block<128>(lanes + buffer * 256, acc);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster_relaxed(map_to(acc_empty(buffer), 0));
          if (++buffer == 2) buffer = 0, turn ^= 1;
        }
      }
      if (!on) break;
      if (bad) {
#pragma unroll
        for (int i = 0; i < 64; ++i) acc[i] = 0;
      }
      // the results of this lane's row: 128 of them, or gated 64
      constexpr int kMine = GATED ? 64 : 128;
      const int n = tile.column + half * kMine;
      if (GATED) {
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const float2 g = unpack2(acc[i]), u = unpack2(acc[32 + i]);
          acc[i] = pack2(gate(g.x, u.x), gate(g.y, u.y));
        }
      }
      if (GATED && p.codes) {
        float amax = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const float2 y = unpack2(acc[i]);
          if (n + 2 * i < p.width) amax = fmaxf(amax, fabsf(y.x));
          if (n + 2 * i + 1 < p.width) amax = fmaxf(amax, fabsf(y.y));
        }
        // the row's other 64 results are another warp's
        const uint32_t here = lane * C::kRow + 64 + (tiles & 1) * 4;
        sts_u32(stage + here, __float_as_uint(amax));
        __syncwarp();
        if (lane == 0) mbar_arrive(both(q));
        on = __all_sync(~0u, mbar_wait(both(q), tiles & 1, abort_flag));
        if (!on) break;
        amax = fmaxf(amax, __uint_as_float(lds_u32(pieces + (warp ^ 4) * 32 * C::kRow + here)));
        const float step = __fdiv_rn(amax, 448.0f), s = step == 0.f ? 1.0f : step;
        uint32_t codes[16];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float y[8];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 v = unpack2(acc[4 * i + j]);
            y[2 * j] = v.x, y[2 * j + 1] = v.y;
          }
          const uint2 c = quantize8(y, s);
          codes[2 * i] = c.x, codes[2 * i + 1] = c.y;
        }
        if (rows > 0 && n < p.width) {
          uint8_t* const to = p.codes + row0 * p.width + n;
          if (vec) store_piece<true, 1>(stage, to, p.width, rows, p.width - n, codes);
          else store_piece<false, 1>(stage, to, p.width, rows, p.width - n, codes);
          if (half == 0 && lane < rows) p.scales[(row0 + lane) * ((p.width + 127) / 128) + tile.column / 128] = s;
        }
      } else if (rows > 0) {
        // pieces of 64 bytes: 32 results of 16 bits, or 16 of 32
        const int wanted = min(kMine, p.width - n);
        uint8_t* const to = static_cast<uint8_t*>(p.out) + (row0 * p.out_stride + n) * size;
        const bool whole = vec && wanted * size % 16 == 0;
        if (size == 2) {
#pragma unroll
          for (int c = 0; c < kMine / 32; ++c) {
            uint32_t v[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float2 y = unpack2(acc[16 * c + i]);
              v[i] = round_pair(y.x, y.y, p.out_type == 0);
            }
            if (32 * c >= wanted) continue;
            if (whole) store_piece<true, 2>(stage, to + 64 * c, p.out_stride * 2, rows, (wanted - 32 * c) * 2, v);
            else store_piece<false, 2>(stage, to + 64 * c, p.out_stride * 2, rows, (wanted - 32 * c) * 2, v);
          }
        } else {
#pragma unroll
          for (int c = 0; c < kMine / 16; ++c) {
            uint32_t v[16];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float2 y = unpack2(acc[8 * c + i]);
              v[2 * i] = __float_as_uint(y.x), v[2 * i + 1] = __float_as_uint(y.y);
            }
            if (16 * c >= wanted) continue;
            if (whole) store_piece<true, 4>(stage, to + 64 * c, p.out_stride * 4, rows, (wanted - 16 * c) * 4, v);
            else store_piece<false, 4>(stage, to + 64 * c, p.out_stride * 4, rows, (wanted - 16 * c) * 4, v);
          }
        }
      }
      ++tiles;
    }
  } else {
    regs_shrink<72>();
    if (warp == 8) {
      // ------------------------------------------------ loads
      int s = 0, phase = 0, left = stages_to_fill(p, rank);
      uint32_t used = 0, filled = 0, seconds = 0;
      for (int t = blockIdx.x / 2; on && find_tile<C::BM, C::kOut>(p, groups, t, &tile); t += step) {
        // a box of 128 rows for each CTA that has some
        const bool second = tile.count > 128, boxed = !p.rows && (rank == 0 || second);
        const uint32_t bytes = 2 * C::kStageB + (p.rows ? 0 : second ? 2 : 1) * C::kStageA;
        for (int k = 0; k < blocks; ++k) {
          if (left == 0 || !__all_sync(~0u, mbar_wait(empty(s), phase ^ 1, abort_flag))) {
            on = false;
            break;
          }
          left -= left > 0;
          const uint32_t a = stages + s * C::kStage, b = a + C::kStageA, bar = map_to(full(s), 0);
          const int x = k * C::kK;
          if (elect_one()) {
            if (rank == 0) mbar_arrive_expect_tx(full(s), bytes);
            if (GATED) {
              tma_load_3d_pair(b, &tw, x, tile.column + 64 * (int)rank, tile.e, bar);
              tma_load_3d_pair(b + 8192, &tw, x, p.width + tile.column + 64 * (int)rank, tile.e, bar);
            } else {
              tma_load_3d_pair(b, &tw, x, tile.column + 128 * (int)rank, tile.e, bar);
            }
            if (boxed) tma_load_2d_pair(a, &tx, x, tile.row + 128 * (int)rank, bar);
          }
          __syncwarp();
          used |= 1u << s;
          ++filled, seconds = seconds << 1 | second;
          if (++s == C::kStages) s = 0, phase ^= 1;
        }
      }
      tell_stop(loads_stopped, s, phase, used);
      if (lane == 0) sts_u32(fills, filled), sts_u32(fills + 4, seconds);
    } else if (warp == 9 && rank == 0) {
      // ------------------------------------------------ products of both CTAs
      const uint32_t idesc = FP8 ? idesc_e4m3_f32(256, 256) : idesc_16_f32(p.x_type == 0, 256, 256, false);
      int s = 0, phase = 0, buffer = 0, turn = 0;
      for (int t = blockIdx.x / 2; on && find_tile<C::BM, C::kOut>(p, groups, t, &tile); t += step) {
        for (int k = 0; k < blocks; ++k) {
          if (FP8 || k == 0) on = __all_sync(~0u, mbar_wait(acc_empty(buffer), turn ^ 1, abort_flag));
          on = on && __all_sync(~0u, mbar_wait(full(s), phase, abort_flag));
          // (the second CTA's are among them: written there, multiplied here)
          if (on && p.rows) on = __all_sync(~0u, mbar_wait_cluster<true>(landed(s), phase, abort_flag));
          if (!on) break;
          if (p.rows) fence_proxy_async_smem();
          tc_fence_after();
          const uint32_t a = stages + s * C::kStage, d = tmem + buffer * 256;
          if (elect_one()) {
            if (FP8) umma_f8_k128_pair(d, sw128_desc(a), sw128_desc(a + C::kStageA), idesc, 0);
            else umma_f16_k64_pair(d, sw128_desc(a), sw128_desc(a + C::kStageA), idesc, k > 0);
            umma_commit_pair(empty(s));
            if (FP8 || k + 1 == blocks) umma_commit_pair(acc_full(buffer));
          }
          __syncwarp();
          if (FP8 || k + 1 == blocks) {
            if (++buffer == 2) buffer = 0, turn ^= 1;
          }
          if (++s == C::kStages) s = 0, phase ^= 1;
        }
      }
      tell_stop(products_stopped, s, phase, 0);
    } else if (warp == 9 && p.rows) {
      // ------------------------------------------------ the second CTA's gathered rows, told to the first
      if (lane == 0) {
        int s = 0, phase = 0;
        for (int t = blockIdx.x / 2; on && find_tile<C::BM, C::kOut>(p, groups, t, &tile); t += step) {
          for (int k = 0; k < blocks; ++k) {
            on = mbar_wait(landed(s), phase, abort_flag);
            if (!on) break;
            fence_proxy_async_smem();
            mbar_arrive_shared(map_to(landed(s), 0));
            if (++s == C::kStages) s = 0, phase ^= 1;
          }
        }
      }
      __syncwarp();
    } else if (warp >= 10 && p.rows) {
      // ------------------------------------------------ gathered rows
      const int g = warp - 10;
      on = gather_rows<C::kStages, C::kStage, C::BM, C::kOut>(p, groups, blockIdx.x / 2, step, 128 * (int)rank, 128, FP8 ? 1 : 2, 0, blocks,
                                                              stages, g, abort_flag, empty(0), landed(0));
    }
  }
  if (!on) give_up(p, bars + 496, 2);
  __syncwarp();
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  if (*abort_flag) {  // (the same in both CTAs)
    if (rank == 1 && threadIdx.x < 2) st_cluster_u32(map_to(fills + 8 + 4 * threadIdx.x, 0), lds_u32(fills + 4 * threadIdx.x));
    if (rank == 0 && warp == 9) end_products(where_stopped(products_stopped), empty(0), C::kStages);
    __syncwarp();
    cluster_sync();
    // Both CTAs' copies arrive at the first's barriers, which expect those of both.  Where the second stopped earlier, its
    // bytes are taken off; where it went on, its copies alone are expected.
    if (rank == 0 && threadIdx.x == 256) {
      Stopped l = where_stopped(loads_stopped);
      const int ahead = (int)(lds_u32(fills + 8) - lds_u32(fills));
      const auto bytes = [&](bool rows) { return C::kStageB + (rows && !p.rows ? C::kStageA : 0u); };
      for (int i = 1; i <= -ahead; ++i)
        mbar_complete_tx(full((l.s + C::kStages - i) % C::kStages), bytes(lds_u32(fills + 4) >> (i - 1) & 1));
      for (int i = ahead - 1; i >= 0; --i) {
        mbar_arrive_expect_tx(full(l.s), bytes(lds_u32(fills + 12) >> i & 1));
        l.used |= 1u << l.s;
        if (++l.s == C::kStages) l.s = 0, l.phase ^= 1;
      }
      end_loads(l, full(0), C::kStages);
    }
    __syncwarp();
    cluster_sync();
  }
  if (warp == 9) tmem_dealloc_pair(tmem, 512);
}

}  // namespace dsa
