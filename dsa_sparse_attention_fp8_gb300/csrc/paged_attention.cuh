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
#include "ptx.cuh"

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
  int group;                   // Hq / Hkv
  int tile_tokens;             // tokens of a 128-row query tile: 128 / group
  int sink_tiles;              // ceil(sinks / 128)
  float* part;                 // [grid][2][256][DP] split units' outputs ...
  float2* part_ml;             // [grid][2][256] ... their maxima and sums ...
  uint32_t* counter;           // [grid] ... and the parts that have arrived
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

// ---------------------------------------------------------------------------
// The tensor-core kernel
// ---------------------------------------------------------------------------
constexpr int kAttnTile = 128;        // keys per tile (two pages)
constexpr int kAttnThreads = 384;     // 8 softmax warps, TMA, MMA, 2 housekeeping
constexpr int kAttnTmaWarp = 8;
constexpr int kAttnMmaWarp = 9;
constexpr int kAttnMaxGrid = 160;
constexpr float kAttnRescaleLog2 = 8.0f;  // rescale the output when the max grows by more than 2^8
constexpr int kAttnUnitCharge = 1;    // a unit's set-up, in key tiles

// A unit of work: up to two query tiles (2 * tile_tokens tokens) of one
// request and key head, over the key tiles that any of its rows sees: the
// first `ns` tiles (sinks), then those from `lo` on.
struct AttnUnit {
  int ntok;      // tokens
  int p0;        // position of the first
  int lo, ns, n; // first window tile, sink tiles before it, tiles in all
  int weight;    // cost of a key tile
};

__device__ __forceinline__ AttnUnit attn_unit(const AttnParams& p, int q, int seq, int u) {
  AttnUnit x;
  const int t0 = u * 2 * p.tile_tokens;
  x.ntok = min(2 * p.tile_tokens, q - t0);
  x.p0 = seq - q + t0;
  x.lo = 0;
  x.ns = 0;
  if (p.window > 0) {
    x.lo = max(0, x.p0 - p.window + 1) / kAttnTile;
    x.ns = min(p.sink_tiles, x.lo);
  }
  x.n = x.ns + (x.p0 + x.ntok - 1) / kAttnTile + 1 - x.lo;
  x.weight = x.ntok > p.tile_tokens ? 2 : 1;
  return x;
}

// New tokens and length of request r; q = 0 where its metadata make no sense.
__device__ __forceinline__ bool attn_request(const AttnParams& p, int r, int* row0, int* q, int* seq) {
  const int s0 = __ldg(p.start + r), s1 = __ldg(p.start + r + 1);
  *seq = __ldg(p.seq_lens + r);
  *row0 = s0;
  const bool ok = s0 >= 0 && s1 >= s0 && s1 <= p.T && *seq >= s1 - s0 &&
                  (int64_t)*seq <= (int64_t)p.max_blocks * kPageTokens;
  *q = ok ? s1 - s0 : 0;
  return ok;
}

__device__ __forceinline__ int attn_units(const AttnParams& p, int q) {
  return (q + 2 * p.tile_tokens - 1) / (2 * p.tile_tokens);
}

// Where a CTA is in the work: all units' costs laid end to end, requests
// outermost, then key heads, then units; the CTA owns [x0, x1).
struct AttnWalk {
  int r, head, u, nu;
  int row0, q, seq;
  int64_t s;     // cost before this unit
  int64_t x0, x1, share;
  AttnUnit unit;
  int j0, j1;    // this CTA's key tiles of the unit

  __device__ __forceinline__ void enter(const AttnParams& p) {
    unit = attn_unit(p, q, seq, u);
    // tile j lies at s + (charge + j) * weight
    const int64_t w = unit.weight;
    j0 = (int)max((int64_t)0, (x0 - s + w - 1) / w - kAttnUnitCharge);
    if (x0 <= s) j0 = 0;
    j1 = (int)min((int64_t)unit.n, (x1 - s + w - 1) / w - kAttnUnitCharge);
  }
  __device__ __forceinline__ bool inside(const AttnParams& p) const { return r < p.R && s < x1; }
  __device__ __forceinline__ void next(const AttnParams& p) {
    s += (int64_t)(unit.n + kAttnUnitCharge) * unit.weight;
    if (s >= x1) return;
    if (++u == nu) {
      u = 0;
      if (++head == p.Hkv) {
        head = 0;
        do {
          if (++r >= p.R) return;
          attn_request(p, r, &row0, &q, &seq);
        } while (q == 0);
        nu = attn_units(p, q);
      }
    }
    enter(p);
  }
  // The CTAs that own the unit's first and last key tile.
  __device__ __forceinline__ int first_cta() const {
    return (int)((s + (int64_t)kAttnUnitCharge * unit.weight) / share);
  }
  __device__ __forceinline__ int last_cta() const {
    return (int)((s + (int64_t)(kAttnUnitCharge + unit.n - 1) * unit.weight) / share);
  }
};

template <int DP>
struct AttnCfg {
  static constexpr int kHalves = DP / 64;
  static constexpr int kTileBytes = kHalves * 128 * 128;  // 128 rows of 64 elements, a half after the other
  static constexpr int kStages = DP == 128 ? 5 : 8;
  static constexpr int kSmem = (2 + kStages) * kTileBytes + 3072;
};

struct AttnSmem {
  uint64_t q_full[2], q_empty[2], kv_full[8], kv_empty[8], s_full[2], p_full[2], o_full[2], drain;
  uint32_t tmem;
  int32_t abort, last;
  int32_t begin_r, begin_head, begin_u;
  int64_t begin_s, total;
  int64_t warp_cost[kAttnThreads / 32];
  uint8_t bad[16];       // per key tile of the ring: bit i = page i is bad
  float2 ml[2][128];     // the two streams' maxima and sums
};
static_assert(sizeof(AttnSmem) <= 3072, "shared memory");

// tensor-memory columns of stream x
__device__ __forceinline__ uint32_t attn_col_s(int x) { return (uint32_t)x * 128; }
__device__ __forceinline__ uint32_t attn_col_o(int x) { return 256u + (uint32_t)x * 128; }

template <bool BF16>
__device__ __forceinline__ uint32_t attn_pack(float lo, float hi) {
  if (BF16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Finds where this CTA's share of the work begins: every CTA sums the
// requests' costs itself (a thread per request, a warp together for requests
// of several units).  Called by all threads; the result is in shared memory.
__device__ __forceinline__ void attn_locate(const AttnParams& p, AttnSmem* sm, int64_t* x0, int64_t* x1,
                                            int64_t* share) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per = (p.R + kAttnThreads - 1) / kAttnThreads;
  const int r0 = threadIdx.x * per;
  // cost of one key head of request r; lanes of a warp call it together
  auto cost = [&](int r, bool* bad) -> int64_t {
    int row0 = 0, q = 0, seq = 0;
    if (r < p.R && !attn_request(p, r, &row0, &q, &seq)) *bad = true;
    const int nu = attn_units(p, q);
    int64_t c = 0;
    if (nu == 1) {
      const AttnUnit x = attn_unit(p, q, seq, 0);
      c = (int64_t)(x.n + kAttnUnitCharge) * x.weight;
    }
    uint32_t many = __ballot_sync(0xffffffffu, nu > 1);
    while (many) {
      const int src = __ffs(many) - 1;
      many &= many - 1;
      const int q_s = __shfl_sync(0xffffffffu, q, src), seq_s = __shfl_sync(0xffffffffu, seq, src);
      const int nu_s = __shfl_sync(0xffffffffu, nu, src);
      int64_t sum = 0;
      for (int u = lane; u < nu_s; u += 32) {
        const AttnUnit x = attn_unit(p, q_s, seq_s, u);
        sum += (int64_t)(x.n + kAttnUnitCharge) * x.weight;
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (lane == src) c = sum;
    }
    return c;
  };
  bool bad = false;
  int64_t sum = 0, c_last = 0;
  for (int i = 0; i < per; ++i) {
    c_last = cost(r0 + i, &bad) * p.Hkv;
    sum += c_last;
  }
  if (bad && blockIdx.x == 0) raise_status(p.status, kStatusBadMetadata);
  int64_t inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  if (lane == 31) sm->warp_cost[warp] = inc;
  __syncthreads();
  int64_t before = inc - sum, total = 0;
  for (int w = 0; w < kAttnThreads / 32; ++w) {
    if (w < warp) before += sm->warp_cost[w];
    total += sm->warp_cost[w];
  }
  // shares of at least 4 single tiles: a split costs a unit's set-up and a merge
  *share = max((total + gridDim.x - 1) / (int64_t)gridDim.x, (int64_t)4);
  *x0 = (int64_t)blockIdx.x * *share;
  *x1 = min(*x0 + *share, total);
  const bool mine = *x0 < total && before <= *x0 && *x0 < before + sum;
  if (__any_sync(0xffffffffu, mine)) {
    int found = -1;
    int64_t at = before, cost_found = 0;
    for (int i = 0; i < per; ++i) {
      const int64_t c = per == 1 ? c_last : cost(r0 + i, &bad) * p.Hkv;
      if (mine && found < 0 && *x0 < at + c) {
        found = r0 + i;
        cost_found = c;
      }
      if (found < 0) at += c;
    }
    const int src = __ffs(__ballot_sync(0xffffffffu, mine)) - 1;
    const int r = __shfl_sync(0xffffffffu, found, src);
    const int64_t begin = __shfl_sync(0xffffffffu, at, src);
    const int64_t per_head = __shfl_sync(0xffffffffu, cost_found, src) / p.Hkv;
    const int head = (int)((*x0 - begin) / per_head);
    int64_t s = begin + head * per_head;
    int row0, q, seq;
    attn_request(p, r, &row0, &q, &seq);
    const int nu = attn_units(p, q);
    for (int u0 = 0; u0 < nu; u0 += 32) {
      int64_t c = 0;
      if (u0 + lane < nu) {
        const AttnUnit x = attn_unit(p, q, seq, u0 + lane);
        c = (int64_t)(x.n + kAttnUnitCharge) * x.weight;
      }
      int64_t end = c;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, end, o);
        if (lane >= o) end += y;
      }
      const uint32_t past = __ballot_sync(0xffffffffu, c > 0 && *x0 < s + end);
      if (past) {
        if (lane == __ffs(past) - 1) {
          sm->begin_r = r;
          sm->begin_head = head;
          sm->begin_u = u0 + lane;
          sm->begin_s = s + end - c;
        }
        break;
      }
      s += __shfl_sync(0xffffffffu, end, 31);
    }
  }
}

// Two streams of 128 query rows run side by side, each with its own score and
// output tiles in tensor memory (S, which its probabilities overwrite, and O:
// 2 x 256 columns, all of it) and its own four softmax warps, so that the
// tensor core works on one stream while the other's softmax runs.  A unit of
// two query tiles gives each stream one tile and both read the same K and V
// tiles.  A unit of one query tile (decode; the end of a prompt) gives both
// streams that tile and alternate key tiles: the two halves are joined at the
// end, in tensor memory.
//   warps 0-3, 4-7   softmax of stream 0, 1: thread = row;
//   warp 8           TMA: query tiles, K and V tiles through the block table;
//   warp 9           MMA: S = Q K^T, O += P V (P from tensor memory);
//   warps 10-11      rows that belong to no valid request: zeros.
template <int DP, bool BF16>
__global__ void __launch_bounds__(kAttnThreads, 1)
    paged_attention_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                           const __grid_constant__ CUtensorMap tv, const __grid_constant__ AttnParams p) {
  using C = AttnCfg<DP>;
  extern __shared__ __align__(1024) unsigned char attn_smem[];
  const uint32_t q_s = smem_u32(attn_smem);
  const uint32_t kv_s = q_s + 2 * C::kTileBytes;
  AttnSmem* sm = reinterpret_cast<AttnSmem*>(attn_smem + (2 + C::kStages) * C::kTileBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&sm->q_full[i]), 1);
      mbar_init(smem_u32(&sm->q_empty[i]), 1);
      mbar_init(smem_u32(&sm->s_full[i]), 1);
      mbar_init(smem_u32(&sm->p_full[i]), 4);
      mbar_init(smem_u32(&sm->o_full[i]), 1);
    }
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(smem_u32(&sm->kv_full[i]), 1);
      mbar_init(smem_u32(&sm->kv_empty[i]), 1);
    }
    mbar_init(smem_u32(&sm->drain), 1);
    sm->abort = 0;
    fence_barrier_init();
  }
  if (warp == kAttnMmaWarp) {
    tmem_alloc(smem_u32(&sm->tmem), 512);
    tmem_relinquish();
  }
  if (warp == kAttnTmaWarp && lane == 0) {
    tma_prefetch_desc(&tq);
    tma_prefetch_desc(&tk);
    tma_prefetch_desc(&tv);
  }
  AttnWalk w;
  attn_locate(p, sm, &w.x0, &w.x1, &w.share);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm->tmem;
  volatile int* abort_flag = &sm->abort;
  bool ok = true;
  // warp-uniform waits; after one gave up the role walks on without working
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (ok) {
      ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(bar), parity, abort_flag));
      if (!ok) *abort_flag = 1;
    }
    return ok;
  };
  if (w.x0 < w.x1) {
    w.r = sm->begin_r;
    w.head = sm->begin_head;
    w.u = sm->begin_u;
    w.s = sm->begin_s;
    attn_request(p, w.r, &w.row0, &w.q, &w.seq);
    w.nu = attn_units(p, w.q);
    w.enter(p);
  } else {
    w.r = p.R;
  }

  if (warp < 8) {
    // ================================================================ softmax
    regs_grow<216>();
    const int x = warp >> 2;                  // stream
    const int row = threadIdx.x & 127;        // row of its tile
    const int wg = warp & 3;
    const uint32_t lanes = tmem + ((uint32_t)(wg * 32) << 16);
    uint32_t n_s = 0, n_o[2] = {0, 0}, tile0 = 0;  // phases so far; key tiles before this unit
    for (; w.inside(p); w.next(p)) {
      const int n = w.j1 - w.j0;
      if (n <= 0) continue;
      const bool two = w.unit.ntok > p.tile_tokens;
      const int tok0 = two ? x * p.tile_tokens : 0;  // this stream's first token in the unit
      const int ntok = two ? (x ? w.unit.ntok - p.tile_tokens : p.tile_tokens) : w.unit.ntok;
      const int rows = ntok * p.group;
      const bool live = wg * 32 < rows;       // some row of this warp is real
      const int tok = min(row / p.group, ntok - 1);
      const int pos = w.unit.p0 + tok0 + tok;
      const int pos_lo = w.unit.p0 + tok0, pos_hi = pos_lo + ntok - 1;
      float m = -INFINITY, l = 0.f;
      int done = 0;
      for (int j = two ? 0 : x; j < n; j += two ? 1 : 2) {
        wait(&sm->s_full[x], n_s & 1);
        ++n_s;
        if (live && ok) {
          tc_fence_after();
          uint32_t s[128];
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld<32>(lanes + attn_col_s(x) + 32 * c, s + 32 * c);
          const int jj = w.j0 + j;
          const int s0 = (jj < w.unit.ns ? jj : w.unit.lo + jj - w.unit.ns) * kAttnTile;
          const uint32_t bad = sm->bad[(tile0 + j) & 15];
          const bool whole = s0 + kAttnTile - 1 <= pos_lo && bad == 0 &&
                             (p.window == 0 || s0 > pos_hi - p.window || s0 + kAttnTile - 1 < p.sinks);
          tmem_ld_wait();
          if (!whole) {
            const int hi = pos - s0, lo = p.window > 0 ? hi - p.window : -1, sk = p.sinks - s0;
#pragma unroll
            for (int c = 0; c < 128; ++c) {
              const bool seen = c <= hi && (c > lo || c < sk) && !((bad >> (c / 64)) & 1u);
              if (!seen) s[c] = 0xFF800000u;  // -inf
            }
          }
          float mx[8];
#pragma unroll
          for (int c = 0; c < 8; ++c) mx[c] = __uint_as_float(s[c]);
#pragma unroll
          for (int c = 8; c < 128; ++c) mx[c & 7] = fmaxf(mx[c & 7], __uint_as_float(s[c]));
          const float top = fmaxf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])),
                                  fmaxf(fmaxf(mx[4], mx[5]), fmaxf(mx[6], mx[7]))) * p.scale_log2;
          const bool grow = top > m + kAttnRescaleLog2;
          const float m_new = grow ? top : m;
          if (__any_sync(0xffffffffu, grow && done > 0)) {
            // the scores' arrival says that the stream's previous product is done
            const float a = grow && m != -INFINITY ? ex2(m - m_new) : 1.0f;
            for (int c = 0; c < DP; c += 32) {
              uint32_t o[32];
              tmem_ld<32>(lanes + attn_col_o(x) + c, o);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * a);
              tmem_st<32>(lanes + attn_col_o(x) + c, o);
            }
            l *= a;
          }
          m = m_new;
          const float shift = m == -INFINITY ? 0.f : -m;
          const uint64_t mul = pack2(p.scale_log2, p.scale_log2), sub = pack2(shift, shift);
          uint64_t sum[4] = {0, 0, 0, 0};
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t pr[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float2 z = unpack2(fma2(pack2(__uint_as_float(s[32 * c + 2 * i]),
                                                  __uint_as_float(s[32 * c + 2 * i + 1])), mul, sub));
              const float e0 = ex2(z.x), e1 = ex2(z.y);
              sum[i & 3] = add2(sum[i & 3], pack2(e0, e1));
              pr[i] = attn_pack<BF16>(e0, e1);
            }
            tmem_st<16>(lanes + attn_col_s(x) + 16 * c, pr);
          }
          const float2 t = unpack2(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])));
          l += t.x + t.y;
          tmem_st_wait();
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm->p_full[x]));
        ++done;
      }
      tile0 += n;

      // ---- the unit's end: out = O / l, or the part of a split unit
      const int c0 = w.first_cta(), c1 = w.last_cta();
      const bool split = c0 != c1;
      // which streams have an output, and its factors
      float f0 = 1.f, f1 = 0.f;
      const bool has0 = two ? x == 0 : true, has1 = two ? x == 1 : n > 1;
      if (has0 || !two) wait(&sm->o_full[0], n_o[0] & 1);
      if (has1) wait(&sm->o_full[1], n_o[1] & 1);
      ++n_o[0];
      if (two || n > 1) ++n_o[1];
      tc_fence_after();
      int col0 = 0, cols = DP;
      if (!two) {
        // both streams' warps share the rows: each takes half of the columns
        sm->ml[x][row] = make_float2(m, l);
        named_bar_sync(1, 256);
        const float2 a = sm->ml[0][row], b = sm->ml[1][row];
        m = fmaxf(a.x, b.x);
        f0 = a.x == -INFINITY ? 0.f : ex2(a.x - m);
        f1 = b.x == -INFINITY ? 0.f : ex2(b.x - m);
        l = a.y * f0 + b.y * f1;
        col0 = x * (DP / 2);
        cols = DP / 2;
      } else {
        f0 = f1 = 1.f;
      }
      const bool row_ok = row < rows;
      const int token = w.row0 + w.u * 2 * p.tile_tokens + tok0 + tok;
      const int head = w.head * p.group + row % p.group;
      const float inv = split ? 1.0f : (l > 0.f ? 1.0f / l : 0.f);
      const int slot = (int)blockIdx.x * 2 + (w.s >= w.x0 ? 1 : 0);
      const int prow = two ? x * 128 + row : row;
      if (live && ok) {
        f0 *= inv;
        f1 *= inv;
        uint16_t* orow = p.out + (int64_t)token * p.out_token + (int64_t)head * p.out_head;
        float* srow = p.part + ((int64_t)slot * 256 + prow) * DP;
#pragma unroll
        for (int c = 0; c < DP; c += 16) {
          if (c >= cols) break;
          const int at = col0 + c;
          uint32_t a[16], b[16];
          float o[16];
          if (has0) tmem_ld<16>(lanes + attn_col_o(0) + at, a);
          if (has1) tmem_ld<16>(lanes + attn_col_o(1) + at, b);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            o[i] = 0.f;
            if (has0) o[i] = __uint_as_float(a[i]) * f0;
            if (has1) o[i] += __uint_as_float(b[i]) * f1;
          }
          if (row_ok && at < p.D) {
            if (split) {
#pragma unroll
              for (int i = 0; i < 16; i += 4)
                __stcg(reinterpret_cast<float4*>(srow + at + i), make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]));
            } else {
              uint32_t v[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) v[i] = attn_pack<BF16>(o[2 * i], o[2 * i + 1]);
              reinterpret_cast<uint4*>(orow + at)[0] = make_uint4(v[0], v[1], v[2], v[3]);
              reinterpret_cast<uint4*>(orow + at)[1] = make_uint4(v[4], v[5], v[6], v[7]);
            }
          }
        }
        if (row_ok && col0 == 0) {
          if (split)
            __stcg(p.part_ml + (int64_t)slot * 256 + prow, make_float2(m, l));
          else if (p.lse)
            p.lse[(int64_t)token * p.Hq + head] =
                l > 0.f ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
        }
      }
      tc_fence_before();
      if (split) {
        // the unit's last CTA to arrive joins the parts, in CTA order
        __threadfence();
        named_bar_sync(1, 256);
        if (threadIdx.x == 0) {
          const uint32_t parts = (uint32_t)(c1 - c0 + 1);
          const bool last = atomicAdd(p.counter + c0, 1u) == parts - 1;
          if (last) p.counter[c0] = 0;
          sm->last = last;
        }
        named_bar_sync(1, 256);
        if (sm->last) {
          __threadfence();
          const int parts = c1 - c0 + 1;
          const int all = w.unit.ntok * p.group;            // rows of both tiles
          const int rows0 = p.tile_tokens * p.group;        // rows of the first tile
          for (int i = warp; i < all; i += 8) {
            const int pr = two && i >= rows0 ? 128 + i - rows0 : i;
            // part k lies in slot 1 of the CTA where the unit begins, in slot 0 of the others
            auto at = [&](int k) -> int64_t {
              return ((int64_t)(c0 + k) * 2 + (k == 0 && w.s >= (int64_t)c0 * w.share ? 1 : 0)) * 256 + pr;
            };
            float top = -INFINITY;
            for (int k = lane; k < parts; k += 32) top = fmaxf(top, __ldcg(p.part_ml + at(k)).x);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            float sum = 0.f, acc[DP / 32];
#pragma unroll
            for (int c = 0; c < DP / 32; ++c) acc[c] = 0.f;
            for (int k0 = 0; k0 < parts; k0 += 32) {
              float f = 0.f;
              if (k0 + lane < parts) {
                const float2 v = __ldcg(p.part_ml + at(k0 + lane));
                f = v.x == -INFINITY ? 0.f : ex2(v.x - top);
                sum += v.y * f;
              }
              const int most = min(32, parts - k0);
#pragma unroll 4
              for (int k = 0; k < most; ++k) {
                const float fk = __shfl_sync(0xffffffffu, f, k);
                const float* src = p.part + at(k0 + k) * DP + lane * (DP / 32);
                if (lane * (DP / 32) < p.D) {
                  if (DP == 128) {
                    const float4 v = __ldcg(reinterpret_cast<const float4*>(src));
                    acc[0] += v.x * fk;
                    acc[1] += v.y * fk;
                    acc[2 % (DP / 32)] += v.z * fk;
                    acc[3 % (DP / 32)] += v.w * fk;
                  } else {
                    const float2 v = __ldcg(reinterpret_cast<const float2*>(src));
                    acc[0] += v.x * fk;
                    acc[1] += v.y * fk;
                  }
                }
              }
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            const float r = sum > 0.f ? 1.0f / sum : 0.f;
            const int64_t t = w.row0 + w.u * 2 * p.tile_tokens + i / p.group;
            const int h = w.head * p.group + i % p.group;
            uint16_t* orow = p.out + t * p.out_token + (int64_t)h * p.out_head + lane * (DP / 32);
            if (lane * (DP / 32) < p.D) {
#pragma unroll
              for (int c = 0; c < DP / 32; c += 2)
                *reinterpret_cast<uint32_t*>(orow + c) = attn_pack<BF16>(acc[c] * r, acc[c + 1] * r);
            }
            if (lane == 0 && p.lse)
              p.lse[t * p.Hq + h] = sum > 0.f ? (top + log2f(sum)) * 0.69314718055994531f : -INFINITY;
          }
        }
      }
      // the other stream's warps may still read this one's output
      if (!two) named_bar_sync(1, 256);
    }
    if (!ok) raise_status(p.status, kStatusTimeout);
  } else {
    regs_shrink<72>();
    if (warp == kAttnTmaWarp) {
      // ================================================================ TMA
      uint32_t n_kv = 0, n_q = 0, tile0 = 0;
      auto load = [&](const CUtensorMap* map, int head, int page0, int page1) {
        const uint32_t st = n_kv % C::kStages, round = n_kv / C::kStages;
        if (round > 0) wait(&sm->kv_empty[st], (round - 1) & 1);
        if (!ok) return;
        if (lane == 0) {
          const uint32_t bar = smem_u32(&sm->kv_full[st]), dst = kv_s + st * C::kTileBytes;
          mbar_arrive_expect_tx(bar, C::kTileBytes);
#pragma unroll
          for (int h = 0; h < C::kHalves; ++h) {
            tma_load_4d(dst + h * 16384, map, h * 64, head, 0, page0, bar);
            tma_load_4d(dst + h * 16384 + 8192, map, h * 64, head, 0, page1, bar);
          }
        }
        __syncwarp();
        ++n_kv;
      };
      auto load_q = [&](int head, int token) {
        const uint32_t st = n_q & 1, round = n_q >> 1;
        if (round > 0) wait(&sm->q_empty[st], (round - 1) & 1);
        if (!ok) return;
        if (lane == 0) {
          const uint32_t bar = smem_u32(&sm->q_full[st]), dst = q_s + st * C::kTileBytes;
          mbar_arrive_expect_tx(bar, (uint32_t)(C::kHalves * p.tile_tokens * p.group * 128));
#pragma unroll
          for (int h = 0; h < C::kHalves; ++h)
            tma_load_3d(dst + h * 16384, &tq, h * 64, head * p.group, token, bar);
        }
        __syncwarp();
        ++n_q;
      };
      for (; w.inside(p) && ok; w.next(p)) {
        const int n = w.j1 - w.j0;
        if (n <= 0) continue;
        const bool two = w.unit.ntok > p.tile_tokens;
        const int token = w.row0 + w.u * 2 * p.tile_tokens;
        const int p1 = w.unit.p0 + w.unit.ntok - 1;
        const int first = p.window > 0 ? max(0, w.unit.p0 - p.window + 1) : 0;
        const int32_t* bt = p.block_table + (int64_t)w.r * p.max_blocks;
        auto tile_of = [&](int jj) { return jj < w.unit.ns ? jj : w.unit.lo + jj - w.unit.ns; };
        // page ids of 16 tiles, a pair of lanes each: the pool's end (zeros)
        // for pages that no row sees and for bad ones
        auto ids = [&](int j) -> int {
          const int jj = w.j0 + j + (lane >> 1);
          if (j + (lane >> 1) >= n) return 0;
          const int b = tile_of(jj) * 2 + (lane & 1);
          const int64_t t0 = (int64_t)b * kPageTokens;
          if (t0 > p1 || !(t0 + kPageTokens > first || t0 < p.sinks)) return (int)p.num_pages;
          const int id = __ldg(bt + b);
          if (id < 0 || id >= p.num_pages) {
            raise_status(p.status, kStatusBadPage);
            return -1;
          }
          return id;
        };
        int here = ids(0), ahead = ids(16);
        int pg[2][2] = {{0, 0}, {0, 0}};  // the newest key tile's pages, and those of the one before
        auto load_k = [&](int j) {
          if (j > 0 && (j & 15) == 0) {
            here = ahead;
            ahead = ids(j + 16);
          }
          pg[1][0] = pg[0][0];
          pg[1][1] = pg[0][1];
          int a = __shfl_sync(0xffffffffu, here, (j & 15) * 2);
          int b = __shfl_sync(0xffffffffu, here, (j & 15) * 2 + 1);
          if (lane == 0) sm->bad[(tile0 + j) & 15] = (uint8_t)((a < 0 ? 1 : 0) | (b < 0 ? 2 : 0));
          __syncwarp();
          pg[0][0] = a < 0 ? (int)p.num_pages : a;
          pg[0][1] = b < 0 ? (int)p.num_pages : b;
          load(&tk, w.head, pg[0][0], pg[0][1]);
        };
        load_k(0);
        load_q(w.head, token);
        if (two) {
          load_q(w.head, token + p.tile_tokens);
          load(&tv, w.head, pg[0][0], pg[0][1]);
          for (int j = 1; j < n && ok; ++j) {
            load_k(j);
            load(&tv, w.head, pg[0][0], pg[0][1]);
          }
        } else {
          if (n > 1) load_k(1);
          for (int j = 0; j < n && ok; ++j) {
            const int i = j + 1 < n ? 1 : 0;
            load(&tv, w.head, pg[i][0], pg[i][1]);
            if (j + 2 < n) load_k(j + 2);
          }
        }
        tile0 += n;
      }
      // every copy has landed before the CTA leaves
      for (uint32_t i = n_kv > C::kStages ? n_kv - C::kStages : 0; i < n_kv; ++i)
        mbar_wait(smem_u32(&sm->kv_full[i % C::kStages]), (i / C::kStages) & 1, nullptr);
      for (uint32_t i = n_q > 2 ? n_q - 2 : 0; i < n_q; ++i)
        mbar_wait(smem_u32(&sm->q_full[i & 1]), (i >> 1) & 1, nullptr);
    } else if (warp == kAttnMmaWarp) {
      // ================================================================ MMA
      const uint32_t id_qk = idesc_16_f32(BF16, 128, 128, false);
      const uint32_t id_pv = idesc_16_f32(BF16, 128, (uint32_t)p.D, true);
      const int ksteps = p.D / 16;
      uint32_t n_kv = 0, n_q = 0, n_p[2] = {0, 0};
      auto qk = [&](int x, uint32_t q_slot, uint32_t st) {
        if (lane == 0) {
          const uint64_t a = sw128_desc(q_s + q_slot * C::kTileBytes), b = sw128_desc(kv_s + st * C::kTileBytes);
#pragma unroll
          for (int k = 0; k < DP / 16; ++k)
            if (k < ksteps) {
              const uint64_t off = (uint64_t)((k >> 2) * 16384 + (k & 3) * 32) >> 4;
              umma_f16(tmem + attn_col_s(x), a + off, b + off, id_qk, k > 0);
            }
          umma_commit(smem_u32(&sm->s_full[x]));
        }
      };
      auto pv = [&](int x, uint32_t st, bool accumulate) {
        if (lane == 0) {
          const uint64_t b = sw128_desc_mn(kv_s + st * C::kTileBytes, 16384, 1024);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            umma_f16_ta(tmem + attn_col_o(x), tmem + attn_col_s(x) + 8 * k, b + (uint64_t)(k * 2048 >> 4), id_pv,
                        accumulate || k > 0);
        }
      };
      auto commit = [&](uint64_t* bar) {
        if (lane == 0) umma_commit(smem_u32(bar));
      };
      auto kv_wait = [&](uint32_t i) { return wait(&sm->kv_full[i % C::kStages], (i / C::kStages) & 1); };
      for (; w.inside(p) && ok; w.next(p)) {
        const int n = w.j1 - w.j0;
        if (n <= 0) continue;
        const bool two = w.unit.ntok > p.tile_tokens;
        // values past the request's end, in its last page, may be anything: 0 * NaN would spoil the sum
        auto clean = [&](int j, uint32_t st) {
          const int jj = w.j0 + j;
          const int s0 = (jj < w.unit.ns ? jj : w.unit.lo + jj - w.unit.ns) * kAttnTile;
          const int from = w.seq - s0;
          if (from >= kAttnTile || from <= 0 || from % kPageTokens == 0) return;
          const int to = from < kPageTokens ? kPageTokens : kAttnTile;
          const uint32_t base = kv_s + st * C::kTileBytes;
          for (int i = lane; i < (to - from) * 8; i += 32)
#pragma unroll
            for (int h = 0; h < C::kHalves; ++h) sts_v4(base + h * 16384 + from * 128 + i * 16, make_uint4(0, 0, 0, 0));
          fence_proxy_async_smem();
          __syncwarp();
        };
        if (two) {
          const uint32_t qa = n_q & 1, qb = qa ^ 1;
          if (!wait(&sm->q_full[qa], (n_q >> 1) & 1)) break;
          ++n_q;
          if (!kv_wait(n_kv)) break;
          tc_fence_after();
          qk(0, qa, n_kv % C::kStages);
          if (n == 1) commit(&sm->q_empty[qa]);
          if (!wait(&sm->q_full[qb], (n_q >> 1) & 1)) break;
          ++n_q;
          qk(1, qb, n_kv % C::kStages);
          if (n == 1) commit(&sm->q_empty[qb]);
          commit(&sm->kv_empty[n_kv % C::kStages]);
          ++n_kv;
          for (int j = 0; j < n; ++j) {
            const uint32_t v = n_kv % C::kStages, k = (n_kv + 1) % C::kStages;
            if (!kv_wait(n_kv)) break;
            clean(j, v);
            if (!wait(&sm->p_full[0], n_p[0] & 1)) break;
            ++n_p[0];
            tc_fence_after();
            pv(0, v, j > 0);
            if (j + 1 < n) {
              if (!kv_wait(n_kv + 1)) break;
              qk(0, qa, k);
              if (j + 2 == n) commit(&sm->q_empty[qa]);
            } else {
              commit(&sm->o_full[0]);
            }
            if (!wait(&sm->p_full[1], n_p[1] & 1)) break;
            ++n_p[1];
            tc_fence_after();
            pv(1, v, j > 0);
            commit(&sm->kv_empty[v]);
            ++n_kv;
            if (j + 1 < n) {
              qk(1, qb, k);
              if (j + 2 == n) commit(&sm->q_empty[qb]);
              commit(&sm->kv_empty[k]);
              ++n_kv;
            } else {
              commit(&sm->o_full[1]);
            }
          }
        } else {
          const uint32_t qa = n_q & 1;
          if (!wait(&sm->q_full[qa], (n_q >> 1) & 1)) break;
          ++n_q;
          for (int j = 0; j < min(2, n); ++j) {
            if (!kv_wait(n_kv)) break;
            tc_fence_after();
            qk(j, qa, n_kv % C::kStages);
            if (j + 1 == n) commit(&sm->q_empty[qa]);
            commit(&sm->kv_empty[n_kv % C::kStages]);
            ++n_kv;
          }
          for (int j = 0; j < n && ok; ++j) {
            const int x = j & 1;
            const uint32_t v = n_kv % C::kStages;
            if (!kv_wait(n_kv)) break;
            clean(j, v);
            if (!wait(&sm->p_full[x], n_p[x] & 1)) break;
            ++n_p[x];
            tc_fence_after();
            pv(x, v, j > 1);
            commit(&sm->kv_empty[v]);
            ++n_kv;
            if (j + 2 < n) {
              if (!kv_wait(n_kv)) break;
              tc_fence_after();
              qk(x, qa, n_kv % C::kStages);
              if (j + 3 == n) commit(&sm->q_empty[qa]);
              commit(&sm->kv_empty[n_kv % C::kStages]);
              ++n_kv;
            } else {
              commit(&sm->o_full[x]);
            }
          }
        }
      }
      // every product issued has completed before tensor memory is released
      commit(&sm->drain);
      if (!mbar_wait(smem_u32(&sm->drain), 0, nullptr)) ok = false;
      if (!ok) {
        sm->abort = 1;
        raise_status(p.status, kStatusTimeout);
      }
    } else {
      // ================================================================ rows of no request
      const int64_t lo = (int64_t)blockIdx.x * p.T / gridDim.x, hi = ((int64_t)blockIdx.x + 1) * p.T / gridDim.x;
      for (int64_t t0 = lo + (warp - 10) * 32; t0 < hi; t0 += 64) {
        const int t = (int)t0 + lane;
        bool none = false;
        if (t < hi) {
          const int r = find_request(p.start, p.R, t);
          int row0, q, seq;
          none = !attn_request(p, r, &row0, &q, &seq) || t < row0 || t >= row0 + q;
        }
        uint32_t todo = __ballot_sync(0xffffffffu, none);
        while (todo) {
          const int64_t row = t0 + __ffs(todo) - 1;
          todo &= todo - 1;
          for (int i = lane; i < p.Hq * (p.D / 8); i += 32)
            *reinterpret_cast<uint4*>(p.out + row * p.out_token + (int64_t)(i / (p.D / 8)) * p.out_head +
                                      i % (p.D / 8) * 8) = make_uint4(0, 0, 0, 0);
          if (p.lse)
            for (int i = lane; i < p.Hq; i += 32) p.lse[row * p.Hq + i] = -INFINITY;
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (sm->abort)
    for (int k = 0; k < 100; ++k) __nanosleep(1000);  // copies that the drain gave up on
  if (warp == kAttnMmaWarp) tmem_dealloc(tmem, 512);
}

}  // namespace dsa
