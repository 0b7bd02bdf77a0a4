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
#include <cstddef>
#include <cstdint>
#include <type_traits>

#include "common.cuh"
#include "ptx_serving.cuh"

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
  bool give_up;                // for tests: the loading warp gives up at once
  int group;                   // Hq / Hkv
  int tile_tokens;             // tokens of a 128-row query tile: 128 / group
  int tile_tokens32;           // tokens of 32 rows: 32 / group
  int sink_tiles;              // ceil(sinks / 128)
  float* part;                 // [grid][2][DP / 4][256][4] split units' outputs ...
  float2* part_ml;             // [grid][2][256] ... their maxima and sums ...
  uint32_t* counter;           // [3][kAttnMaxGrid] ... and the parts that have arrived (see below)
};

constexpr int kAttnTile = 128;        // keys per tile (two pages)
constexpr int kAttnSoftmaxWarps = 8;
constexpr int kAttnWalkWarp = 8;
constexpr int kAttnMmaWarp = 9;       // and 10: one for each stream
constexpr int kAttnTmaWarp = 11;
constexpr int kAttnConvertWarp = 12;  // to 15, with an E4M3 cache
constexpr int kAttnMaxGrid = 160;
// A row's probabilities are 2^(score - m) with m the maximum of the tiles up to
// its last rescale, or a little less; a tile whose probabilities add up to more
// than attn_most_sum gets a new m.  FP16 holds 65,504 at most and loses what is
// below 2^-25: there m lies 6 under the maximum, so that the largest probability
// is 2^6 at least and what is lost or off by rounding below the normal numbers
// comes to 2^-31 of the row's sum for each key, 2^-11 (a rounding of the output)
// for a million of them.  Of a flat tile's 128 probabilities of 2^6 the sum is an
// eighth of the most.
template <bool BF16>
__device__ constexpr float attn_most_sum() { return BF16 ? 16384.0f : 65504.0f; }
template <bool BF16>
__device__ constexpr float attn_lift() { return BF16 ? 0.0f : 6.0f; }
constexpr float kAttnRescaleLog2 = 8.0f;  // (with E4M3 caches: when the maximum grows by more than 2^8)
// The most that a CTA's work may cost: places in it are 32 bits, and a unit of
// 2^25 may begin before it or end after it.  At some 0.3 us a key tile and stream
// that is minutes (2.8e7 for a prompt of a million tokens under 128 heads).
constexpr int64_t kAttnMaxShare = 1 << 30;
constexpr int kAttnUnitCharge = 1;    // a unit's set-up, in key tiles (2 and 3 change no measured batch by 2 %)
// Over E4M3 caches, units of at most 32 rows to a stream and this many key tiles
// or more give each warp of a stream all rows and a quarter of a tile's keys.
// That shortens each tile and costs a join of the warps' parts: 464 us instead
// of 600 for four requests of 231,000 tokens, 171 instead of 204 for 64 in a
// window of 4096, 96 instead of 106 for 64 of 2,000; 216 and 218 for 256 of
// 1,000; but 510 instead of 481 for 1,000 requests of 300, 23.6 instead of 21.5
// for one of 1,024 (split).  16-bit caches, whose softmax keeps the tile's
// probabilities in registers, lose by it (28.8 instead of 20.6 us for one
// request of 1,024 tokens, 218 instead of 201 for 64 of 1,000 to 8,000).
constexpr int kAttnFewTiles = 8;
// Parts of a unit split over more CTAs than this are joined in groups first,
// by one CTA of each group: one request of 100,000 tokens over one key head,
// 131 parts, bf16: of 128 query heads 59 us, 196 if one CTA joins them all; of
// 8 query heads 27 and 39.  Up to two groups' worth the second round of
// arrivals costs what it saves (four requests of 20,000 tokens over four key
// heads, 10 parts each: 50 us either way); groups of 6 give 67 and 28.
// A unit's count of arrivals is at its first CTA, that of its first group
// kAttnMaxGrid further on, those of the other groups at the group's first CTA
// another kAttnMaxGrid further on (two units share a CTA only as the last one
// of the one and the first of the other).
constexpr int kAttnUngrouped = 24;
constexpr int kAttnGroup = 12;

// A unit of work: the query rows of one request that two streams of 128 rows
// take at a time, over the key tiles that any of its rows sees: the first `ns`
// tiles (sinks), then those from `lo` on.
enum AttnKind : int {
  kOneTile = 0,   // one query tile of one key head: the streams take turns at the key tiles
  kTwoTiles = 1,  // two query tiles of one key head: a stream each, the same key tiles
  kTwoHeads = 2,  // a query tile each of two neighbouring key heads: a stream each, its head's key tiles
};
struct AttnUnit {
  int kind;
  int ntok;      // tokens
  int p0;        // position of the first
  int lo, ns, n; // first window tile, sink tiles before it, tiles in all
  __device__ __forceinline__ int lg_weight() const { return kind != kOneTile; }  // cost of a key tile: 1 or 2
  __device__ __forceinline__ int cost() const;
};

// Requests of at most one query tile take their key heads in pairs: a page's
// rows of two neighbouring heads lie next to each other, and DRAM gives twice
// the bytes of an E4M3 row for the same effort.
__device__ __forceinline__ bool attn_pairs(const AttnParams& p, int q) { return q <= p.tile_tokens && p.Hkv > 1; }

__device__ __forceinline__ AttnUnit attn_unit(const AttnParams& p, int q, int seq, int u, int head) {
  AttnUnit x;
  const int t0 = u * 2 * p.tile_tokens;
  x.ntok = min(2 * p.tile_tokens, q - t0);
  x.kind = x.ntok > p.tile_tokens ? kTwoTiles : attn_pairs(p, q) && head + 1 < p.Hkv ? kTwoHeads : kOneTile;
  x.p0 = seq - q + t0;
  x.lo = 0;
  x.ns = 0;
  if (p.window > 0) {
    x.lo = max(0, x.p0 - p.window + 1) / kAttnTile;
    x.ns = min(p.sink_tiles, x.lo);
  }
  x.n = x.ns + (x.p0 + x.ntok - 1) / kAttnTile + 1 - x.lo;
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

__device__ __forceinline__ int AttnUnit::cost() const { return (n + kAttnUnitCharge) << lg_weight(); }

__device__ __forceinline__ int attn_units(const AttnParams& p, int q) {
  return (q + 2 * p.tile_tokens - 1) / (2 * p.tile_tokens);
}

// Where a CTA is in the work: all units' costs laid end to end, requests
// outermost, then key heads, then units, and cut into equal shares.  Places
// are relative to the CTA's share [0, len).
struct AttnWalk {
  int r, head, u, nu;
  int row0, q, seq;
  int s;         // cost before this unit (negative: it began in an earlier share)
  int len, share;
  AttnUnit unit;
  int j0, j1;    // this CTA's key tiles of the unit

  __device__ __forceinline__ void enter(const AttnParams& p) {
    unit = attn_unit(p, q, seq, u, head);
    // tile j lies at s + (charge + j) * weight
    const int lg = unit.lg_weight();
    j0 = s >= 0 ? 0 : max(0, ((lg - s) >> lg) - kAttnUnitCharge);
    j1 = min(unit.n, ((len - s + lg) >> lg) - kAttnUnitCharge);
  }
  __device__ __forceinline__ bool inside() const { return s < len; }
  __device__ __forceinline__ void next(const AttnParams& p) {
    s += unit.cost();
    if (s >= len) return;
    if (++u == nu) {
      u = 0;
      head += unit.kind == kTwoHeads ? 2 : 1;
      if (head == p.Hkv) {
        head = 0;
        do {
          ++r;  // there is one with rows: the share goes on
          attn_request(p, r, &row0, &q, &seq);
        } while (q == 0);
        nu = attn_units(p, q);
      }
    }
    enter(p);
  }
  // The CTAs that own the unit's first and last key tile.
  __device__ __forceinline__ int cta_of(int j) const {
    const int at = s + ((kAttnUnitCharge + j) << unit.lg_weight());
    return (int)blockIdx.x + (at >= 0 ? at / share : -((share - 1 - at) / share));
  }
};

constexpr int kAttnMiscBytes = 3 * 1024;  // of AttnSmem
template <int DP, bool FP8>
struct AttnCfg {
  static constexpr int kHalves = DP / 64;
  static constexpr int kTileBytes = kHalves * 128 * 128;  // 128 rows of 64 16-bit elements, a half after the other
  static constexpr int kRawBytes = 128 * 128;             // 128 rows of 128 E4M3 codes
  // Tiles in flight.  16-bit caches: one ring of K and V tiles.  E4M3 caches: a
  // ring of K tiles as they are, one of V tiles as they are and one of V tiles
  // as BF16, and the scales of kScaleTiles key tiles (128 of K, 128 of V).
  static constexpr int kStages = DP == 128 ? 5 : 8;
  static constexpr int kKStages = 3, kVRawStages = 2, kVStages = 2, kScaleTiles = 8;
  static constexpr int kThreads = FP8 ? 512 : 384;
  static constexpr int kQ = 0, kKv = 2 * kTileBytes;
  static constexpr int kV = kKv + kKStages * kRawBytes, kVRaw = kV + kVStages * kTileBytes;
  static constexpr int kScale = kVRaw + kVRawStages * kRawBytes;  // then the query rows' factors, 128 for each slot
  static constexpr int kOnes = kScale + (kScaleTiles + 1) * 1024;  // 128 scales of 1
  static constexpr int kMisc = FP8 ? kOnes + 512 : kKv + kStages * kTileBytes;
  static constexpr int kSmem = kMisc + kAttnMiscBytes;
  // Registers a thread.  16-bit caches: 168 (65,536 / 384, in eights).  E4M3
  // caches: 128 at launch, the softmax warps taking some of the others'.
  static constexpr int kSoftmaxRegs = 176, kIssueRegs = 72, kConvertRegs = 88;
  static_assert(2 * kSoftmaxRegs + kIssueRegs + kConvertRegs <= 4 * 128, "the block's registers");
  static_assert(kSmem <= 232448, "shared memory");
  static_assert(!FP8 || DP == 128, "E4M3 rows are 128 bytes, whatever the head's size");
};

// One unit's part of a CTA's share, as the walking warp hands it to the others.
struct AttnItem {
  int n;          // tiles of K (0: the end); of two heads, those of both in turn
  int ntok;       // tokens of the unit
  int kind;       // AttnKind
  int p0;         // position of the first token
  int lo[2], hi[2];  // positions of each stream's first and last token
  int few;           // each warp of a stream has all of its rows (at most 32), and 32 of a tile's keys
  int from[2], step; // a stream's first key tile of the part, and how many on its next is
  int ns, skip;   // the request's key tile j0 + i is the part's i-th while that is below ns, else it is j0 + i + skip
  int j0;
  int token, head, r, seq;
  int c0, c1;     // the CTAs of the unit's first and last key tile
  int slot;       // where this CTA's part goes, if the unit is split: 1 if it begins here
  int begins;     // whether it begins in c0's share
  int q0;         // query tiles loaded before
};
constexpr int kAttnItems = 4;

struct AttnSmem {
  uint64_t q_full[2], q_empty[2], kv_full[8], kv_empty[8], s_full[2], p_full[2], o_full[2], turn[2];
  uint64_t raw_full[2], raw_empty[2], q_ready[2], scale_empty[8];
  uint64_t item_full[kAttnItems], item_empty[kAttnItems], drain[2];
  AttnItem item[kAttnItems];
  uint32_t tmem;
  int32_t abort, last;
  int32_t begin_r, begin_head, begin_u, begin_s;
  int64_t warp_cost[16];
  uint8_t bad[16];       // per key tile of the ring: bit i = page i is bad
  float swap[2][128];    // a value of each row, between the two streams
};
static_assert(sizeof(AttnSmem) <= kAttnMiscBytes, "shared memory");
static_assert(AttnCfg<128, false>::kStages <= 8 && AttnCfg<64, false>::kStages <= 8 &&
                  AttnCfg<128, true>::kKStages + AttnCfg<128, true>::kVStages <= 8 &&
                  AttnCfg<128, true>::kVRawStages <= 2 && AttnCfg<128, true>::kScaleTiles <= 8,
              "a barrier for each place of a ring");

// The order in which an item's K and V tiles are loaded, as places in the
// ring: K0 V0 K1 V1 ... where the streams share the tiles, and K0 K1 V0 K2 V1
// K3 ... where they alternate (each stream's next K ahead of its V).
__device__ __forceinline__ uint32_t attn_k_place(int step, int j) {
  return step == 1 || j == 0 ? 2 * j : 2 * j - 1;
}
__device__ __forceinline__ uint32_t attn_v_place(int step, int j, int n) {
  return step == 1 || j + 1 == n ? 2 * j + 1 : 2 * j + 2;
}

// tensor-memory columns of stream x
__device__ __forceinline__ uint32_t attn_col_s(int x) { return (uint32_t)x * 128; }
__device__ __forceinline__ uint32_t attn_col_o(int x) { return 256u + (uint32_t)x * 128; }

// A bounded wait as small as it can be: the kernel has some thirty, and its
// code has to stay in the instruction caches (a limit that is no constant made
// the long decode 494 us of 466).
__device__ __forceinline__ bool attn_wait(uint32_t bar, uint32_t parity, const volatile int* abort_flag,
                                          uint32_t limit = kWaitLimit) {
#pragma unroll 1
  for (uint32_t i = 0; i < limit; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 255u) == 255u && abort_flag && *abort_flag) return false;
  }
  return false;
}
// Once a role's wait has given up all others' follow, so an item in work is
// done with, one way or the other, long before the walking warp's wait for its
// place runs out; and that warp hands out an item, or ends, long before the
// waits for an item do.  (These have to agree: the softmax warps meet at
// barriers.)
constexpr uint32_t kAttnWalkLimit = 16 * kWaitLimit, kAttnItemLimit = 64 * kWaitLimit;

// a / b for 0 <= a < 2^52, 0 < b: in 32 bits where both fit (any batch but one
// of days of work), else by way of FP64, whose quotient is off by one at most
// (the compiler's division of 64-bit integers is a hundred instructions, and
// this card's FP64 has long latencies).
__device__ __forceinline__ int64_t attn_divide(int64_t a, int64_t b) {
  if ((uint64_t)(a | b) >> 32 == 0) return (uint32_t)a / (uint32_t)b;
  int64_t q = (int64_t)((double)a / (double)b);
  if (q * b > a) --q;
  if ((q + 1) * b <= a) ++q;
  return q;
}

// Finds where this CTA's share of the work begins: every CTA sums the
// requests' costs itself (a thread per request, a warp together for requests
// of several units).  Called by all threads; the result is in shared memory.
__device__ __forceinline__ void attn_locate(const AttnParams& p, AttnSmem* sm, int* len, int* share_out) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int threads = (int)blockDim.x, per = (p.R + threads - 1) / threads;
  // (one request a thread: neighbours in different warps, which have to sum the
  // requests of several units one after the other)
  const int r0 = per > 1 ? threadIdx.x * per : lane * (threads / 32) + warp;
  extern __shared__ __align__(1024) unsigned char attn_smem[];
  int64_t* const costs = reinterpret_cast<int64_t*>(attn_smem);  // (before anything else is there)
  // cost of request r; lanes of a warp call it together
  auto cost = [&](int r, bool* bad) -> int64_t {
    int row0 = 0, q = 0, seq = 0;
    if (r < p.R && !attn_request(p, r, &row0, &q, &seq)) *bad = true;
    const int nu = attn_units(p, q);
    int64_t c = 0;
    if (nu == 1) {
      c = (int64_t)attn_unit(p, q, seq, 0, p.Hkv - 1).cost() * p.Hkv;
      if (attn_pairs(p, q)) c = (int64_t)attn_unit(p, q, seq, 0, 0).cost() * (p.Hkv / 2) + c / p.Hkv * (p.Hkv & 1);
    }
    uint32_t many = __ballot_sync(0xffffffffu, nu > 1);
    while (many) {
      const int src = __ffs(many) - 1;
      many &= many - 1;
      const int q_s = __shfl_sync(0xffffffffu, q, src), seq_s = __shfl_sync(0xffffffffu, seq, src);
      const int nu_s = __shfl_sync(0xffffffffu, nu, src);
      int64_t sum = 0;
      for (int u = lane; u < nu_s; u += 32) sum += attn_unit(p, q_s, seq_s, u, 0).cost();
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (lane == src) c = sum * p.Hkv;
    }
    return c;
  };
  // the sum first, then, in the warp of the share's first request, its place
  bool bad = false, mine = false;
  int64_t sum = 0, before = 0, total = 0, share = 0, x0 = 0, at = 0, cost_found = 0;
  int found = -1;
#pragma unroll 1
  for (int phase = 0; phase < 2; ++phase) {
#pragma unroll 1
    for (int i = 0; i < per; ++i) {
      const int64_t c = cost(r0 + i, &bad);
      if (phase == 0) {
        sum += c;
      } else {
        if (mine && found < 0 && x0 < at + c) {
          found = r0 + i;
          cost_found = c;
        }
        if (found < 0) at += c;
      }
    }
    if (phase == 1) break;
    if (per == 1) {
      costs[r0] = sum;
      __syncthreads();
      sum = costs[threadIdx.x];
      fence_proxy_async_smem();  // (a query tile is loaded there)
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
    before = inc - sum;
#pragma unroll 1
    for (int w = 0; w < threads / 32; ++w) {
      if (w < warp) before += sm->warp_cost[w];
      total += sm->warp_cost[w];
    }
    // shares of at least 4 single tiles: a split costs a unit's set-up and a merge
    share = max(attn_divide(total + gridDim.x - 1, gridDim.x), (int64_t)4);
    if (share > kAttnMaxShare) {
      if (threadIdx.x == 0 && blockIdx.x == 0) raise_status(p.status, kStatusBadMetadata);
      share = kAttnMaxShare;
    }
    x0 = (int64_t)blockIdx.x * share;
    *share_out = (int)share;
    *len = (int)max(min(share, total - x0), (int64_t)0);
    mine = x0 < total && before <= x0 && x0 < before + sum;
    at = before;
    if (per == 1) {
      found = threadIdx.x;
      cost_found = sum;
    }
    if (per == 1 || !__any_sync(0xffffffffu, mine)) break;
  }
  if (__any_sync(0xffffffffu, mine)) {
    const int src = __ffs(__ballot_sync(0xffffffffu, mine)) - 1;
    const int r = __shfl_sync(0xffffffffu, found, src);
    const int64_t begin = __shfl_sync(0xffffffffu, at, src);
    const int64_t all = __shfl_sync(0xffffffffu, cost_found, src);
    int row0, q, seq;
    attn_request(p, r, &row0, &q, &seq);
    const bool pairs = attn_pairs(p, q);
    const int64_t per_head = pairs ? attn_unit(p, q, seq, 0, 0).cost() : attn_divide(all, p.Hkv);
    const int at_head = (int)attn_divide(x0 - begin, per_head), head = at_head * (pairs ? 2 : 1);
    int64_t s = begin + at_head * per_head;
    const int nu = attn_units(p, q);
    for (int u0 = 0; u0 < nu; u0 += 32) {
      int64_t c = 0;
      if (u0 + lane < nu) {
        c = attn_unit(p, q, seq, u0 + lane, head).cost();
      }
      int64_t end = c;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, end, o);
        if (lane >= o) end += y;
      }
      const uint32_t past = __ballot_sync(0xffffffffu, c > 0 && x0 < s + end);
      if (past) {
        if (lane == __ffs(past) - 1) {
          sm->begin_r = r;
          sm->begin_head = head;
          sm->begin_u = u0 + lane;
          sm->begin_s = (int)(s + end - c - x0);
        }
        break;
      }
      s += __shfl_sync(0xffffffffu, end, 31);
    }
  }
}

template <bool BF16>
__device__ __forceinline__ uint32_t attn_pack(float lo, float hi) {
  if (BF16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Four E4M3 codes as BF16, exactly (through FP16, which holds them all).
__device__ __forceinline__ void e4m3_to_bf16(uint32_t codes, uint32_t* lo, uint32_t* hi) {
  const __half2_raw a = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(codes & 0xFFFFu), __NV_E4M3);
  const __half2_raw b = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(codes >> 16), __NV_E4M3);
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&a));
  const float2 g = __half22float2(*reinterpret_cast<const __half2*>(&b));
  *lo = attn_pack<true>(f.x, f.y);
  *hi = attn_pack<true>(g.x, g.y);
}

// Which of 32 keys a row sees, as bits: key i of them lies i - `back` tokens
// after the row's own, and `first` is the first one's position.
__device__ __forceinline__ uint32_t attn_seen(const AttnParams& p, int back, int first, bool gone) {
  auto below = [](int n) -> uint32_t { return n <= 0 ? 0u : n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u; };  // bits [0, n)
  uint32_t seen = p.window > 0 ? ~below(back - p.window + 1) | below(p.sinks - first) : 0xFFFFFFFFu;
  if (back < 32) seen &= below(back + 1);
  return gone ? 0u : seen;
}

// Keys of the tile at position s0 that lie between the first tokens and the
// window of a unit's first row, at position p0: [from, to), as places in the
// tile.  No row of the unit sees them, so they may hold anything; whole pages
// of them are never loaded.
__device__ __forceinline__ void attn_hidden(const AttnParams& p, int p0, int s0, int* from, int* to) {
  *from = min(max(p.sinks - s0, 0), kAttnTile);
  *to = p.window > 0 ? min(max(max(p0 - p.window + 1, 0) - s0, 0), kAttnTile) : 0;
}

// E4M3 caches: a row's scores at `base` times their keys' scales, then -inf over
// those that the row, at `pos`, does not see.  In that order: the scale of a
// hidden key may be anything, and that of a key which other rows see 0 or
// negative.  What follows takes scales of 1 for such a tile.  Few tiles come
// here, and code that stands among the softmax loops costs every tile (inlined
// with 32 scores at a time 486 us for the long decode, so 470).
__device__ __noinline__ void attn_scale_and_mask(const AttnParams& p, uint32_t base, const ulonglong2* k_scale,
                                                 int from_key, int to_key, int pos, int s0, uint32_t bad) {
#pragma unroll 1
  for (int c = from_key; c < to_key; c += 16) {
    uint32_t v[16];
    tmem_ld<16>(base + c, v);
    const uint32_t seen = attn_seen(p, pos - s0 - c, s0 + c, bad >> (c / 64) & 1u);
    tmem_ld_wait16(v);
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      const ulonglong2 ks = k_scale[(c + i) / 4];
      const float2 z0 = unpack2(mul2(pack2(__uint_as_float(v[i]), __uint_as_float(v[i + 1])), ks.x));
      const float2 z1 = unpack2(mul2(pack2(__uint_as_float(v[i + 2]), __uint_as_float(v[i + 3])), ks.y));
      v[i] = seen >> i & 1u ? __float_as_uint(z0.x) : 0xFF800000u;
      v[i + 1] = seen >> (i + 1) & 1u ? __float_as_uint(z0.y) : 0xFF800000u;
      v[i + 2] = seen >> (i + 2) & 1u ? __float_as_uint(z1.x) : 0xFF800000u;
      v[i + 3] = seen >> (i + 3) & 1u ? __float_as_uint(z1.y) : 0xFF800000u;
    }
    tmem_st<16>(base + c, v);
  }
  tmem_st_wait();
}

// Zeros over the scales of the values of a tile that no row of the item at `at`
// sees: between the first tokens and the window, past the unit's end, in bad
// pages.  They may be anything (those of pages that are not loaded are what
// another tile left there), and 0 * NaN would spoil the probabilities.  A warp
// does it together before it reads them; all that do write the same.
__device__ __noinline__ void attn_hide_scales(const AttnParams& p, uint32_t at, uint32_t scales, int s0, uint32_t bad) {
  const int p0 = (int)lds_u32(at + (uint32_t)offsetof(AttnItem, p0));
  const int end = p0 + (int)lds_u32(at + (uint32_t)offsetof(AttnItem, ntok)) - s0;
  int from, to;
  attn_hidden(p, p0, s0, &from, &to);
  for (int i = lane_id(); i < kAttnTile; i += 32)
    if (i >= end || (i >= from && i < to) || (bad >> (i / kPageTokens) & 1u)) sts_u32(scales + 4 * i, 0u);
  fence_proxy_async_smem();
  __syncwarp();
}

// The pages of an item's key tiles, looked up by a warp 16 tiles ahead, a pair
// of lanes for each tile.
struct AttnPages {
  const int32_t* bt;
  int j0, ns, skip, keys, first, last;  // first window position, last position that some row sees
  int here, ahead;

  // the id of this lane's page for tile key + lane / 2: the pool's end (zeros)
  // for a page that no row sees, -1 for a bad one
  __device__ __forceinline__ int look(const AttnParams& p, int key) const {
    const int lane = lane_id(), i = key + (lane >> 1), jj = j0 + i;
    if (i >= keys) return 0;
    const int b = (jj < ns ? jj : jj + skip) * 2 + (lane & 1);
    const int64_t t0 = (int64_t)b * kPageTokens;
    if (t0 > last || !(t0 + kPageTokens > first || t0 < p.sinks)) return (int)p.num_pages;
    const int id = __ldg(bt + b);
    if (id < 0 || id >= p.num_pages) {
      raise_status(p.status, kStatusBadPage);
      return -1;
    }
    return id;
  }
  __device__ __forceinline__ void begin(const AttnParams& p, uint32_t at, int n) {
    auto field = [&](size_t offset) { return (int)lds_u32(at + (uint32_t)offset); };
    const int p0 = field(offsetof(AttnItem, p0));
    bt = p.block_table + (int64_t)field(offsetof(AttnItem, r)) * p.max_blocks;
    j0 = field(offsetof(AttnItem, j0));
    ns = field(offsetof(AttnItem, ns));
    skip = field(offsetof(AttnItem, skip));
    keys = n >> (field(offsetof(AttnItem, kind)) == kTwoHeads);
    first = p.window > 0 ? max(0, p0 - p.window + 1) : 0;
    last = p0 + field(offsetof(AttnItem, ntok)) - 1;
    here = look(p, 0);
    ahead = look(p, 16);
  }
  // both pages of key tile `key`, asked for in order (several times if need be)
  __device__ __forceinline__ void get(const AttnParams& p, int key, bool again, int* a, int* b) {
    if (key > 0 && (key & 15) == 0 && !again) {
      here = ahead;
      ahead = look(p, key + 16);
    }
    *a = __shfl_sync(0xffffffffu, here, (key & 15) * 2);
    *b = __shfl_sync(0xffffffffu, here, (key & 15) * 2 + 1);
  }
};

// Four columns of a row's output in a CTA's slot (four of all rows next to each
// other, so that threads with a row each write and read them together).
template <int DP>
__device__ __forceinline__ float4* attn_part(const AttnParams& p, int slot, int row, int c4) {
  return reinterpret_cast<float4*>(p.part) + (uint32_t)(slot * (DP / 4) + c4) * 256 + row;
}

// Joins parts of a unit, in order.  Of few rows each warp of the streams that
// had a row has a part of its own.
//   kJoinWarps  those of this CTA's warps
//   kJoinGroup  of a unit split over many CTAs: those of this CTA's group
//   kJoinUnit   the unit's: those of its CTAs' warps, of its CTAs, or of their
//               groups, whichever come to at most kAttnUngrouped
// into the output, or (where that is not all of the unit) into the first one's
// place.  A CTA's parts lie in its slot 1 if the unit begins in its share, else
// in slot 0.  A thread has a row, and every so many-th four columns of it: with
// few rows several threads share one.  Bound by the latency of its loads (a
// thread has N of a part under way, or one of four parts), and by that of its
// own code: it runs a few times in a call, so its loops stay small.
enum AttnJoin : int { kJoinWarps, kJoinGroup, kJoinUnit };
// log2 of a CTA's parts
__device__ __forceinline__ int attn_lg_parts(int few, int kind) { return few ? (kind == kOneTile ? 3 : 2) : 0; }
template <int DP, bool BF16, int N>
__device__ __noinline__ void attn_join_rows(const AttnParams& p, const AttnItem& item, int what, int all, int lg_pad) {
  const int ctas = item.c1 - item.c0 + 1, mine = (int)blockIdx.x - item.c0;
  const int lg_all = attn_lg_parts(item.few, item.kind);
  const int lg = what == kJoinWarps || (what == kJoinUnit && ctas << lg_all <= kAttnUngrouped) ? lg_all : 0;
  const int step = what == kJoinUnit && ctas > kAttnUngrouped ? kAttnGroup : 1;
  const int first = what == kJoinWarps ? mine : what == kJoinGroup ? mine / kAttnGroup * kAttnGroup : 0;
  const int parts = (what == kJoinWarps   ? 1
                     : what == kJoinGroup ? min(kAttnGroup, ctas - first)
                                          : (ctas + step - 1) / step) << lg;
  const bool into_part = what == kJoinGroup || (what == kJoinWarps && ctas > 1);
  const int rows0 = min(item.ntok, p.tile_tokens) * p.group;  // rows of the first tile
  const int i = threadIdx.x & ((1 << lg_pad) - 1), c0 = threadIdx.x >> lg_pad, per = kAttnSoftmaxWarps * 32 >> lg_pad;
  const int row = i >= rows0 ? 128 + i - rows0 : i;
  // a part's place among the maxima and sums, [slot][256]; its outputs' is
  // [slot][DP / 4][256]
  auto place = [&](int k) -> uint32_t {
    const int cta = first + (k >> lg) * step;
    return (uint32_t)((item.c0 + cta) * 2 + (cta == 0 && item.begins ? 1 : 0)) * 256 + row + (k & ((1 << lg) - 1)) * 32;
  };
  auto outputs = [&](uint32_t at) {
    return reinterpret_cast<float4*>(p.part) + (at & ~255u) * (DP / 4) + (at & 255u);
  };
  float top = -INFINITY, sum = 0.f;
  if (i < all) {
    const bool other_head = item.kind == kTwoHeads && i >= rows0;
    const int q = other_head ? i - rows0 : i;
    const int64_t t = item.token + q / p.group;
    const int h = (item.head + other_head) * p.group + q % p.group;
    uint16_t* const out = p.out + t * p.out_token + (int64_t)h * p.out_head;
#pragma unroll 1
    for (int c = c0; c < p.D / 4; c += N * per) {
      float4 acc[N];
#pragma unroll
      for (int n = 0; n < N; ++n) acc[n] = make_float4(0.f, 0.f, 0.f, 0.f);
      top = -INFINITY;
      sum = 0.f;
#pragma unroll(N == 1 ? 4 : 1)
      for (int k = 0; k < parts; ++k) {
        const uint32_t at = place(k);
        const float2 ml = __ldcg(p.part_ml + at);
        const float4* src = outputs(at) + c * 256;
        float4 v[N];
#pragma unroll
        for (int n = 0; n < N; ++n)
          v[n] = c + n * per < p.D / 4 ? __ldcg(src + n * per * 256) : make_float4(0.f, 0.f, 0.f, 0.f);
        const float t = fmaxf(top, ml.x);
        const float a = t == -INFINITY ? 0.f : ex2(top - t), b = t == -INFINITY ? 0.f : ex2(ml.x - t);
        top = t;
        sum = sum * a + ml.y * b;
#pragma unroll
        for (int n = 0; n < N; ++n) {
          acc[n].x = acc[n].x * a + v[n].x * b;
          acc[n].y = acc[n].y * a + v[n].y * b;
          acc[n].z = acc[n].z * a + v[n].z * b;
          acc[n].w = acc[n].w * a + v[n].w * b;
        }
      }
      const float r = into_part ? 1.0f : sum > 0.f ? 1.0f / sum : 0.f;
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const int at = c + n * per;
        if (at >= p.D / 4) break;
        if (into_part)
          __stcg(outputs(place(0)) + at * 256, acc[n]);
        else
          *reinterpret_cast<uint2*>(out + at * 4) = make_uint2(attn_pack<BF16>(acc[n].x * r, acc[n].y * r),
                                                               attn_pack<BF16>(acc[n].z * r, acc[n].w * r));
      }
    }
    if (!into_part && c0 == 0 && p.lse)
      p.lse[t * p.Hq + h] = sum > 0.f ? (top + log2f(sum)) * 0.69314718055994531f : -INFINITY;
  }
  if (into_part) {  // (once no thread of the row reads the first part's any more)
    named_bar_sync(1, kAttnSoftmaxWarps * 32);
    if (i < all && c0 == 0) __stcg(p.part_ml + place(0), make_float2(top, sum));
  }
}
template <int DP, bool BF16>
__device__ __forceinline__ void attn_join(const AttnParams& p, const AttnItem& item, int what) {
  const int rows0 = min(item.ntok, p.tile_tokens) * p.group;
  const int all = item.kind == kTwoHeads ? 2 * rows0 : item.ntok * p.group;
  const int lg_pad = 32 - __clz(all - 1);
  if (lg_pad <= 4)
    attn_join_rows<DP, BF16, 1>(p, item, what, all, lg_pad);
  else
    attn_join_rows<DP, BF16, 8>(p, item, what, all, lg_pad);
}

// One CTA to an SM, each with an equal share of the work (AttnWalk): whatever
// the batch, all SMs end together, and a unit that lies across a share's end is
// joined by the last of its CTAs to arrive.
//
// Two streams of 128 query rows run side by side, each with its own score and
// output tiles in tensor memory (S, which its probabilities overwrite, and O:
// 2 x 256 columns, all of it) and its own softmax warps, so that the tensor
// core works on one stream while the other's softmax runs.  Rows are the query
// heads of a key head, for as many tokens as fit: a page is read once for all
// of them.  A unit of two query tiles gives each stream one tile, and both read
// the same K and V tiles; one of two key heads gives each stream one head; one
// of a single query tile gives both streams that tile and alternate key tiles:
// the two halves are joined at the end, in tensor memory.
//   warps 0-7   softmax, four for each stream, a thread to a row: the tile's
//               probabilities are taken over the maximum so far in one pass
//               over S, and only where a row's sum shows that this maximum was
//               far too low is the tile taken again over its own (the output
//               so far is scaled then, and only then); the row's sum and
//               maximum in FP32;
//   warp 8      walking: the CTA's share of the work, unit by unit, handed to
//               the others through a ring of four items; V of an E4M3 cache;
//   warps 9, 10 MMA, one for each stream in strict turns: S = Q K^T, O += P V
//               (P from tensor memory);
//   warp 11     TMA: query tiles, K and V tiles through the block table, and
//               zeros in the rows that belong to no valid request;
//   warps 12-15 E4M3 caches: queries into two E4M3 terms, V's codes to BF16.
// E4M3 caches: K's codes go to the tensor core as they are, with each query row
// as two E4M3 terms over a power of two (two 8-bit products cost what one of 16
// bits does; converting K as well took 896 us instead of 790 for four requests
// of 231,000 tokens); a key's scale is applied to its scores and its value's to
// its probabilities.  Few rows over many tiles: kAttnFewTiles.
//
// What bounds it, measured: prefill (8192 tokens after 16,384, 32 heads of 128)
// 1883 us, 1460 TFLOP/s: the tensor core is busy for 77 % of what a library
// product reaches, the rest is the streams' first and last tiles and their
// turns; batched decode of 64 requests (1K to 8K, 16 bits) 197 to 202 us, 6.1
// TB/s, by HBM; long decode over an E4M3 cache (4 x 231,000) 463 us, 4.4 TB/s: by
// the chain of scores, softmax, probabilities and output of each stream, 2.5 us
// for a key tile, of which two run side by side; prompts over an E4M3 cache (8192
// tokens 1010 us) by the softmax, which reads a tile's scores twice and applies
// the scales each time; short prompts (16 of up to 300 tokens 57 us, one of 2000
// 71) by units that shares cut and that are joined; one request of 1024 tokens
// 20 us, launch, set-up and the latency of each step, the kernel's own code
// (115 KB, 155 KB with conversions) among them: hence rolled loops.
template <int DP, bool BF16, bool FP8>
__global__ void __launch_bounds__((AttnCfg<DP, FP8>::kThreads), 1)
    paged_attention_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tq32,
                           const __grid_constant__ CUtensorMap tk,
                           const __grid_constant__ CUtensorMap tv, const __grid_constant__ AttnParams p) {
  using C = AttnCfg<DP, FP8>;
  extern __shared__ __align__(1024) unsigned char attn_smem[];
  const uint32_t q_s = smem_u32(attn_smem) + C::kQ, kv_s = smem_u32(attn_smem) + C::kKv;
  const uint32_t scale_s = smem_u32(attn_smem) + C::kScale, factor_s = scale_s + C::kScaleTiles * 1024;
  AttnSmem* sm = reinterpret_cast<AttnSmem*>(attn_smem + C::kMisc);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&sm->q_full[i]), 1);
      mbar_init(smem_u32(&sm->q_empty[i]), 2 + (FP8 ? kAttnSoftmaxWarps : 0));  // an arrival from each stream
      mbar_init(smem_u32(&sm->s_full[i]), 1);
      mbar_init(smem_u32(&sm->p_full[i]), 4);
      mbar_init(smem_u32(&sm->o_full[i]), 1);
      mbar_init(smem_u32(&sm->turn[i]), 1);
    }
    // (E4M3 caches: K's ring, then that of V as BF16, which four warps fill)
    for (int i = 0; i < 8; ++i) {
      mbar_init(smem_u32(&sm->kv_full[i]), FP8 && i >= C::kKStages ? 4 : 1);
      mbar_init(smem_u32(&sm->kv_empty[i]), 2);
      mbar_init(smem_u32(&sm->scale_empty[i]), 2);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&sm->raw_full[i]), 1);
      mbar_init(smem_u32(&sm->raw_empty[i]), 4);
      mbar_init(smem_u32(&sm->q_ready[i]), 4);
    }
    for (int i = 0; i < kAttnItems; ++i) {
      mbar_init(smem_u32(&sm->item_full[i]), 1);
      mbar_init(smem_u32(&sm->item_empty[i]), kAttnSoftmaxWarps + 3 + (FP8 ? 4 : 0));
    }
    mbar_init(smem_u32(&sm->drain[0]), 1);
    mbar_init(smem_u32(&sm->drain[1]), 1);
    sm->abort = 0;
    fence_barrier_init();
  }
  if (warp == kAttnMmaWarp) {
    tmem_alloc(smem_u32(&sm->tmem), 512);
    tmem_relinquish();
  }
  if (warp == kAttnTmaWarp && lane == 0) {
    tma_prefetch_desc(&tq);
    tma_prefetch_desc(&tq32);
    tma_prefetch_desc(&tk);
    tma_prefetch_desc(&tv);
  }
  if (FP8 && threadIdx.x < 128) sts_u32(smem_u32(attn_smem) + C::kOnes + 4 * threadIdx.x, __float_as_uint(1.0f));
  int len, share;
  attn_locate(p, sm, &len, &share);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm->tmem;
  volatile int* abort_flag = &sm->abort;
  bool ok = true;
  // warp-uniform waits; after one gave up the role ends (the softmax warps,
  // which meet at barriers, go on to the items' end without waiting) and gives
  // no place of a ring back
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (ok) {
      ok = __all_sync(0xffffffffu, attn_wait(smem_u32(bar), parity, abort_flag));
      if (!ok) *abort_flag = 1;
    }
    return ok;
  };
  // a field of the item at `at`: read where it is needed, not kept in registers
#define ATTN_AT(base, field) ((int)lds_u32((base) + (uint32_t)offsetof(AttnItem, field)))
#define ATTN_ITEM(field) ATTN_AT(at, field)

  if (warp < kAttnSoftmaxWarps) {
    // ================================================================ softmax
    if (FP8) regs_grow<C::kSoftmaxRegs>();
    const int x = warp >> 2;                            // stream
    const int tile_row = (warp & 3) * 32 + lane;        // row of its tile
    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    // E4M3 caches: a query tile's slot is free once its rows' factors are read, too
    auto factor_read = [&](uint32_t at) {
      __syncwarp();
      if (lane == 0 && ok) {
        const uint32_t q0 = ATTN_ITEM(q0);
        mbar_arrive(smem_u32(&sm->q_empty[q0 & 1]));
        if (ATTN_ITEM(kind) != kOneTile) mbar_arrive(smem_u32(&sm->q_empty[~q0 & 1]));
      }
    };
    uint32_t n_s = 0, n_o = 0, tile0 = 0;  // score and output tiles so far; key tiles before this item
    for (uint32_t it = 0;; ++it) {
      const uint32_t at = smem_u32(&sm->item[it % kAttnItems]);
      if (!attn_wait(smem_u32(&sm->item_full[it % kAttnItems]), (it / kAttnItems) & 1, nullptr, kAttnItemLimit)) break;
      const int n = ATTN_ITEM(n);
      if (n == 0) break;
      float m = -INFINITY, l = 0.f;
      {
        const uint32_t mine = at + 4 * x;
        const int lo = ATTN_AT(mine, lo), hi = ATTN_AT(mine, hi), step = ATTN_ITEM(step);
        const bool few = FP8 && ATTN_ITEM(few);
        const int row = few ? lane : tile_row;
        const int from_key = few ? tile_row - lane : 0, to_key = few ? from_key + 32 : kAttnTile;  // this warp's keys
        const bool live = row - lane < (hi - lo + 1) * p.group;  // some row of this warp is real
        const bool real = row < (hi - lo + 1) * p.group;  // (the others hold whatever was there: they decide nothing)
        const int pos = min(lo + row / p.group, hi);
        const int ns = ATTN_ITEM(ns), skip = ATTN_ITEM(skip), j0 = ATTN_ITEM(j0);
        const int heads = ATTN_ITEM(kind) == kTwoHeads;
        float factor = p.scale_log2;  // of the row's scores
        for (int j = ATTN_AT(mine, from); j < n; j += step) {
          const int jj = j0 + (j >> heads), s0 = (jj + (jj < ns ? 0 : skip)) * kAttnTile;
          const bool inner = s0 + kAttnTile - 1 <= lo && (p.window == 0 || s0 > hi - p.window || s0 + kAttnTile - 1 < p.sinks);
          wait(&sm->s_full[x], n_s & 1);
          ++n_s;
          // The scores' arrival says that K's tile is done with, too: the fourth
          // warp, which with few rows is not the slowest, gives it back instead of
          // a commit (475 -> 468 us for four requests of 231,000; 16-bit caches,
          // whose softmax is the longer part, lose by it: 1885 -> 1976 us for 8192
          // tokens after 16,384).
          if (FP8 && ok && lane == 0 && (warp & 3) == 3) mbar_arrive(smem_u32(&sm->kv_empty[(tile0 + j) % C::kKStages]));
          if (FP8 && j == ATTN_AT(mine, from)) {
            const uint32_t q = ATTN_ITEM(q0) + (ATTN_ITEM(kind) != kOneTile ? x : 0);
            // (not 0, however small the row's elements: it multiplies -inf)
            factor = fmaxf(p.scale_log2 * __uint_as_float(lds_u32(factor_s + ((q & 1) * 128 + row) * 4)), 0x1p-126f);
            factor_read(at);
          }
          if (live) {
            tc_fence_after();
            const uint32_t base = lanes + attn_col_s(x);
            const uint32_t bad = sm->bad[(tile0 + j) & 15];
            // E4M3 caches: this tile's scales
            const ulonglong2* k_scale = reinterpret_cast<const ulonglong2*>(attn_smem + C::kScale + ((tile0 + j) & 7) * 1024);
            const ulonglong2* const v_scale = k_scale + 32;
            if (!(inner && bad == 0)) {
              // -inf over the scores that the row does not see
              if constexpr (FP8) {
                attn_hide_scales(p, at, scale_s + ((tile0 + j) & 7) * 1024 + 512, s0, bad);
                attn_scale_and_mask(p, base, k_scale, from_key, to_key, pos, s0, bad);
                k_scale = reinterpret_cast<const ulonglong2*>(attn_smem + C::kOnes);
              } else {
#pragma unroll 1
                for (int c = from_key; c < to_key; c += 32) {
                  uint32_t v[32];
                  tmem_ld<32>(base + c, v);
                  const uint32_t seen = attn_seen(p, pos - s0 - c, s0 + c, bad >> (c / 64) & 1u);
                  tmem_ld_wait32(v);
#pragma unroll
                  for (int i = 0; i < 32; ++i) v[i] = seen & (1u << i) ? v[i] : 0xFF800000u;
                  tmem_st<32>(base + c, v);
                }
                tmem_st_wait();
              }
            }
            // the scores' maximum
            auto maximum = [&]() {
              float top = -INFINITY;
#pragma unroll 1
              for (int c = from_key; c < to_key; c += 32) {
                uint32_t v[32];
                tmem_ld<32>(base + c, v);
                tmem_ld_wait32(v);
#pragma unroll
                for (int i = 0; i < 32; i += 4) {
                  float a = __uint_as_float(v[i]), b = __uint_as_float(v[i + 1]);
                  float d = __uint_as_float(v[i + 2]), g = __uint_as_float(v[i + 3]);
                  if (FP8) {
                    const ulonglong2 ks = k_scale[(c + i) / 4];
                    const float2 z0 = unpack2(mul2(pack2(a, b), ks.x)), z1 = unpack2(mul2(pack2(d, g), ks.y));
                    a = z0.x, b = z0.y, d = z1.x, g = z1.y;
                  }
                  top = max3(max3(top, a, b), d, g);
                }
              }
              return top * factor;
            };
            // the row's m becomes that of the maximum `highest` where that is
            // larger and `wanted`
            auto raise = [&](float highest, bool wanted) {
              const float top = highest - attn_lift<BF16>();
              const bool grow = wanted && top > m;
              if (__any_sync(0xffffffffu, m != -INFINITY)) {  // (else there is no output yet, or zeros)
                // the scores' arrival says that the stream's previous product is done
                const float a = grow && m != -INFINITY ? ex2(m - top) : 1.0f;
#pragma unroll 1
                for (int c = 0; c < DP; c += 32) {
                  uint32_t o[32];
                  tmem_ld<32>(lanes + attn_col_o(x) + c, o);
                  tmem_ld_wait32(o);
#pragma unroll
                  for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * a);
                  tmem_st<32>(lanes + attn_col_o(x) + c, o);
                }
                l *= a;
              }
              if (grow) m = top;
            };
            // probabilities of the 32 keys at c: packed, and added to sums
            uint64_t sums[2];
            auto probabilities = [&](int c, uint32_t* pr) {
              const float shift = m == -INFINITY ? 0.f : -m;
              const uint64_t mul = pack2(factor, factor), sub = pack2(shift, shift);
              uint32_t v[32];
              tmem_ld<32>(base + c, v);
              tmem_ld_wait32(v);
#pragma unroll
              for (int i = 0; i < 32; i += 4) {
                ulonglong2 ks = make_ulonglong2(mul, mul);
                if (FP8) {
                  ks = k_scale[(c + i) / 4];
                  ks.x = mul2(ks.x, mul);
                  ks.y = mul2(ks.y, mul);
                }
                const float2 z0 = unpack2(fma2(pack2(__uint_as_float(v[i]), __uint_as_float(v[i + 1])), ks.x, sub));
                const float2 z1 = unpack2(fma2(pack2(__uint_as_float(v[i + 2]), __uint_as_float(v[i + 3])), ks.y, sub));
                uint64_t e0 = pack2(ex2(z0.x), ex2(z0.y)), e1 = pack2(ex2(z1.x), ex2(z1.y));
                sums[0] = add2(sums[0], e0);
                sums[1] = add2(sums[1], e1);
                if (FP8) {
                  const ulonglong2 vs = v_scale[(c + i) / 4];
                  e0 = mul2(e0, vs.x);
                  e1 = mul2(e1, vs.y);
                }
                const float2 p0 = unpack2(e0), p1 = unpack2(e1);
                pr[i / 2] = attn_pack<BF16>(p0.x, p0.y);
                pr[i / 2 + 1] = attn_pack<BF16>(p1.x, p1.y);
              }
            };
            // Probabilities go over scores that this thread has read: those of
            // 64 keys in the first 32 of their columns.
            float sum;
            if constexpr (FP8) {
              // the maximum first, then loops that are not unrolled: with the
              // scales' arithmetic the other form's code (below) is fetched
              // more slowly than it runs (4,400 cycles a tile)
              const float top = maximum();
              const bool low = real && top > m + kAttnRescaleLog2;
              if (__any_sync(0xffffffffu, low)) raise(top, low);
              sums[0] = sums[1] = 0;
#pragma unroll 1
              for (int c = from_key; c < to_key; c += 32) {
                uint32_t pr[16];
                probabilities(c, pr);
                tmem_st<16>(base + (c & 64) + (c & 32) / 2, pr);
              }
              if (few) {
                // zeros for the other warps' keys: this warp's output rows are
                // those of its own keys
                uint32_t zero[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) zero[i] = 0;
#pragma unroll 1
                for (int c = 0; c < kAttnTile; c += 32)
                  if (c != from_key) tmem_st<16>(base + (c & 64) + (c & 32) / 2, zero);
              }
              const float2 t = unpack2(add2(sums[0], sums[1]));
              sum = t.x + t.y;
            } else {
              // One pass with the maximum that the row has: the probabilities
              // stay in registers until their sum says that it will do.  If
              // not (on each row's first tile, and few after it) the row gets
              // the right one first: the scores are still there.
              uint32_t pr[64];
              // Each row by itself, so that its result depends on no other row.
              bool low = real && m == -INFINITY, raised = false;
              for (;;) {
                if (!__any_sync(0xffffffffu, low)) {
                  sums[0] = sums[1] = 0;
#pragma unroll
                  for (int c = 0; c < kAttnTile; c += 32) probabilities(c, pr + c / 2);
                  const float2 t = unpack2(add2(sums[0], sums[1]));
                  sum = t.x + t.y;
                  low = real && !raised && !(sum <= attn_most_sum<BF16>());
                  if (!__any_sync(0xffffffffu, low)) break;
                }
                raise(maximum(), low);
                raised |= low;
                low = false;
              }
              tmem_st<32>(base, pr);
              tmem_st<32>(base + 64, pr + 32);
            }
            l += sum;
            tmem_st_wait();
            tc_fence_before();
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&sm->p_full[x]));
        }
      }
      tile0 += n;

      if (FP8 && ATTN_AT(at + 4 * x, from) >= n) factor_read(at);
      // ---- the unit's end: out = O / l, or the part of a split unit
      const int kind = ATTN_ITEM(kind);
      const bool two = kind != kOneTile;  // each stream has rows of its own
      const int first = kind == kTwoTiles && x ? p.tile_tokens : 0;  // this stream's first token in the unit
      const int rows = min(p.tile_tokens, ATTN_ITEM(ntok) - first) * p.group;
      const bool few = FP8 && ATTN_ITEM(few);
      const int row = few ? lane : tile_row;
      const bool live = row - lane < rows;
      const bool split = ATTN_ITEM(c0) != ATTN_ITEM(c1);
      if (two || x < n) {  // this stream had a tile
        wait(&sm->o_full[x], n_o & 1);
        ++n_o;
      }
      tc_fence_after();
      // which streams have an output, and its factors; where they share the
      // rows, all of their warps split the columns
      float f0 = 1.f, f1 = 1.f;
      // (of few rows each warp has parts of its own, joined as a split unit's are)
      const bool has0 = two || few ? x == 0 : true, has1 = two || few ? x == 1 && (two || n > 1) : n > 1;
      const int cols = two || few ? DP : DP / 2, col0 = two || few ? 0 : x * (DP / 2);
      if (!two && !few) {
        tc_fence_before();
        sm->swap[x][row] = m;
        named_bar_sync(1, kAttnSoftmaxWarps * 32);
        const float a = sm->swap[0][row], b = sm->swap[1][row], mine = m;
        m = fmaxf(a, b);
        f0 = a == -INFINITY ? 0.f : ex2(a - m);
        f1 = b == -INFINITY ? 0.f : ex2(b - m);
        named_bar_sync(1, kAttnSoftmaxWarps * 32);
        sm->swap[x][row] = mine == -INFINITY ? 0.f : l * (x ? f1 : f0);
        named_bar_sync(1, kAttnSoftmaxWarps * 32);
        l = sm->swap[0][row] + sm->swap[1][row];
        tc_fence_after();  // the other stream's output is there: its warps came here after it
      }
      if (live && ok) {
        const int prow = few ? x * 128 + tile_row : two ? x * 128 + row : row;
        const int slot = (int)blockIdx.x * 2 + ATTN_ITEM(slot);
        const int64_t token = ATTN_ITEM(token) + first + row / p.group;
        const int head = (ATTN_ITEM(head) + (kind == kTwoHeads ? x : 0)) * p.group + row % p.group;
        const bool parts = split || few;
        const float inv = parts ? 1.0f : (l > 0.f ? 1.0f / l : 0.f);
        f0 *= inv;
        f1 *= inv;
#pragma unroll 1
        for (int c = col0; c < col0 + cols; c += 16) {
          uint32_t a[16], b[16];
          float o[16];
          if (has0) tmem_ld<16>(lanes + attn_col_o(0) + c, a);
          if (has1) tmem_ld<16>(lanes + attn_col_o(1) + c, b);
          if (has0) tmem_ld_wait16(a);
          if (has1) tmem_ld_wait16(b);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            o[i] = 0.f;
            if (has0) o[i] = __uint_as_float(a[i]) * f0;
            if (has1) o[i] += __uint_as_float(b[i]) * f1;
          }
          if (row < rows && c < p.D) {
            if (parts) {
#pragma unroll
              for (int i = 0; i < 16; i += 4)
                __stcg(attn_part<DP>(p, slot, prow, (c + i) / 4), make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]));
            } else {
              uint4* dst = reinterpret_cast<uint4*>(p.out + token * p.out_token + (int64_t)head * p.out_head + c);
              uint32_t v[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) v[i] = attn_pack<BF16>(o[2 * i], o[2 * i + 1]);
              dst[0] = make_uint4(v[0], v[1], v[2], v[3]);
              dst[1] = make_uint4(v[4], v[5], v[6], v[7]);
            }
          }
        }
        if (row < rows && col0 == 0) {
          if (parts)
            __stcg(p.part_ml + slot * 256 + prow, make_float2(m, l));
          else if (p.lse)
            p.lse[token * p.Hq + head] = l > 0.f ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
        }
      }
      tc_fence_before();
      const int c0 = ATTN_ITEM(c0), ctas = ATTN_ITEM(c1) - c0 + 1;
      if (few && (!split || ctas << attn_lg_parts(1, kind) > kAttnUngrouped)) {
        named_bar_sync(1, kAttnSoftmaxWarps * 32);
        attn_join<DP, BF16>(p, *(const AttnItem*)&sm->item[it % kAttnItems], kJoinWarps);
        // (the parts' places are free for the next unit's)
        if (!split) named_bar_sync(1, kAttnSoftmaxWarps * 32);
      }
      if (split) {
        // the last CTA of a group to arrive, then the last of a unit, joins the
        // parts, in CTA order
        for (int what = ctas > kAttnUngrouped ? kJoinGroup : kJoinUnit; what <= kJoinUnit; ++what) {
          __threadfence();
          named_bar_sync(1, kAttnSoftmaxWarps * 32);
          if (threadIdx.x == 0) {
            const int first = ((int)blockIdx.x - c0) / kAttnGroup * kAttnGroup;
            uint32_t* const count = p.counter + c0 + (what == kJoinUnit ? 0 : kAttnMaxGrid + (first ? kAttnMaxGrid + first : 0));
            const int most = what == kJoinGroup       ? min(kAttnGroup, ctas - first)
                             : ctas > kAttnUngrouped ? (ctas + kAttnGroup - 1) / kAttnGroup
                                                     : ctas;
            const bool all = atomicAdd(count, 1u) == (uint32_t)(most - 1);
            if (all) *count = 0;
            sm->last = all;
          }
          named_bar_sync(1, kAttnSoftmaxWarps * 32);
          if (!*(volatile int*)&sm->last) break;
          __threadfence();
          attn_join<DP, BF16>(p, *(const AttnItem*)&sm->item[it % kAttnItems], what);
        }
      }
      // the other stream's warps may still read this one's output
      if (!two && !few) named_bar_sync(1, kAttnSoftmaxWarps * 32);
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sm->item_empty[it % kAttnItems]));
    }
    if (!ok) raise_status(p.status, kStatusTimeout);
  } else {
    if (FP8) {
      if (warp < kAttnConvertWarp)
        regs_shrink<C::kIssueRegs>();
      else
        regs_shrink<C::kConvertRegs>();
    }
    // every item is taken, also after a wait gave up: the softmax warps go on
    auto each_item = [&](auto& serve) {
      for (uint32_t it = 0;; ++it) {
        const uint32_t at = smem_u32(&sm->item[it % kAttnItems]);
        if (!attn_wait(smem_u32(&sm->item_full[it % kAttnItems]), (it / kAttnItems) & 1, nullptr, kAttnItemLimit)) break;
        const int n = ATTN_ITEM(n);
        if (n == 0) break;
        if (ok) serve(at, n);
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm->item_empty[it % kAttnItems]));
      }
    };
    // E4M3 caches: the next tile of K, with the scales of both, or of V
    uint32_t n_t = 0;  // tiles so far
    auto load8 = [&](bool is_k, int head, int page0, int page1) {
      const uint32_t t = n_t, ring = is_k ? C::kKStages : C::kVRawStages, st = t % ring, round = t / ring;
      if (round > 0) wait(is_k ? &sm->kv_empty[st] : &sm->raw_empty[st], (round - 1) & 1);
      if (is_k && t >= 8) wait(&sm->scale_empty[t & 7], (t / 8 - 1) & 1);
      if (!ok) return;
      const uint32_t bar = smem_u32(is_k ? &sm->kv_full[st] : &sm->raw_full[st]);
      const uint32_t dst = smem_u32(attn_smem) + (is_k ? C::kKv : C::kVRaw) + st * C::kRawBytes;
      const int none = (int)p.num_pages, page = lane & 1 ? page1 : page0;
      const uint32_t held = is_k ? (page0 < none) + (page1 < none) : 0;
      if (lane == 0) mbar_arrive_expect_tx(bar, C::kRawBytes + held * 512);
      __syncwarp();
      if (lane < 2) tma_load_4d(dst + lane * 8192, is_k ? &tk : &tv, 0, head, 0, page, bar);
      if (is_k && lane < 4 && page < none) {
        const int w = lane >> 1;
        bulk_load(scale_s + (t & 7) * 1024 + w * 512 + (lane & 1) * 256,
                  p.scale[w] + (int64_t)head * p.scale_head[w] + page * p.scale_page[w], 256, bar);
      }
      __syncwarp();
      ++n_t;
    };
    auto landed = [&](uint64_t* full, uint32_t n, uint32_t ring) {
      for (uint32_t i = n > ring ? n - ring : 0; i < n; ++i) attn_wait(smem_u32(&full[i % ring]), (i / ring) & 1, nullptr);
    };
    if (warp == kAttnTmaWarp) {
      // ================================================================ TMA
      uint32_t n_kv = 0, n_q = 0, tile0 = 0;
      if (p.give_up) {  // as if its first wait had: nothing is loaded, and all the others' waits end by that
        ok = false;
        *abort_flag = 1;
      }
      // One tile of K or V from its two pages.  With
      // an E4M3 cache K's tile brings the scales of both.
      auto load = [&](const CUtensorMap* map, int head, int page0, int page1) {
        const uint32_t st = n_kv % C::kStages, round = n_kv / C::kStages;
        if (round > 0) wait(&sm->kv_empty[st], (round - 1) & 1);
        if (!ok) return;
        // (a copy costs its issuing thread some 150 cycles: a lane for each)
        const uint32_t bar = smem_u32(&sm->kv_full[st]), dst = kv_s + st * C::kTileBytes;
        if (lane == 0) mbar_arrive_expect_tx(bar, C::kTileBytes);
        __syncwarp();
        if (lane < 2 * C::kHalves)
          tma_load_4d(dst + lane * 8192, map, (lane >> 1) * 64, head, 0, lane & 1 ? page1 : page0, bar);
        __syncwarp();
        ++n_kv;
      };
      // a query tile; of few rows, a box of them
      auto load_q = [&](int head, int token, bool few) {
        const uint32_t st = n_q & 1, round = n_q >> 1;
        if (round > 0) wait(&sm->q_empty[st], (round - 1) & 1);
        if (!ok) return;
        const uint32_t bar = smem_u32(&sm->q_full[st]), dst = q_s + st * C::kTileBytes;
        const int tokens = few ? p.tile_tokens32 : p.tile_tokens;
        if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)(C::kHalves * tokens * p.group * 128));
        __syncwarp();
        if (lane < C::kHalves) tma_load_3d(dst + lane * 16384, few ? &tq32 : &tq, lane * 64, head * p.group, token, bar);
        __syncwarp();
        ++n_q;
      };
      auto serve = [&](uint32_t at, int n) {
        const int kind = ATTN_ITEM(kind), heads = kind == kTwoHeads;
        const int token = ATTN_ITEM(token), head = ATTN_ITEM(head);
        AttnPages pages;
        pages.begin(p, at, n);
        int a0 = 0, a1 = 0, b0 = 0, b1 = 0;  // the newest K tile's pages, and those of the one before
        // tiles in the order in which they are used (attn_k_place, attn_v_place;
        // with E4M3 caches K's alone), the query tiles after the first two
        const int places = FP8 ? n : 2 * n;
#pragma unroll 1
        for (int i = 0; i < places && ok; ++i) {
          bool is_k = FP8 || (i & 1) == 0;
          int j = FP8 ? i : i >> 1;
          if (!FP8 && kind != kTwoTiles) {
            is_k = i == 0 || ((i & 1) && i != 2 * n - 1);
            j = is_k ? (i + 1) >> 1 : i == 2 * n - 1 ? n - 1 : (i >> 1) - 1;
          }
          if (is_k) {
            b0 = a0;
            b1 = a1;
            pages.get(p, j >> heads, j & heads, &a0, &a1);
            if (lane == 0) sm->bad[(tile0 + j) & 15] = (uint8_t)((a0 < 0 ? 1 : 0) | (a1 < 0 ? 2 : 0));
            __syncwarp();
            if (a0 < 0) a0 = (int)p.num_pages;
            if (a1 < 0) a1 = (int)p.num_pages;
          }
          const bool older = !is_k && kind != kTwoTiles && j + 1 < n;  // V's pages are not the newest K's
          const int h = head + (j & heads), page0 = older ? b0 : a0, page1 = older ? b1 : a1;
          if (FP8)
            load8(true, h, page0, page1);
          else
            load(is_k ? &tk : &tv, h, page0, page1);
          const int queries = kind != kOneTile ? 2 : 1;
          for (int k = i; k < queries && (k == i || i + 1 == places); ++k)
            load_q(head + (k & heads), token + (kind == kTwoTiles && k ? p.tile_tokens : 0),
                   ATTN_ITEM(ntok) <= p.tile_tokens32);
        }
        tile0 += n;
      };
      each_item(serve);
      // rows that belong to no valid request
      const int64_t lo = (int64_t)blockIdx.x * p.T / gridDim.x, hi = ((int64_t)blockIdx.x + 1) * p.T / gridDim.x;
      for (int64_t t0 = lo; t0 < hi; t0 += 32) {
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
      // every copy has landed before the CTA leaves
      if (FP8)
        landed(sm->kv_full, n_t, C::kKStages);
      else
        landed(sm->kv_full, n_kv, C::kStages);
      landed(sm->q_full, n_q, 2);
    } else if (warp < kAttnTmaWarp && warp >= kAttnMmaWarp) {
      // ================================================================ MMA
      // A warp for each stream: products run in the order they are issued and
      // hardly ahead of the issuing thread (a pause of 100 cycles in it costs
      // the tensor core 150, a commit 115), so one stream's waits have to fall
      // into the other's products.
      const int x = warp - kAttnMmaWarp;
      const uint32_t id_qk = FP8 ? idesc_e4m3_f32(128, 128) : idesc_16_f32(BF16, 128, 128, false);
      const uint32_t id_pv = idesc_16_f32(BF16, 128, (uint32_t)p.D, true);
      const uint32_t ksteps = FP8 ? (uint32_t)(p.D + 31) / 32 : (uint32_t)p.D / 16;
      uint32_t n_p = 0, kv0 = 0;  // probabilities so far; the ring's place before this item
      // Every place of the rings is waited for, in order, and given back: when
      // the products that read it are done, or at once where the tile is the
      // other stream's.  (A wait on a barrier that may
      // be two phases on, or not yet at the phase before, would be mistaken.)
      uint32_t kv_seen = 0, q_seen = 0;
      auto kv_wait = [&](uint32_t place, int step, int n) {
        while (kv_seen <= place) {
          const uint32_t st = kv_seen % C::kStages;
          if (!wait(&sm->kv_full[st], (kv_seen / C::kStages) & 1)) return false;
          if (step == 2) {
            const int i = (int)(kv_seen - kv0);
            const int j = i == 2 * n - 1 ? n - 1 : i & 1 ? (i + 1) / 2 : max(i / 2 - 1, 0);
            if ((j & 1) != x && lane == 0) mbar_arrive(smem_u32(&sm->kv_empty[st]));
          }
          ++kv_seen;
        }
        return true;
      };
      // E4M3 caches: K's and V's rings have a place for each key tile
      uint32_t t_seen[2] = {0, 0};
      auto tile_wait = [&](int v, uint32_t tile, int step) {
        uint32_t& seen = t_seen[v];
        while (seen <= tile) {
          const uint32_t st = v ? C::kKStages + seen % C::kVStages : seen % C::kKStages;
          if (!wait(&sm->kv_full[st], (seen / (v ? C::kVStages : C::kKStages)) & 1)) return false;
          if (step == 2 && (int)((seen - kv0 / 2) & 1) != x && lane == 0) mbar_arrive(smem_u32(&sm->kv_empty[st]));
          ++seen;
        }
        return true;
      };
      auto q_wait = [&](uint32_t place, uint32_t own) {
        uint64_t* full = FP8 ? sm->q_ready : sm->q_full;
        while (q_seen <= place) {
          if (!wait(&full[q_seen & 1], (q_seen >> 1) & 1)) return false;
          if (q_seen != own && lane == 0) mbar_arrive(smem_u32(&sm->q_empty[q_seen & 1]));
          ++q_seen;
        }
        return true;
      };
      auto commit = [&](uint64_t* bar) {
        if (lane == 0) umma_commit(smem_u32(bar));
      };
      // The streams take turns, a turn being a tile's P V and the next one's
      // Q K^T: left alone, the two warps' products interleave, both end
      // together and the tensor core idles while both softmaxes run.
      uint32_t turns = 0;
      auto take_turn = [&]() {
        const uint32_t i = turns++;
        if (x == 0 && i == 0) return true;
        return wait(&sm->turn[x], (i + x + 1) & 1);
      };
      auto pass_turn = [&]() {
        if (lane == 0) mbar_arrive(smem_u32(&sm->turn[x ^ 1]));
      };
      auto serve = [&](uint32_t at, int n) {
        const int step = ATTN_ITEM(step), from = ATTN_AT(at + 4 * x, from);
        const int kind = ATTN_ITEM(kind), heads = kind == kTwoHeads;
        const uint32_t q0 = ATTN_ITEM(q0), q = q0 + (kind != kOneTile ? x : 0);
        const uint32_t own = from < n ? q : 0xFFFFFFFFu;
        // Values that no row sees may be anything, and 0 * NaN would spoil the
        // sum.  The key tile that holds the request's end inside a page ...
        const int j0 = ATTN_ITEM(j0), ns = ATTN_ITEM(ns), skip = ATTN_ITEM(skip);
        int tail = n, end;
        {
          const int last = j0 + (n >> heads) - 1;
          end = ATTN_ITEM(seq) - (last < ns ? last : last + skip) * kAttnTile;
          if (!FP8 && end < kAttnTile && end % kPageTokens != 0) tail = n - 1 - heads;
        }
        // ... and, with a window, the last tile of the first tokens and the
        // window's first one (the item's key tiles `edge` and `edge` + 1)
        const int edge = p.window > 0 ? ns - 1 - j0 : n;
        const uint32_t tile0 = kv0 / 2;
        // half of Q K^T: 64 of the dimensions, or (E4M3) one of the queries' two terms
        auto qk = [&](int j, int h) {
          const uint32_t q_tile = q_s + (q & 1) * C::kTileBytes + h * 16384;
          if (lane != 0) return;
          if (FP8)
            umma_f8_k128(tmem + attn_col_s(x), sw128_desc(q_tile),
                         sw128_desc(kv_s + (tile0 + j) % C::kKStages * C::kRawBytes), id_qk, h > 0, ksteps);
          else
            umma_f16_k64(tmem + attn_col_s(x), sw128_desc(q_tile),
                         sw128_desc(kv_s + (kv0 + attn_k_place(step, j)) % C::kStages * C::kTileBytes + h * 16384), id_qk,
                         h > 0, ksteps - 4 * h);
        };
        auto k_wait = [&](int j) { return FP8 ? tile_wait(0, tile0 + j, step) : kv_wait(kv0 + attn_k_place(step, j), step, n); };
        auto v_wait = [&](int j) { return FP8 ? tile_wait(1, tile0 + j, step) : kv_wait(kv0 + attn_v_place(step, j, n), step, n); };
        auto v_release = [&](int j) {
          commit(&sm->kv_empty[FP8 ? C::kKStages + (tile0 + j) % C::kVStages : (kv0 + attn_v_place(step, j, n)) % C::kStages]);
        };
        // Round by round: the P V of tile j and the Q K^T of the next; before the
        // first a Q K^T alone, and in the last of an odd n nothing for stream 1.
        bool first = true;
#pragma unroll 1
        for (int j = from - step; j - from < n; j += step, first = false) {
          const bool more = j + step < n, tile = !first && j < n;
          if (first && !q_wait(q, own)) return;  // (no tile for this stream: the places are taken below)
          const uint32_t v_s = FP8 ? smem_u32(attn_smem) + C::kV + (tile0 + j) % C::kVStages * C::kTileBytes
                                   : kv_s + (kv0 + attn_v_place(step, j, n)) % C::kStages * C::kTileBytes;
          if (tile) {
            if (!v_wait(j)) return;
            const bool at_edge = !FP8 && (uint32_t)((j >> heads) - edge) < 2u;
            if (j >= tail || at_edge) {
              // (in shared tiles each stream's warp writes the same zeros)
              auto zeros = [&](int from, int to) {
#pragma unroll 1
                for (int i = from * 8 + lane; i < to * 8; i += 32)
#pragma unroll
                  for (int h = 0; h < C::kHalves; ++h) sts_v4(v_s + h * 16384 + i * 16, make_uint4(0, 0, 0, 0));
              };
              if (j >= tail) zeros(end, end < kPageTokens ? kPageTokens : kAttnTile);
              if (at_edge) {
                const int jj = j0 + (j >> heads);
                int from, to;
                attn_hidden(p, ATTN_ITEM(p0), (jj < ns ? jj : jj + skip) * kAttnTile, &from, &to);
                zeros(from, to);
              }
              fence_proxy_async_smem();
              __syncwarp();
            }
          }
          if (more && !k_wait(j + step)) return;
          if (tile) {
            if (!wait(&sm->p_full[x], n_p & 1)) return;
            ++n_p;
            if (FP8 && lane == 0) {  // the tile's scales have been used
              const uint32_t bar = smem_u32(&sm->scale_empty[(tile0 + j) & 7]);
              mbar_arrive(bar);
              if (step == 2) mbar_arrive(bar);
            }
          }
          if (!first && !take_turn()) return;
          tc_fence_after();
          if (tile && lane == 0)
            umma_f16_ta_k128(tmem + attn_col_o(x), tmem + attn_col_s(x), sw128_desc_mn(v_s, 16384, 1024), id_pv,
                             j > from);
          // the turn passes a few products early: the other warp wakes up meanwhile
#pragma unroll
          for (int h = 0; h < C::kHalves; ++h) {
            if (h == C::kHalves - 1 && !first) pass_turn();
            if (more) qk(j + step, h);
          }
          if (more) {
            commit(&sm->s_full[x]);
            if (!FP8) commit(&sm->kv_empty[(kv0 + attn_k_place(step, j + step)) % C::kStages]);
            if (j + 2 * step >= n) commit(&sm->q_empty[q & 1]);
          } else if (tile) {
            commit(&sm->o_full[x]);
          }
          if (tile) v_release(j);
        }
        if (!q_wait(q0 + (kind != kOneTile ? 1 : 0), own)) return;
        if (!FP8)
          kv_wait(kv0 + 2 * n - 1, step, n);
        else if (tile_wait(0, tile0 + n - 1, step))
          tile_wait(1, tile0 + n - 1, step);
      };
      auto served = [&](uint32_t at, int n) {
        serve(at, n);
        kv0 += 2 * n;
      };
      each_item(served);
      // every product issued has completed before tensor memory is released
      commit(&sm->drain[x]);
      if (!attn_wait(smem_u32(&sm->drain[x]), 0, nullptr)) ok = false;
      if (!ok) {
        sm->abort = 1;
        raise_status(p.status, kStatusTimeout);
      }
    } else if (FP8 && warp >= kAttnConvertWarp) {
      // ================================================================ converting
      const int cw = warp - kAttnConvertWarp, tid = cw * 32 + lane;
      uint32_t tile0 = 0;
      // A query tile in place: each row, scaled by a power of two to a maximum
      // in [128, 256), as the sum of two E4M3 terms (8 significant bits as two
      // times 4: exact but for elements under 2^-9 of the row's maximum, which
      // are off by half of E4M3's smallest step, 2^-10, and so by 2^-17 of it at
      // most).  So Q K^T needs no conversion of K:
      // two products with its codes cost what one in 16 bits does.
      auto split_q = [&](uint32_t place, int rows, int copies) {
        if (!wait(&sm->q_full[place & 1], (place >> 1) & 1)) return false;
        const uint32_t tile = q_s + (place & 1) * C::kTileBytes;
#pragma unroll 2
        for (int r = cw; r < rows; r += 4) {
          // a lane's 4 elements
          const uint2 w = lds_v2(tile + (lane / 16) * 16384 + r * 128 + (((lane % 16 / 2) ^ (r & 7)) << 4) + 8 * (lane & 1));
          float f[4] = {__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u), __uint_as_float(w.y << 16),
                        __uint_as_float(w.y & 0xFFFF0000u)};
          float top = fmaxf(fmaxf(fabsf(f[0]), fabsf(f[1])), fmaxf(fabsf(f[2]), fabsf(f[3])));
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
          const uint32_t e = min(max(__float_as_uint(top) >> 23, 8u), 254u);
          const float up = __uint_as_float((261u - e) << 23);  // 2^(7 - exponent)
          uint32_t c1 = 0, c2 = 0;
#pragma unroll
          for (int i = 0; i < 4; i += 2) {
            const float2 v = make_float2(f[i] * up, f[i + 1] * up);
            const uint32_t a = __nv_cvt_float2_to_fp8x2(v, __NV_SATFINITE, __NV_E4M3);
            const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)a, __NV_E4M3);
            const float2 g = __half22float2(*reinterpret_cast<const __half2*>(&h));
            const uint32_t b = __nv_cvt_float2_to_fp8x2(make_float2(v.x - g.x, v.y - g.y), __NV_SATFINITE, __NV_E4M3);
            c1 |= (a & 0xFFFFu) << (8 * i);
            c2 |= (b & 0xFFFFu) << (8 * i);
          }
          __syncwarp();  // the whole row has been read
          const uint32_t to = tile + r * 128 + (((lane / 4) ^ (r & 7)) << 4) + 4 * (lane & 3);
          for (int k = 0; k < copies; ++k) {  // of few rows, one for each 32 rows of the tile
            sts_u32(to + k * 4096, c1);
            sts_u32(to + k * 4096 + 16384, c2);
          }
          if (lane == 0) sts_u32(factor_s + ((place & 1) * 128 + r) * 4, (e - 7u) << 23);  // 2^(exponent - 7)
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm->q_ready[place & 1]));
        return true;
      };
      const int units = p.D / 16;  // of a row
      auto serve = [&](uint32_t at, int n) {
        const int ntok = ATTN_ITEM(ntok);
        const uint32_t q0 = ATTN_ITEM(q0);
        const int kind = ATTN_ITEM(kind), rows = min(ntok, p.tile_tokens) * p.group;
        const int copies = ATTN_ITEM(few) ? 4 : 1;
        if (!split_q(q0, rows, copies)) return;
        if (kind != kOneTile && !split_q(q0 + 1, kind == kTwoHeads ? rows : (ntok - p.tile_tokens) * p.group, copies)) return;
        // V's codes to BF16 (exactly), into the layout that its product reads
#pragma unroll 1
        for (uint32_t t = tile0; t < tile0 + n; ++t) {
          const uint32_t rst = t % C::kVRawStages, st = t % C::kVStages;
          if (!wait(&sm->raw_full[rst], (t / C::kVRawStages) & 1)) return;
          if (t >= C::kVStages && !wait(&sm->kv_empty[C::kKStages + st], (t / C::kVStages - 1) & 1)) return;
          const uint32_t src = smem_u32(attn_smem) + C::kVRaw + rst * C::kRawBytes;
          const uint32_t dst = smem_u32(attn_smem) + C::kV + st * C::kTileBytes;
          // rows that no row sees (past the request's end, between the first
          // tokens and the window) may be anything, NaN too: zeros
          const int jj = ATTN_ITEM(j0) + ((int)(t - tile0) >> (kind == kTwoHeads));
          const int s0 = (jj < ATTN_ITEM(ns) ? jj : jj + ATTN_ITEM(skip)) * kAttnTile;
          const int end = ATTN_ITEM(seq) - s0;
          int from, to;
          attn_hidden(p, ATTN_ITEM(p0), s0, &from, &to);
          const int cc = tid & 7;  // 16 codes: 32 bytes of a row's half cc / 4
          const uint32_t unit = 2 * (cc & 3);
          if (cc < units) {
#pragma unroll 1
            for (int r0 = tid >> 3; r0 < 128; r0 += 64) {
              uint4 v[4];  // loaded ahead of the stores
#pragma unroll
              for (int i = 0; i < 4; ++i) v[i] = lds_v4(src + (r0 + 16 * i) * 128 + cc * 16);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int row = r0 + 16 * i;
                uint4 lo, hi;
                if (row >= end || (row >= from && row < to)) v[i] = make_uint4(0, 0, 0, 0);
                e4m3_to_bf16(v[i].x, &lo.x, &lo.y);
                e4m3_to_bf16(v[i].y, &lo.z, &lo.w);
                e4m3_to_bf16(v[i].z, &hi.x, &hi.y);
                e4m3_to_bf16(v[i].w, &hi.z, &hi.w);
                const uint32_t to = dst + (cc / 4) * 16384 + row * 128;
                sts_v4(to + ((unit ^ (row & 7)) << 4), lo);
                sts_v4(to + (((unit + 1) ^ (row & 7)) << 4), hi);
              }
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(smem_u32(&sm->kv_full[C::kKStages + st]));
            mbar_arrive(smem_u32(&sm->raw_empty[rst]));
          }
        }
        tile0 += n;
      };
      each_item(serve);
    } else if (warp == kAttnWalkWarp) {
      // ================================================================ walking
      AttnWalk w;
      w.len = len;
      w.share = share;
      w.s = 0;
      if (len > 0) {
        w.r = sm->begin_r;
        w.head = sm->begin_head;
        w.u = sm->begin_u;
        w.s = sm->begin_s;
        attn_request(p, w.r, &w.row0, &w.q, &w.seq);
        w.nu = attn_units(p, w.q);
        w.enter(p);
      }
      uint32_t it = 0;
      int q0 = 0;
      // false where no place got free in time: what lies there may be in use, so
      // nothing is put over it, and the walk is over
      auto hand = [&](int n) {
        const uint32_t st = it % kAttnItems, round = it / kAttnItems;
        if (round > 0 && !__all_sync(0xffffffffu, attn_wait(smem_u32(&sm->item_empty[st]), (round - 1) & 1, nullptr,
                                                            kAttnWalkLimit))) {
          *abort_flag = 1;
          if (lane == 0) raise_status(p.status, kStatusTimeout);
          return false;
        }
        if (lane == 0) {
          AttnItem* i = &sm->item[st];
          i->n = n;
          if (n > 0) {
            i->ntok = w.unit.ntok;
            i->kind = w.unit.kind;
            i->p0 = w.unit.p0;
            const int last = w.unit.p0 + w.unit.ntok - 1;
            const bool tiles = w.unit.kind == kTwoTiles;
            i->lo[0] = w.unit.p0;
            i->hi[0] = tiles ? w.unit.p0 + p.tile_tokens - 1 : last;
            i->lo[1] = tiles ? w.unit.p0 + p.tile_tokens : w.unit.p0;
            i->hi[1] = last;
            // (a rule on the unit, so that its CTAs agree)
            i->few = FP8 && w.unit.ntok <= p.tile_tokens32 && w.unit.n >= kAttnFewTiles;
            i->from[0] = 0;
            i->from[1] = tiles ? 0 : 1;
            i->step = tiles ? 1 : 2;
            i->ns = w.unit.ns;
            i->skip = w.unit.lo - w.unit.ns;
            i->j0 = w.j0;
            i->token = w.row0 + w.u * 2 * p.tile_tokens;
            i->head = w.head;
            i->r = w.r;
            i->seq = w.seq;
            i->c0 = w.cta_of(0);
            i->c1 = w.cta_of(w.unit.n - 1);
            i->slot = w.s >= 0;
            i->begins = w.s >= (i->c0 - (int)blockIdx.x) * share;
            i->q0 = q0;
            q0 += w.unit.kind != kOneTile ? 2 : 1;
          }
          mbar_arrive(smem_u32(&sm->item_full[st]));
        }
        __syncwarp();
        ++it;
        return true;
      };
      // With E4M3 caches this warp loads V as well, an item behind the walk (one
      // warp with both loads is what the kernel waits for: each copy costs it
      // some 150 cycles).
      auto load_v = [&](uint32_t item) {
        const uint32_t at = smem_u32(&sm->item[item % kAttnItems]);
        const int n = ATTN_ITEM(n), heads = ATTN_ITEM(kind) == kTwoHeads, head = ATTN_ITEM(head);
        if (!ok) return;
        AttnPages pages;
        pages.begin(p, at, n);
#pragma unroll 1
        for (int j = 0; j < n && ok; ++j) {
          int a, b;
          pages.get(p, j >> heads, j & heads, &a, &b);
          load8(false, head + (j & heads), a < 0 ? (int)p.num_pages : a, b < 0 ? (int)p.num_pages : b);
        }
      };
      bool handed = true;
      for (; handed && w.inside(); w.next(p)) {
        if (w.j1 <= w.j0) continue;
        handed = hand((w.j1 - w.j0) << (w.unit.kind == kTwoHeads));
        if (FP8 && handed && it > 1) load_v(it - 2);
      }
      if (handed) handed = hand(0);
      if (FP8 && handed && it > 1) load_v(it - 2);
      if (FP8) landed(sm->raw_full, n_t, C::kVRawStages);
    }
  }
#undef ATTN_ITEM
#undef ATTN_AT
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (sm->abort)
    for (int k = 0; k < 100; ++k) __nanosleep(1000);  // copies that the drain gave up on
  if (warp == kAttnMmaWarp) tmem_dealloc(tmem, 512);
}

}  // namespace dsa
