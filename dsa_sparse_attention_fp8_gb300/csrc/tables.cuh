// Block tables and slot maps of one step, built from the requests' lengths.
//
// Request r brings q[r] new tokens and holds seq[r] tokens after the step, so
// it needs need[r] = ceil(seq / 64) - ceil((seq - q) / 64) pages more than its
// block-table row already lists.  With start = exclusive sums of q and taken =
// exclusive sums of need, the step's pages are free_pages[0 .. taken[R]) in
// request order, and token t of request r sits at position
// seq - q + (t - start[r]), slot = page * 64 + position % 64 ("HBM 索引架构设计"
// §2.3).
#pragma once

#include <cstdint>

#include "common.cuh"

namespace dsa {

constexpr int kTablesThreads = 512;
constexpr int kTablesMaxRequests = 16384;

struct TablesParams {
  const int32_t* q_lens;      // [R]
  const int32_t* seq_lens;    // [R]
  int R;
  const int32_t* free_pages;  // [num_free]
  int num_free;
  int32_t* block_table;       // [R, max_blocks]
  int max_blocks;
  int T;                      // rows of positions and slot_mapping
  int32_t* start;             // [R + 1]
  int32_t* positions;         // [T]
  int64_t* slots;             // [T]
  int32_t* used;              // [1]
  int32_t* status;
};

// A request's rows and pages.  Lengths that make no sense hold rows as far as
// possible (so that the later requests' rows stay where the caller put them)
// but neither pages nor slots.
struct TablesRequest {
  int q, seq;
  int before, need;  // blocks held before the step, blocks added
  bool ok;
};

__device__ __forceinline__ TablesRequest tables_request(const TablesParams& p, int r) {
  TablesRequest x;
  x.q = __ldg(p.q_lens + r);
  x.seq = __ldg(p.seq_lens + r);
  x.ok = x.q >= 0 && x.q <= p.T && x.seq >= x.q && (int64_t)x.seq <= (int64_t)p.max_blocks * kPageTokens;
  if (x.q < 0 || x.q > p.T) x.q = 0;
  x.before = x.ok ? (int)(((int64_t)x.seq - x.q + kPageTokens - 1) / kPageTokens) : 0;
  x.need = x.ok ? (int)(((int64_t)x.seq + kPageTokens - 1) / kPageTokens) - x.before : 0;
  return x;
}

__device__ __forceinline__ int32_t tables_clamp(int64_t x) {
  return x > INT32_MAX ? INT32_MAX : (int32_t)x;
}

// The last i with a[i] <= x, for a nondecreasing a[0 .. n) with a[0] <= x.
__device__ __forceinline__ int tables_find(const int32_t* a, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a[mid] <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// One launch: every CTA sums the lengths of all requests itself (two sums per
// request from 8 bytes that L2 holds; no second launch and no hand-over
// between CTAs), keeps both exclusive sums in shared memory and then serves a
// share of the tokens and of the new table entries, each found by a binary
// search in shared memory.  Bound by latency: the lengths are read three times,
// one global latency after the other (for the sums, the exclusive sums and a
// token's request): 64 requests of one token 6.2 us, of which a launch is 2.7;
// 2048 requests with 75,000 tokens 8.4 us (0.9 MB).
__global__ void __launch_bounds__(kTablesThreads) block_tables_kernel(const __grid_constant__ TablesParams p) {
  extern __shared__ int32_t tables_smem[];
  int32_t* start = tables_smem;           // [R + 1]
  int32_t* taken = tables_smem + p.R + 1; // [R + 1]
  __shared__ int64_t warp_q[kTablesThreads / 32], warp_n[kTablesThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (p.R + kTablesThreads - 1) / kTablesThreads;
  const int r0 = tid * per, r1 = min(r0 + per, p.R);
  int64_t sum_q = 0, sum_n = 0;
  bool bad = false;
  for (int r = r0; r < r1; ++r) {
    const TablesRequest x = tables_request(p, r);
    sum_q += x.q;
    sum_n += x.need;
    bad |= !x.ok;
  }
  int64_t inc_q = sum_q, inc_n = sum_n;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t a = __shfl_up_sync(0xffffffffu, inc_q, o), b = __shfl_up_sync(0xffffffffu, inc_n, o);
    if (lane >= o) { inc_q += a; inc_n += b; }
  }
  if (lane == 31) { warp_q[warp] = inc_q; warp_n[warp] = inc_n; }
  __syncthreads();
  int64_t at_q = inc_q - sum_q, at_n = inc_n - sum_n, all_q = 0, all_n = 0;
  for (int w = 0; w < kTablesThreads / 32; ++w) {
    if (w < warp) { at_q += warp_q[w]; at_n += warp_n[w]; }
    all_q += warp_q[w];
    all_n += warp_n[w];
  }
  for (int r = r0; r < r1; ++r) {
    const TablesRequest x = tables_request(p, r);
    start[r] = tables_clamp(at_q);
    taken[r] = tables_clamp(at_n);
    if (blockIdx.x == 0) p.start[r] = tables_clamp(at_q);
    at_q += x.q;
    at_n += x.need;
  }
  if (tid == 0) {
    start[p.R] = tables_clamp(all_q);
    taken[p.R] = tables_clamp(all_n);
    if (blockIdx.x == 0) {
      p.start[p.R] = tables_clamp(all_q);
      p.used[0] = tables_clamp(all_n);
      if (all_n > p.num_free) raise_status(p.status, kStatusNoPages);
      if (all_q > p.T) raise_status(p.status, kStatusBadMetadata);
    }
  }
  if (bad && blockIdx.x == 0) raise_status(p.status, kStatusBadMetadata);
  __syncthreads();

  const int total = start[p.R], pages = taken[p.R];
  const int64_t step = (int64_t)gridDim.x * kTablesThreads;
  for (int64_t t = (int64_t)blockIdx.x * kTablesThreads + tid; t < p.T; t += step) {
    int pos = 0;
    int64_t slot = -1;
    if (t < total) {
      const int r = tables_find(start, p.R, (int)t);
      const TablesRequest x = tables_request(p, r);
      if (x.ok) {
        pos = x.seq - x.q + ((int)t - start[r]);
        const int blk = pos / kPageTokens;
        int page = -1;
        if (blk < x.before) {
          page = __ldg(p.block_table + (int64_t)r * p.max_blocks + blk);
          if (page < 0) raise_status(p.status, kStatusBadPage);
        } else {
          const int64_t i = (int64_t)taken[r] + (blk - x.before);
          if (i < p.num_free) page = __ldg(p.free_pages + i);
        }
        if (page >= 0) slot = (int64_t)page * kPageTokens + pos % kPageTokens;
      }
    }
    p.positions[t] = pos;
    p.slots[t] = slot;
  }
  for (int64_t i = (int64_t)blockIdx.x * kTablesThreads + tid; i < pages; i += step) {
    const int r = tables_find(taken, p.R, (int)i);
    const TablesRequest x = tables_request(p, r);
    const int j = (int)i - taken[r];
    if (j < x.need)
      p.block_table[(int64_t)r * p.max_blocks + x.before + j] = i < p.num_free ? __ldg(p.free_pages + i) : -1;
  }
}

}  // namespace dsa
