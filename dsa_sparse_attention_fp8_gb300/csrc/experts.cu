// C ABI of the operators behind the norm's 8-bit rows: the block-scaled product, the products grouped by expert, the router
// and the weighted sum of the experts' rows.  See include/dsa_indexer.h for the contract of every entry point.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <mutex>
#include <type_traits>

#include "combine.cuh"
#include "dsa_indexer.h"
#include "host.h"
#include "host_tensors.h"
#include "matmul.cuh"
#include "route.cuh"

namespace {

using namespace dsa_host;

bool is_float(int type) { return type == DSA_TYPE_BF16 || type == DSA_TYPE_FP16 || type == DSA_TYPE_FP32; }

// The tensor maps of rows (unless they are gathered) and weights, in boxes of `box` and `w_box` rows and 128 bytes of K.
int product_maps(const dsa::MatmulParams& p, int box, int w_box, CUtensorMap* tx, CUtensorMap* tw) {
  const int size = element_bytes(p.x_type);
  const CUtensorMapDataType type = size == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                   : p.x_type == DSA_TYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  if (!p.rows) {
    const int64_t xd[2] = {p.K, p.x_rows}, xs[1] = {p.x_stride * size};
    const int xb[2] = {128 / size, box};
    if (const int rc = make_map(tx, "x", type, size, p.x, 2, xd, xs, xb, true)) return rc;
  }
  const int64_t wd[3] = {p.K, p.N, p.E}, ws[2] = {p.w_stride * size, p.w_group * size};
  const int wb[3] = {128 / size, w_box, 1};
  return make_map(tw, "weight", type, size, p.w, 3, wd, ws, wb, true);
}

// Tiles of `tile` rows that so many groups of M rows in all can have.
int64_t row_tiles(int64_t M, int64_t groups, int tile) {
  const int64_t used = std::min(groups, M);
  return used + (M - used) / tile;
}

// The current device: its number and SMs.
struct Device {
  int id = -1, sms = 0;
  Device() {
    if (cudaGetDevice(&id) == cudaSuccess) sms = sm_count();
  }
};

// What a kernel needs once a device: its shared memory allowed, and how many clusters of 1 to 8 CTAs run at once.
class Ready {
 public:
  // The counts by size, or null with the error recorded.
  const int* on(const Device& d, const void* kernel, int threads, int smem) {
    if (d.id < 0 || d.id >= kDevices) return fail(DSA_ERR_CUDA, "no CUDA device, or more than %d", kDevices), nullptr;
    Slot& s = slot_[d.id];
    if (s.done.load(std::memory_order_acquire)) return s.clusters;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return fail(DSA_ERR_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(e)), nullptr;
    int found[9] = {};
    for (int size = 1; size <= 8; ++size) {
      cudaLaunchConfig_t c{};
      cudaLaunchAttribute a[1];
      a[0].id = cudaLaunchAttributeClusterDimension;
      a[0].val.clusterDim.x = size, a[0].val.clusterDim.y = 1, a[0].val.clusterDim.z = 1;
      c.gridDim = dim3(size), c.blockDim = dim3(threads), c.dynamicSmemBytes = smem, c.attrs = a, c.numAttrs = 1;
      if (cudaOccupancyMaxActiveClusters(&found[size], kernel, &c) != cudaSuccess) found[size] = 0, cudaGetLastError();
    }
    if (found[1] < 1 || found[2] < 1) return fail(DSA_ERR_CUDA, "the products' kernels do not fit the device"), nullptr;
    const std::lock_guard<std::mutex> hold(lock_);
    if (!s.done.load(std::memory_order_relaxed)) {
      std::copy(found, found + 9, s.clusters);
      s.done.store(true, std::memory_order_release);
    }
    return s.clusters;
  }

 private:
  static constexpr int kDevices = 64;
  struct Slot {
    std::atomic<bool> done{false};
    int clusters[9] = {};
  };
  Slot slot_[kDevices];
  std::mutex lock_;
};

// Launches a kernel, in clusters of `size` CTAs, that waits for what is before it in the stream by itself: it is set up while
// the kernel before drains (DSA_PDL=0: not).
template <typename... P, typename... A>
int launch(const char* name, void (*kernel)(P...), dim3 grid, int block, int size, int smem, cudaStream_t st, const A&... args) {
  cudaLaunchConfig_t c{};
  cudaLaunchAttribute a[2];
  a[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a[0].val.programmaticStreamSerializationAllowed = env_int("DSA_PDL", 1, 0, 1);
  a[1].id = cudaLaunchAttributeClusterDimension;
  a[1].val.clusterDim.x = size, a[1].val.clusterDim.y = 1, a[1].val.clusterDim.z = 1;
  c.gridDim = grid, c.blockDim = dim3(block), c.dynamicSmemBytes = smem;
  c.stream = st, c.attrs = a, c.numAttrs = size > 1 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&c, kernel, args...);
  if (e != cudaSuccess) return fail(DSA_ERR_CUDA, "%s: %s", name, cudaGetErrorString(e));
  return check_launch(name);
}

// How a product's tiles go to CTAs: clusters of `size`, so many of them, and about how long it takes in microseconds.
struct Plan {
  double us;
  int size, clusters;
};

// Tiles of BM rows, a tile's K shared by a cluster.
template <bool FP8, bool GATED, bool WIDE, int BM, int ROUND = GATED || WIDE ? 32 : 64>
struct Few {
  using C = dsa::FewCfg<FP8, GATED, WIDE, BM, ROUND>;
  static constexpr auto kKernel = dsa::few_rows_kernel<FP8, GATED, WIDE, BM, ROUND>;
  static inline Ready ready;

  // A CTA alone takes as long for a block of K wherever it lies, bound by what one SM draws from L2 (measured of one tile of 64
  // rows, 128 weight rows and 7168 elements of K, in L2: 21.0 us by one CTA, 9.4 by four, 7.7 by eight).  CTAs that share a
  // tile join their sums, round by round.
  static constexpr double kBlock = (C::kStageA + C::kStageB) / 110e3 + 0.06, kRoundUs = C::BN == 256 ? 1.8 : 0.8;

  static int plan(const dsa::MatmulParams& p, int64_t groups, const Device& d, Plan* best) {
    *best = {1e30, 0, 0};
    const int* const clusters = ready.on(d, (const void*)kKernel, dsa::kMatmulThreads, C::kSmem);
    if (!clusters) return DSA_ERR_CUDA;
    const int64_t tiles = row_tiles(p.M, groups, BM) * ((p.width + C::kOut - 1) / C::kOut);
    const int blocks = (p.K + C::kK - 1) / C::kK, rounds = (std::min(BM, p.M) + ROUND - 1) / ROUND;
    for (int s = 1; s <= 8 && (s == 1 || (2 * s <= blocks && tiles * s <= d.sms)); ++s) {
      const int n = clusters[s];
      if (n < 1) continue;
      const double us = (double)((tiles + n - 1) / n) * ((blocks + s - 1) / s * kBlock + (s == 1 ? 0.5 : 0.4 + 0.1 * s + rounds * kRoundUs));
      if (us < best->us) *best = {us, s, n};
    }
    return DSA_OK;
  }

  static int run(dsa::MatmulParams p, int64_t groups, const Device& d, cudaStream_t st) {
    Plan plan;
    if (const int rc = Few::plan(p, groups, d, &plan)) return rc;
    return run(p, groups, plan, st);
  }
  static int run(dsa::MatmulParams p, int64_t groups, Plan plan, cudaStream_t st) {
    CUtensorMap tx{}, tw{};
    p.box = p.M <= 32 * groups ? 32 : BM;
    if (const int rc = product_maps(p, p.box, C::kBox, &tx, &tw)) return rc;
    const int64_t columns = (p.width + C::kOut - 1) / C::kOut, tiles = row_tiles(p.M, groups, BM) * columns;
    if (tiles > INT32_MAX / 2) return fail(DSA_ERR_UNSUPPORTED, "%lld tiles of results", (long long)tiles);
    p.most_tiles = (int)(INT32_MAX / 2 / columns);
    set_last_launches(1);
    return launch("few_rows_kernel", kKernel, (unsigned)(std::min<int64_t>(tiles, plan.clusters) * plan.size), dsa::kMatmulThreads, plan.size,
                  C::kSmem, st, tx, tw, p);
  }
};

// Tiles of 256 rows by pairs of CTAs.
template <bool FP8, bool GATED>
struct Many {
  using C = dsa::ManyCfg<FP8, GATED>;
  static constexpr auto kKernel = dsa::many_rows_kernel<FP8, GATED>;
  static inline Ready ready;

  static int plan(const dsa::MatmulParams& p, int64_t groups, const Device& d, Plan* best) {
    const int* const clusters = ready.on(d, (const void*)kKernel, dsa::kMatmulThreads, C::kSmem);
    if (!clusters) return DSA_ERR_CUDA;
    const int n = clusters[2];
    const int64_t tiles = row_tiles(p.M, groups, C::BM) * ((p.width + C::kOut - 1) / C::kOut);
    // (8192 rows, K = N = 7168: twelve tiles of 56 blocks to a pair in 300 us)
    *best = {(double)((tiles + n - 1) / n) * ((p.K + C::kK - 1) / C::kK * 0.43 + 1.0), 2, n};
    return DSA_OK;
  }

  static int run(dsa::MatmulParams p, int64_t groups, const Device& d, cudaStream_t st) {
    Plan plan;
    if (const int rc = Many::plan(p, groups, d, &plan)) return rc;
    return run(p, groups, plan, st);
  }
  static int run(dsa::MatmulParams p, int64_t groups, const Plan& plan, cudaStream_t st) {
    CUtensorMap tx{}, tw{};
    if (const int rc = product_maps(p, 128, C::kBox, &tx, &tw)) return rc;
    const int64_t columns = (p.width + C::kOut - 1) / C::kOut, tiles = row_tiles(p.M, groups, C::BM) * columns;
    if (tiles > INT32_MAX / 2) return fail(DSA_ERR_UNSUPPORTED, "%lld tiles of results", (long long)tiles);
    p.most_tiles = (int)(INT32_MAX / 2 / columns);
    set_last_launches(1);
    return launch("many_rows_kernel", kKernel, (unsigned)(std::min<int64_t>(tiles, plan.clusters) * 2), dsa::kMatmulThreads, 2, C::kSmem, st, tx, tw, p);
  }
};

// The variant for a product's sizes.
template <bool FP8, bool GATED>
int run_variant(const dsa::MatmulParams& p, int64_t groups, cudaStream_t st) {
  using Few64 = Few<FP8, GATED, false, 64>;
  // A tile of few joined in one round, for which it has a stage less: a round's sums are given back by a release of the cluster's
  // scope, which costs a microsecond and more (96 rows, K 7168, N 4096, in two rounds 12.3 us, in one 10.7; of many tiles, which
  // are not shared, 36 rows to each of 64 groups of BF16, K 2048, N 3584, the stage counts: 154 with it, 161 without).
  using Joined64 = Few<FP8, GATED, false, 64, 64>;
  using Joined128 = Few<FP8, GATED, false, 128, GATED ? 32 : 128>;
  using Wide64 = Few<FP8, false, !GATED, 64>;
  using Few128 = Few<FP8, GATED, false, 128>;
  using Pairs = Many<FP8, GATED>;
  const Device d;
  if (d.sms <= 0) return fail(DSA_ERR_CUDA, "no CUDA device");
  const int64_t tiles = row_tiles(p.M, groups, 64) * ((p.width + 127) / 128);
  if (groups > 1 && tiles > 2 * d.sms) {
    // Bound by the weights' way from HBM.  Tiles fit the rows of a group; 256 weight rows to a tile, so that rows are read less
    // often.  Of 64 groups, as uneven as a router's choices make them, in us, by rows to a group in the mean:
    //   E4M3, K 2048, N 7168, tiles of 64 x 128, 64 x 256, 128 x 128 and by pairs: 16 rows 203, 157, 183, 198; 32 207, 163, 188,
    //     200; 48 234, 189, 196, 205; 96 345, 274, 270, 217.
    //   E4M3, gated, gathered, K 7168, N 4096, tiles of 64 rows, of 128 and by pairs: 32 300, 310, 395; 48 338, 317, 399; 96 459,
    //     416, 418; 128 552, 479, 436.
    //   BF16, K 2048, N 3584, as the first: 32 146, 150, 153, 153; 48 159, 162, 156, 155; 96 217, 183, 175, 161.
    //   BF16, gated, gathered, K 3584, N 2048, as the second: 32 153, 160, 155; 48 170, 164, 158; 96 186, 185, 163; 128 223, 180, 166.
    // (So 16-bit gated products of 33 to 96 rows would be better off by pairs, by 4 to 12 %.)  The mean is over all groups, as the
    // host knows no more: where eight of 256 groups have 256 rows each and the others none (BF16, K = N = 2048), tiles of 64
    // rows take 32.6 us and pairs would take 18.0.
    if (p.M <= 32 * groups) {
      if constexpr (GATED) return Few64::run(p, groups, d, st);
      else return Wide64::run(p, groups, d, st);
    }
    return p.M <= (GATED ? 96 : 48) * groups ? Few128::run(p, groups, d, st) : Pairs::run(p, groups, d, st);
  }
  // Few tiles: as the CTAs that share their K take.
  Plan few, some, many;
  if (const int rc = Joined64::plan(p, groups, d, &few)) return rc;
  if (const int rc = Joined128::plan(p, groups, d, &some)) return rc;
  if (const int rc = Pairs::plan(p, groups, d, &many)) return rc;
  if (many.us < few.us && many.us < some.us) return Pairs::run(p, groups, many, st);
  return some.us < few.us ? Joined128::run(p, groups, some, st) : Joined64::run(p, groups, few, st);
}

// The checks that both products share, and their launch.  p has the sizes, strides and pointers.
int run_matmul(dsa::MatmulParams p, int64_t groups, cudaStream_t st) {
  if (p.M < 0 || p.x_rows < 0) return fail(DSA_ERR_INVALID_ARG, "a negative number of rows");
  if (p.N < 1 || p.K < 1) return fail(DSA_ERR_INVALID_ARG, "N=%d, K=%d: both must be positive", p.N, p.K);
  if (p.M > 1 << 30 || p.x_rows > 1 << 30) return fail(DSA_ERR_UNSUPPORTED, "%d rows of %d: at most 2^30", p.M, p.x_rows);
  if (p.N > 1 << 28 || p.K > 1 << 28) return fail(DSA_ERR_UNSUPPORTED, "N=%d, K=%d: at most 2^28", p.N, p.K);
  if (p.gated && p.N % 2) return fail(DSA_ERR_INVALID_ARG, "gated weights have two halves: N=%d is odd", p.N);
  p.width = p.gated ? p.N / 2 : p.N;
  const bool fp8 = p.x_type == DSA_TYPE_E4M3;
  if (fp8 && p.gated && p.width % 64)
    return fail(DSA_ERR_UNSUPPORTED, "gated E4M3 weights: N/2=%d is no multiple of 64", p.width);
  if ((p.out || !p.codes) && !is_float(p.out_type)) return fail(DSA_ERR_UNSUPPORTED, "out_type=%d: BF16, FP16 or FP32 is wanted", p.out_type);
  if (p.out && p.M > 1 && p.out_stride < p.width) return fail(DSA_ERR_INVALID_ARG, "out's row stride is shorter than a row");
  const int size = element_bytes(p.x_type), unit = 16 / size;
  if (!stride_ok(p.x_stride, p.x_rows, unit) || !stride_ok(p.w_stride, p.N, unit) || !stride_ok(p.w_group, groups, unit))
    return fail(DSA_ERR_INVALID_ARG, "strides of rows and weights must be multiples of 16 bytes");
  if (!apart(p.x_stride, p.x_rows) || !apart(p.w_stride, p.N) || !apart(p.w_group, groups))
    return fail(DSA_ERR_INVALID_ARG, "a stride of 0 over more than one row");
  if (p.rows && p.x_stride * size / 16 > (INT64_C(1) << 32) / std::max(1, p.x_rows))
    return fail(DSA_ERR_UNSUPPORTED, "gathered rows lie over more than 64 GB");
  if (p.M == 0) return DSA_OK;
  if ((p.out != nullptr) == (p.codes != nullptr) || (p.codes != nullptr) != (p.scales != nullptr))
    return fail(DSA_ERR_INVALID_ARG, "either out or out_codes and out_scales");
  if (p.codes && !p.gated) return fail(DSA_ERR_UNSUPPORTED, "8-bit results are those of gated products");
  if (!p.x || !p.w) return fail(DSA_ERR_INVALID_ARG, "null pointer");
  if (fp8 && (!p.x_scales || !p.w_scales)) return fail(DSA_ERR_INVALID_ARG, "E4M3 rows and weights need their scales");
  if (!aligned(p.x, 16) || !aligned(p.w, 16)) return fail(DSA_ERR_INVALID_ARG, "rows and weights must be 16-byte aligned");
  if (p.out && !aligned(p.out, element_bytes(p.out_type))) return fail(DSA_ERR_INVALID_ARG, "out is not aligned to its elements");
  p.kb = (p.K + dsa::kMatmulBlock - 1) / dsa::kMatmulBlock;
  p.nb = (p.N + dsa::kMatmulBlock - 1) / dsa::kMatmulBlock;
  if (!fp8) p.x_scales = p.w_scales = nullptr;
  p.load_stages = env_int("DSA_LOAD_STAGES", -1, -1, 1 << 20);
  if (env_int("DSA_WAIT_LIMIT", (int)dsa::kWaitLimit, 0, (int)dsa::kWaitLimit) == 0) p.load_stages = 0;
  if (fp8) return p.gated ? run_variant<true, true>(p, groups, st) : run_variant<true, false>(p, groups, st);
  return p.gated ? run_variant<false, true>(p, groups, st) : run_variant<false, false>(p, groups, st);
}

template <int V, typename T>
int launch_route(const dsa::RouteParams& p, cudaStream_t st) {
  static PerDevice few, many, wide;
  constexpr int kWarps = dsa::kFewThreads / 32;
  if (p.T <= kWarps * dsa::kFewCtas) {
    int ctas = 1;
    while (ctas * kWarps < p.T) ctas *= 2;
    const auto kernel = dsa::route_few_kernel<V, T>;
    if (const int rc = allow_smem(few, (const void*)kernel, dsa::counts_bytes(kWarps, dsa::kRouteMaxExperts))) return rc;
    set_last_launches(1);
    return launch("route_few_kernel", kernel, ctas, dsa::kFewThreads, ctas, dsa::counts_bytes(kWarps, p.E), st, p);
  }
  const unsigned grid = (unsigned)(((int64_t)p.T * 32 + dsa::kRouteThreads - 1) / dsa::kRouteThreads);
  if (const int rc = launch("route_choose_kernel", dsa::route_choose_kernel<V, T>, grid, dsa::kRouteThreads, 1, 0, st, p)) return rc;
  const auto kernel = dsa::route_place_kernel;
  constexpr int kPlaceWarps = dsa::kPlaceThreads / 32;
  if (const int rc = allow_smem(many, (const void*)kernel, dsa::counts_bytes(kPlaceWarps, dsa::kRouteMaxExperts))) return rc;
  const cudaError_t e = wide.once([&] { return cudaFuncSetAttribute((const void*)kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1); });
  if (e != cudaSuccess) return fail(DSA_ERR_CUDA, "route_place_kernel: %s", cudaGetErrorString(e));
  set_last_launches(2);
  return launch("route_place_kernel", kernel, dsa::kPlaceCtas, dsa::kPlaceThreads, dsa::kPlaceCtas, dsa::counts_bytes(kPlaceWarps, p.E), st, p);
}

template <int V>
int launch_route(const dsa::RouteParams& p, int type, cudaStream_t st) {
  if (type == DSA_TYPE_BF16) return launch_route<V, __nv_bfloat16>(p, st);
  if (type == DSA_TYPE_FP16) return launch_route<V, __half>(p, st);
  return launch_route<V, float>(p, st);
}

template <typename T>
int launch_combine(const dsa::CombineParams& p, bool vec, cudaStream_t st) {
  const unsigned slices = (unsigned)std::min(65535, (p.N + dsa::kCombineThreads * 8 - 1) / (dsa::kCombineThreads * 8));
  set_last_launches(1);
  return launch("combine_kernel", vec ? dsa::combine_kernel<T, true> : dsa::combine_kernel<T, false>, dim3(p.T, slices), dsa::kCombineThreads, 1, 0, st, p);
}

}  // namespace

extern "C" {

int dsa_fp8_matmul(const uint8_t* codes, int64_t stride, const float* scales, int T,
                   const uint8_t* w_codes, int64_t w_stride, const float* w_scales, int N, int K,
                   int gated, void* out, int64_t out_stride, int out_type, uint8_t* out_codes,
                   float* out_scales, int32_t* dev_status, dsa_stream_t stream) {
  set_last_launches(0);
  dsa::MatmulParams p{};
  p.x = codes, p.x_scales = scales, p.w = w_codes, p.w_scales = w_scales;
  p.out = out, p.codes = out_codes, p.scales = out_scales, p.status = dev_status;
  p.x_stride = stride, p.w_stride = w_stride, p.out_stride = out_stride;
  p.x_rows = T, p.M = T, p.N = N, p.K = K, p.E = 1;
  p.x_type = DSA_TYPE_E4M3, p.out_type = out_type, p.gated = gated != 0;
  return run_matmul(p, 1, (cudaStream_t)stream);
}

int dsa_grouped_matmul(const void* x, int64_t x_stride, const float* x_scales, int x_type, int x_rows,
                       const int32_t* rows, int M, const void* weight, int64_t w_row_stride,
                       int64_t w_group_stride, const float* w_scales, int N, int K,
                       const int32_t* group_starts, int E, int gated, void* out, int64_t out_stride,
                       int out_type, uint8_t* out_codes, float* out_scales, int32_t* dev_status,
                       dsa_stream_t stream) {
  set_last_launches(0);
  if (x_type != DSA_TYPE_E4M3 && x_type != DSA_TYPE_BF16 && x_type != DSA_TYPE_FP16)
    return fail(DSA_ERR_UNSUPPORTED, "x_type=%d: BF16, FP16 or E4M3 is wanted", x_type);
  if (E < 1) return fail(DSA_ERR_INVALID_ARG, "E=%d < 1", E);
  if (E > dsa::kMatmulMaxGroups) return fail(DSA_ERR_UNSUPPORTED, "E=%d > %d", E, dsa::kMatmulMaxGroups);
  if (!rows && M > 0 && M != x_rows) return fail(DSA_ERR_INVALID_ARG, "without rows, M=%d must be x_rows=%d", M, x_rows);
  if (M > 0 && x_rows < 1) return fail(DSA_ERR_INVALID_ARG, "x_rows=%d < 1", x_rows);
  if (M > 0 && !group_starts) return fail(DSA_ERR_INVALID_ARG, "null pointer");
  dsa::MatmulParams p{};
  p.x = x, p.x_scales = x_scales, p.rows = rows, p.w = weight, p.w_scales = w_scales, p.starts = group_starts;
  p.out = out, p.codes = out_codes, p.scales = out_scales, p.status = dev_status;
  p.x_stride = x_stride, p.w_stride = w_row_stride, p.w_group = w_group_stride, p.out_stride = out_stride;
  p.x_rows = x_rows, p.M = M, p.N = N, p.K = K, p.E = E;
  p.x_type = x_type, p.out_type = out_type, p.gated = gated != 0;
  return run_matmul(p, E, (cudaStream_t)stream);
}

int dsa_route_experts(const void* logits, int64_t stride, int type, const float* bias, int T, int E,
                      int top_k, int scoring, int num_groups, int top_groups, int normalize,
                      float scale, const int32_t* num_tokens, int32_t* expert_ids, float* weights,
                      int32_t* group_starts, int32_t* rows, int32_t* places, dsa_stream_t stream) {
  set_last_launches(0);
  if (T < 0) return fail(DSA_ERR_INVALID_ARG, "T=%d < 0", T);
  if (E < 1) return fail(DSA_ERR_INVALID_ARG, "E=%d < 1", E);
  if (E > dsa::kRouteMaxExperts) return fail(DSA_ERR_UNSUPPORTED, "E=%d > %d", E, dsa::kRouteMaxExperts);
  if (!is_float(type)) return fail(DSA_ERR_UNSUPPORTED, "type=%d: BF16, FP16 or FP32 is wanted", type);
  if (top_k < 1) return fail(DSA_ERR_INVALID_ARG, "top_k=%d < 1", top_k);
  if (top_k > dsa::kRouteMaxTop) return fail(DSA_ERR_UNSUPPORTED, "top_k=%d > %d", top_k, dsa::kRouteMaxTop);
  if (scoring != DSA_SCORE_SIGMOID && scoring != DSA_SCORE_SOFTMAX)
    return fail(DSA_ERR_INVALID_ARG, "scoring=%d is neither DSA_SCORE_SIGMOID nor DSA_SCORE_SOFTMAX", scoring);
  if (num_groups < 1 || E % num_groups) return fail(DSA_ERR_INVALID_ARG, "num_groups=%d does not divide E=%d", num_groups, E);
  if (num_groups > dsa::kRouteMaxRuns)
    return fail(DSA_ERR_UNSUPPORTED, "num_groups=%d > %d", num_groups, dsa::kRouteMaxRuns);
  if (top_groups < 1 || top_groups > num_groups)
    return fail(DSA_ERR_INVALID_ARG, "top_groups=%d outside [1, %d]", top_groups, num_groups);
  if (top_k > top_groups * (E / num_groups))
    return fail(DSA_ERR_INVALID_ARG, "top_k=%d of %d experts in the chosen groups", top_k, top_groups * (E / num_groups));
  if (!(scale == scale) || scale - scale != 0.0f) return fail(DSA_ERR_INVALID_ARG, "scale must be finite");
  if ((int64_t)T * top_k > 1 << 30) return fail(DSA_ERR_UNSUPPORTED, "T=%d times top_k=%d: at most 2^30", T, top_k);
  if (T > 1 && stride < E) return fail(DSA_ERR_INVALID_ARG, "the row stride is shorter than E");
  if (!group_starts) return fail(DSA_ERR_INVALID_ARG, "null pointer");
  if (T && (!logits || !expert_ids || !weights || !rows || !places)) return fail(DSA_ERR_INVALID_ARG, "null pointer");
  dsa::RouteParams p{};
  p.logits = logits, p.bias = bias, p.num_tokens = num_tokens;
  p.ids = expert_ids, p.weights = weights, p.starts = group_starts, p.rows = rows, p.places = places;
  p.stride = stride, p.T = T, p.E = E, p.top_k = top_k;
  p.num_groups = num_groups, p.top_groups = top_groups, p.per = E / num_groups;
  p.scale = scale, p.softmax = scoring == DSA_SCORE_SOFTMAX, p.normalize = normalize != 0;
  const cudaStream_t st = (cudaStream_t)stream;
  // a run's lanes: as many as there are for each of so many runs.  More than 16 experts to a lane, as 3, 5, 9 or 17 runs of
  // many experts make, spill registers: 8192 tokens of 510 experts in 3 runs take 48 us, in 17 runs 78, of 512 in 8 runs 36.
  p.lanes = 32;
  while (32 / p.lanes < num_groups) p.lanes /= 2;
  p.wide = (p.per + p.lanes - 1) / p.lanes;
  if (p.wide <= 1) return launch_route<1>(p, type, st);
  if (p.wide <= 2) return launch_route<2>(p, type, st);
  if (p.wide <= 4) return launch_route<4>(p, type, st);
  if (p.wide <= 8) return launch_route<8>(p, type, st);
  if (p.wide <= 16) return launch_route<16>(p, type, st);
  return launch_route<32>(p, type, st);
}

int dsa_combine_experts(const void* y, int64_t y_stride, int type, int M, const int32_t* places,
                        const float* weights, int T, int top_k, int N, const void* add,
                        int64_t add_stride, void* out, int64_t out_stride, int32_t* dev_status,
                        dsa_stream_t stream) {
  set_last_launches(0);
  if (T < 0 || M < 0) return fail(DSA_ERR_INVALID_ARG, "a negative number of rows");
  if (N < 1) return fail(DSA_ERR_INVALID_ARG, "N=%d < 1", N);
  if (N > 1 << 28) return fail(DSA_ERR_UNSUPPORTED, "N=%d: at most 2^28", N);
  if (top_k < 1) return fail(DSA_ERR_INVALID_ARG, "top_k=%d < 1", top_k);
  if (top_k > dsa::kCombineMaxTop) return fail(DSA_ERR_UNSUPPORTED, "top_k=%d > %d", top_k, dsa::kCombineMaxTop);
  if (!is_float(type)) return fail(DSA_ERR_UNSUPPORTED, "type=%d: BF16, FP16 or FP32 is wanted", type);
  if ((M > 1 && y_stride < N) || (T > 1 && ((add && add_stride < N) || out_stride < N)))
    return fail(DSA_ERR_INVALID_ARG, "a row stride is shorter than N");
  if (T == 0) return DSA_OK;
  if ((M && !y) || !places || !weights || !out) return fail(DSA_ERR_INVALID_ARG, "null pointer");
  const int size = element_bytes(type);
  if (!aligned(y, size) || !aligned(add, size) || !aligned(out, size))
    return fail(DSA_ERR_INVALID_ARG, "rows are not aligned to their elements");
  const dsa::CombineParams p{y, places, weights, add, out, dev_status, y_stride, add_stride, out_stride, M, T, top_k, N};
  auto row16 = [&](const void* ptr, int64_t stride, int64_t n) {
    return !ptr || (aligned(ptr, 16) && (n <= 1 || stride * size % 16 == 0));
  };
  const bool vec = N % 8 == 0 && row16(y, y_stride, M) && row16(add, add_stride, T) && row16(out, out_stride, T);
  const cudaStream_t st = (cudaStream_t)stream;
  if (type == DSA_TYPE_BF16) return launch_combine<__nv_bfloat16>(p, vec, st);
  if (type == DSA_TYPE_FP16) return launch_combine<__half>(p, vec, st);
  return launch_combine<float>(p, vec, st);
}

}  // extern "C"
