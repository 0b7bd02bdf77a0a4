// C ABI of the operators around the paged caches: block tables and slot maps,
// the K/V cache write, attention over the paged K/V cache, and the residual
// addition + root-mean-square norm with 8-bit output.  See
// include/dsa_indexer.h for the contract of every entry point.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "dsa_indexer.h"
#include "host.h"
#include "kvcache.cuh"
#include "norm.cuh"
#include "paged_attention.cuh"
#include "tables.cuh"

namespace {

using namespace dsa_host;

int element_bytes(int type) { return type == DSA_TYPE_FP32 ? 4 : type == DSA_TYPE_E4M3 ? 1 : 2; }

// Whether a stride over n elements is neither negative nor off a multiple of
// `unit` (one element may have any stride: nothing is ever a stride away).
bool stride_ok(int64_t stride, int64_t n, int unit) { return n <= 1 || (stride >= 0 && stride % unit == 0); }

// Whether a stride over n elements keeps them apart, as what is written, or read
// by way of a tensor map, has to be.
bool apart(int64_t stride, int64_t n) { return n <= 1 || stride != 0; }

// A K/V cache as the kernels need it: 16-byte aligned heads, at most 128
// elements each.
int check_cache(const dsa_kv_cache* c, int type, bool written) {
  if (!c) return fail(DSA_ERR_INVALID_ARG, "null cache");
  if (type != DSA_TYPE_BF16 && type != DSA_TYPE_FP16)
    return fail(DSA_ERR_UNSUPPORTED, "type=%d: BF16 or FP16 is wanted", type);
  if (c->type != type && !(c->type == DSA_TYPE_E4M3))
    return fail(DSA_ERR_UNSUPPORTED, "cache type %d: the rows' own type (%d) or E4M3 is wanted", c->type, type);
  if (c->num_kv_heads < 1) return fail(DSA_ERR_INVALID_ARG, "num_kv_heads=%d < 1", c->num_kv_heads);
  if (c->head_dim < 16 || c->head_dim > 128 || c->head_dim % 16)
    return fail(DSA_ERR_UNSUPPORTED, "head_dim=%d: a multiple of 16 in [16, 128] is wanted", c->head_dim);
  if (c->num_pages < 1 || c->num_pages > INT32_MAX / DSA_PAGE_TOKENS)
    return fail(DSA_ERR_INVALID_ARG, "num_pages=%lld outside [1, %d]", (long long)c->num_pages,
                INT32_MAX / DSA_PAGE_TOKENS);
  const int unit = 16 / element_bytes(c->type);
  const int64_t pages = c->num_pages, heads = c->num_kv_heads;
  if (!stride_ok(c->k_page_stride, pages, unit) || !stride_ok(c->v_page_stride, pages, unit) ||
      !stride_ok(c->k_token_stride, DSA_PAGE_TOKENS, unit) || !stride_ok(c->v_token_stride, DSA_PAGE_TOKENS, unit) ||
      !stride_ok(c->k_head_stride, heads, unit) || !stride_ok(c->v_head_stride, heads, unit))
    return fail(DSA_ERR_INVALID_ARG, "cache strides must be multiples of 16 bytes");
  if (!apart(c->k_page_stride, pages) || !apart(c->v_page_stride, pages) ||
      !apart(c->k_token_stride, DSA_PAGE_TOKENS) || !apart(c->v_token_stride, DSA_PAGE_TOKENS) ||
      !apart(c->k_head_stride, heads) || !apart(c->v_head_stride, heads))
    return fail(DSA_ERR_INVALID_ARG, "a cache stride of 0 over more than one element");
  if (!c->k || !c->v) return fail(DSA_ERR_INVALID_ARG, "null cache pointer");
  if (!aligned(c->k, 16) || !aligned(c->v, 16))
    return fail(DSA_ERR_INVALID_ARG, "the caches must be 16-byte aligned");
  if (c->type == DSA_TYPE_E4M3) {
    if (!c->k_scale || !c->v_scale) return fail(DSA_ERR_INVALID_ARG, "an E4M3 cache needs k_scale and v_scale");
    if (!aligned(c->k_scale, 16) || !aligned(c->v_scale, 16) || !stride_ok(c->k_scale_page_stride, pages, 4) ||
        !stride_ok(c->v_scale_page_stride, pages, 4) || !stride_ok(c->k_scale_head_stride, heads, 4) ||
        !stride_ok(c->v_scale_head_stride, heads, 4))
      return fail(DSA_ERR_INVALID_ARG, "scales must be 16-byte aligned, strides multiples of 4 elements");
    if (written && (!apart(c->k_scale_page_stride, pages) || !apart(c->v_scale_page_stride, pages) ||
                    !apart(c->k_scale_head_stride, heads) || !apart(c->v_scale_head_stride, heads)))
      return fail(DSA_ERR_INVALID_ARG, "a stride of 0 over more than one element of scales that are written");
  }
  return DSA_OK;
}

template <typename P>
void set_cache(P* p, const dsa_kv_cache* c) {
  const int size = element_bytes(c->type);
  p->cache[0] = static_cast<uint8_t*>(c->k);
  p->cache[1] = static_cast<uint8_t*>(c->v);
  p->page_stride[0] = c->k_page_stride * size;
  p->page_stride[1] = c->v_page_stride * size;
  p->token_stride[0] = c->k_token_stride * size;
  p->token_stride[1] = c->v_token_stride * size;
  p->head_stride[0] = c->k_head_stride * size;
  p->head_stride[1] = c->v_head_stride * size;
  p->scale[0] = c->k_scale;
  p->scale[1] = c->v_scale;
  p->scale_page[0] = c->k_scale_page_stride;
  p->scale_page[1] = c->v_scale_page_stride;
  p->scale_head[0] = c->k_scale_head_stride;
  p->scale_head[1] = c->v_scale_head_stride;
  p->num_pages = c->num_pages;
}

// ---------------------------------------------------------------- attention
int attention_grid() {
  const int n = sm_count();
  return n <= 0 || n > dsa::kAttnMaxGrid ? dsa::kAttnMaxGrid : n;
}

// Workspace: arrival counters of split units, then their parts' maxima and
// sums and their outputs (two slots of 256 rows for every CTA).
constexpr size_t kAttnCounterBytes = 2048;
static_assert(kAttnCounterBytes >= 3 * dsa::kAttnMaxGrid * 4, "counters");
size_t attention_part_rows() { return (size_t)attention_grid() * 2 * 256; }

// A map over up to four dimensions, innermost first; strides in bytes (of
// dimensions 1 on).  A dimension of one element may have any stride: it gets
// one that the encoder takes.
int make_map(CUtensorMap* m, const char* what, CUtensorMapDataType type, int size, const void* base, int rank,
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

template <int DP, bool BF16, bool FP8>
int launch_attention(const dsa::AttnParams& p, int grid, cudaStream_t st) {
  using C = dsa::AttnCfg<DP, FP8>;
  static PerDevice allowed;
  if (const int rc = allow_smem(allowed, (const void*)dsa::paged_attention_kernel<DP, BF16, FP8>, C::kSmem)) return rc;
  const CUtensorMapDataType type = BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  CUtensorMap tq, tq32, tkv[2];
  const int64_t qd[3] = {p.D, p.Hq, p.T}, qs[2] = {p.q_head * 2, p.q_token * 2};
  const int qb[3] = {64, p.group, p.tile_tokens};
  if (const int rc = make_map(&tq, "q", type, 2, p.q, 3, qd, qs, qb, true)) return rc;
  const int qb32[3] = {64, p.group, std::max(1, p.tile_tokens32)};
  if (const int rc = make_map(&tq32, "q", type, 2, p.q, 3, qd, qs, qb32, true)) return rc;
  // boxes are 128 bytes wide: 64 16-bit dimensions, 128 E4M3 codes (zeros past
  // the head's); V's codes are converted from plain rows
  const int64_t kd[4] = {p.D, p.Hkv, DSA_PAGE_TOKENS, p.num_pages};
  const int kb[4] = {FP8 ? 128 : 64, 1, DSA_PAGE_TOKENS, 1};
  const char* const names[2] = {"k_cache", "v_cache"};
  for (int i = 0; i < 2; ++i) {
    const int64_t ks[3] = {p.head_stride[i], p.token_stride[i], p.page_stride[i]};
    if (const int rc = make_map(&tkv[i], names[i], FP8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : type, FP8 ? 1 : 2, p.cache[i],
                                4, kd, ks, kb, !FP8 || i == 0))
      return rc;
  }
  dsa::paged_attention_kernel<DP, BF16, FP8><<<grid, C::kThreads, C::kSmem, st>>>(tq, tq32, tkv[0], tkv[1], p);
  set_last_launches(1);
  return check_launch("paged_attention_kernel");
}

// Pieces of 8 elements that a thread has of a row.  One where rows are few,
// whose time is a row's latency, or narrow, where more would leave a warp's
// lanes without any; four where many 16-bit rows follow each other, so that
// the shuffles and the barrier of a row's sum cost fewer warps and the loads of
// four rows an SM are under way (16,384 rows of 7168 bf16: 139 us against
// 180, of 256: 18.0 against 11.5; 200 rows of 4096: 4.9 against 4.3); FP32
// rows, whose pieces are twice the bytes, gain nothing by it (16,384 rows of
// 4096: 128 against 124).  Rows too wide for that: four pieces, then eight.
constexpr int kNormFewRows = 8;  // to an SM
constexpr int kNormNarrow = 1024;
template <typename T, bool VEC>
void launch_norm(const dsa::NormParams& p, cudaStream_t st) {
  const int n8 = (p.N + 7) / 8;
  const bool one = sizeof(T) == 4 || p.T <= kNormFewRows * sm_count() || p.N < kNormNarrow;
  const auto block = [&](int vpt) { return std::max(32, ((n8 + vpt - 1) / vpt + 31) / 32 * 32); };
  if (one && block(1) <= 1024)
    dsa::add_rms_norm_kernel<T, VEC, 1><<<p.T, block(1), 0, st>>>(p);
  else if (block(4) <= 512)
    dsa::add_rms_norm_kernel<T, VEC, 4><<<p.T, block(4), 0, st>>>(p);
  else
    dsa::add_rms_norm_kernel<T, VEC, 8><<<p.T, block(8), 0, st>>>(p);
}

}  // namespace

extern "C" {

int dsa_block_tables_build(const int32_t* query_lens, const int32_t* seq_lens, int R,
                           const int32_t* free_pages, int num_free, int32_t* block_table,
                           int max_blocks, int T, int32_t* query_start_loc, int32_t* positions,
                           int64_t* slot_mapping, int32_t* pages_used, int32_t* dev_status,
                           dsa_stream_t stream) {
  set_last_launches(0);
  if (T < 0) return fail(DSA_ERR_INVALID_ARG, "T=%d < 0", T);
  if (R < 1) return fail(DSA_ERR_INVALID_ARG, "R=%d < 1", R);
  if (R > dsa::kTablesMaxRequests)
    return fail(DSA_ERR_UNSUPPORTED, "R=%d > %d", R, dsa::kTablesMaxRequests);
  if (max_blocks < 1) return fail(DSA_ERR_INVALID_ARG, "max_blocks < 1");
  if (num_free < 0) return fail(DSA_ERR_INVALID_ARG, "num_free=%d < 0", num_free);
  if (!query_lens || !seq_lens || (num_free && !free_pages) || !block_table || !query_start_loc ||
      (T && (!positions || !slot_mapping)) || !pages_used)
    return fail(DSA_ERR_INVALID_ARG, "null pointer");
  constexpr int kMost = 2 * (dsa::kTablesMaxRequests + 1) * 4;
  static PerDevice allowed;
  if (const int rc = allow_smem(allowed, (const void*)dsa::block_tables_kernel, kMost)) return rc;
  const dsa::TablesParams p{query_lens, seq_lens, R, free_pages, num_free, block_table, max_blocks, T,
                            query_start_loc, positions, slot_mapping, pages_used, dev_status};
  const int64_t most = std::max<int64_t>(1, ((int64_t)T + dsa::kTablesThreads - 1) / dsa::kTablesThreads);
  const int grid = (int)std::min<int64_t>(most, std::max(1, sm_count()));
  dsa::block_tables_kernel<<<grid, dsa::kTablesThreads, 2 * (R + 1) * 4, (cudaStream_t)stream>>>(p);
  set_last_launches(1);
  return check_launch("block_tables_kernel");
}

int dsa_kv_write(const void* k, int64_t k_token_stride, int64_t k_head_stride, const void* v,
                 int64_t v_token_stride, int64_t v_head_stride, int type, int T,
                 const int64_t* slot_mapping, const dsa_kv_cache* cache, int32_t* dev_status,
                 dsa_stream_t stream) {
  set_last_launches(0);
  if (T < 0) return fail(DSA_ERR_INVALID_ARG, "T=%d < 0", T);
  if (const int rc = check_cache(cache, type, true)) return rc;
  if (T == 0) return DSA_OK;
  if (!k || !v || !slot_mapping) return fail(DSA_ERR_INVALID_ARG, "null pointer");
  const int heads = cache->num_kv_heads;
  if (!aligned(k, 16) || !aligned(v, 16) || !stride_ok(k_token_stride, T, 8) || !stride_ok(v_token_stride, T, 8) ||
      !stride_ok(k_head_stride, heads, 8) || !stride_ok(v_head_stride, heads, 8))
    return fail(DSA_ERR_INVALID_ARG, "k and v must be 16-byte aligned, strides multiples of 8 elements");
  dsa::KvWriteParams p{};
  p.src[0] = static_cast<const uint16_t*>(k);
  p.src[1] = static_cast<const uint16_t*>(v);
  p.src_token[0] = k_token_stride;
  p.src_token[1] = v_token_stride;
  p.src_head[0] = k_head_stride;
  p.src_head[1] = v_head_stride;
  p.slots = slot_mapping;
  p.T = T;
  p.heads = cache->num_kv_heads;
  p.dim = cache->head_dim;
  set_cache(&p, cache);
  p.status = dev_status;
  // a CTA's tokens: as many as make one pass of its lanes, at least one
  p.tokens = std::max(1, dsa::kKvThreads / 16 / heads);
  p.per_token = p.tokens > 1 ? (65536 + heads - 1) / heads : 0;
  const unsigned grid = (unsigned)(((int64_t)T + p.tokens - 1) / p.tokens);
  const cudaStream_t st = (cudaStream_t)stream;
  if (cache->type != DSA_TYPE_E4M3)
    dsa::kv_write_kernel<true, false><<<grid, dsa::kKvThreads, 0, st>>>(p);
  else if (type == DSA_TYPE_BF16)
    dsa::kv_write_kernel<true, true><<<grid, dsa::kKvThreads, 0, st>>>(p);
  else
    dsa::kv_write_kernel<false, true><<<grid, dsa::kKvThreads, 0, st>>>(p);
  set_last_launches(1);
  return check_launch("kv_write_kernel");
}

size_t dsa_paged_attention_workspace_bytes(void) {
  return kAttnCounterBytes + attention_part_rows() * (128 * sizeof(float) + sizeof(float2));
}

int dsa_paged_attention(const void* q, int64_t q_token_stride, int64_t q_head_stride, int type, int T,
                        int Hq, const dsa_kv_cache* cache, const int32_t* query_start_loc,
                        const int32_t* seq_lens, int R, const int32_t* block_table, int max_blocks,
                        float softmax_scale, int window, int num_sinks, void* out,
                        int64_t out_token_stride, int64_t out_head_stride, float* lse,
                        void* workspace, size_t workspace_bytes, int32_t* dev_status,
                        dsa_stream_t stream) {
  set_last_launches(0);
  if (T < 0) return fail(DSA_ERR_INVALID_ARG, "T=%d < 0", T);
  if (R < 1) return fail(DSA_ERR_INVALID_ARG, "R=%d < 1", R);
  if (const int rc = check_cache(cache, type, false)) return rc;
  if (cache->type == DSA_TYPE_E4M3 && type != DSA_TYPE_BF16)
    return fail(DSA_ERR_UNSUPPORTED, "an E4M3 cache takes BF16 queries: FP16's 11 significant bits do not fit their two E4M3 terms");
  if (Hq < 1 || Hq % cache->num_kv_heads || Hq / cache->num_kv_heads > 128)
    return fail(DSA_ERR_UNSUPPORTED, "Hq=%d: a multiple of num_kv_heads=%d, at most 128 query heads to a key head",
                Hq, cache->num_kv_heads);
  if (max_blocks < 1) return fail(DSA_ERR_INVALID_ARG, "max_blocks < 1");
  if (!(softmax_scale > 0.0f) || !(softmax_scale < 1e30f))
    return fail(DSA_ERR_INVALID_ARG, "softmax_scale must be positive and finite");
  if (window < 0 || num_sinks < 0) return fail(DSA_ERR_INVALID_ARG, "window and num_sinks must not be negative");
  if (T == 0) return DSA_OK;
  if (!q || !query_start_loc || !seq_lens || !block_table || !out || !workspace)
    return fail(DSA_ERR_INVALID_ARG, "null pointer");
  if (!aligned(q, 16) || !aligned(out, 16) || !stride_ok(q_token_stride, T, 8) || !stride_ok(q_head_stride, Hq, 8) ||
      !stride_ok(out_token_stride, T, 8) || !stride_ok(out_head_stride, Hq, 8))
    return fail(DSA_ERR_INVALID_ARG, "q and out must be 16-byte aligned, strides multiples of 8 elements");
  if (!apart(q_token_stride, T) || !apart(q_head_stride, Hq) || !apart(out_token_stride, T) ||
      !apart(out_head_stride, Hq))
    return fail(DSA_ERR_INVALID_ARG, "a stride of 0 over more than one element of q or out");
  if (!aligned(workspace, 256)) return fail(DSA_ERR_INVALID_ARG, "workspace is not 256-byte aligned");
  const size_t need = dsa_paged_attention_workspace_bytes();
  if (workspace_bytes < need)
    return fail(DSA_ERR_WORKSPACE_TOO_SMALL, "workspace %zu bytes < %zu needed", workspace_bytes, need);
  dsa::AttnParams p{};
  p.q = static_cast<const uint16_t*>(q);
  p.q_token = q_token_stride;
  p.q_head = q_head_stride;
  p.out = static_cast<uint16_t*>(out);
  p.out_token = out_token_stride;
  p.out_head = out_head_stride;
  p.lse = lse;
  set_cache(&p, cache);
  p.start = query_start_loc;
  p.seq_lens = seq_lens;
  p.block_table = block_table;
  p.R = R;
  p.max_blocks = max_blocks;
  p.T = T;
  p.Hq = Hq;
  p.Hkv = cache->num_kv_heads;
  p.D = cache->head_dim;
  p.window = window;
  p.sinks = num_sinks;
  p.scale_log2 = (float)((double)softmax_scale * 1.4426950408889634);
  p.status = dev_status;
  p.give_up = env_int("DSA_WAIT_LIMIT", (int)dsa::kWaitLimit, 0, (int)dsa::kWaitLimit) == 0;
  p.group = Hq / p.Hkv;
  p.tile_tokens = 128 / p.group;
  p.tile_tokens32 = 32 / p.group;
  p.sink_tiles = num_sinks / dsa::kAttnTile + (num_sinks % dsa::kAttnTile != 0);
  if (sm_count() <= 0) return fail(DSA_ERR_CUDA, "no CUDA device");
  const int grid = attention_grid();
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  p.counter = reinterpret_cast<uint32_t*>(ws);
  p.part = reinterpret_cast<float*>(ws + kAttnCounterBytes);
  p.part_ml = reinterpret_cast<float2*>(p.part + attention_part_rows() * 128);
  const cudaStream_t st = (cudaStream_t)stream;
  const bool wide = p.D > 64;
  if (cache->type == DSA_TYPE_E4M3)
    return launch_attention<128, true, true>(p, grid, st);
  if (type == DSA_TYPE_BF16)
    return wide ? launch_attention<128, true, false>(p, grid, st) : launch_attention<64, true, false>(p, grid, st);
  return wide ? launch_attention<128, false, false>(p, grid, st) : launch_attention<64, false, false>(p, grid, st);
}

int dsa_add_rms_norm(const void* x, int64_t x_stride, const void* residual, int64_t residual_stride,
                     const void* weight, int type, int T, int N, float eps, void* residual_out,
                     int64_t residual_out_stride, void* out, int64_t out_stride, uint8_t* codes,
                     float* scales, dsa_stream_t stream) {
  set_last_launches(0);
  if (T < 0) return fail(DSA_ERR_INVALID_ARG, "T=%d < 0", T);
  if (N < 1) return fail(DSA_ERR_INVALID_ARG, "N=%d < 1", N);
  if (N > dsa::kNormMaxWidth) return fail(DSA_ERR_UNSUPPORTED, "N=%d > %d", N, dsa::kNormMaxWidth);
  if (type != DSA_TYPE_BF16 && type != DSA_TYPE_FP16 && type != DSA_TYPE_FP32)
    return fail(DSA_ERR_UNSUPPORTED, "type=%d: BF16, FP16 or FP32 is wanted", type);
  if (!(eps >= 0.0f) || !(eps < 1e30f)) return fail(DSA_ERR_INVALID_ARG, "eps must be finite and not negative");
  if (!out && !codes) return fail(DSA_ERR_INVALID_ARG, "neither out nor codes is given");
  if ((codes == nullptr) != (scales == nullptr))
    return fail(DSA_ERR_INVALID_ARG, "codes and scales are given together or not at all");
  if (x_stride < N || (residual && residual_stride < N) || (residual_out && residual_out_stride < N) ||
      (out && out_stride < N))
    return fail(DSA_ERR_INVALID_ARG, "a row stride is shorter than N");
  if (T == 0) return DSA_OK;
  if (!x || !weight) return fail(DSA_ERR_INVALID_ARG, "null pointer");
  const int size = element_bytes(type);
  const dsa::NormParams p{x, residual, weight, residual_out, out, codes, scales, x_stride, residual_stride,
                          residual_out_stride, out_stride, T, N, eps};
  auto row16 = [&](const void* ptr, int64_t stride) { return !ptr || (aligned(ptr, 16) && stride * size % 16 == 0); };
  const bool vec = N % 8 == 0 && row16(x, x_stride) && row16(residual, residual_stride) && aligned(weight, 16) &&
                   row16(residual_out, residual_out_stride) && row16(out, out_stride) && aligned(codes, 8);
  const cudaStream_t st = (cudaStream_t)stream;
  if (type == DSA_TYPE_BF16)
    vec ? launch_norm<__nv_bfloat16, true>(p, st) : launch_norm<__nv_bfloat16, false>(p, st);
  else if (type == DSA_TYPE_FP16)
    vec ? launch_norm<__half, true>(p, st) : launch_norm<__half, false>(p, st);
  else
    vec ? launch_norm<float, true>(p, st) : launch_norm<float, false>(p, st);
  set_last_launches(1);
  return check_launch("add_rms_norm_kernel");
}

}  // extern "C"
