// Scored paged attention: the entry points (argument checks, dispatch) and the kernel.
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "paged_kv.h"
#include "pkv_internal.h"
#include "pkv_scored.cuh"

namespace pkv {
namespace {

// One warp per (query token, head): it walks the visible keys in order, its lanes holding D / 32 dims each,
// with a running maximum and sum. C: the cache's element type.
template <int D, typename C>
__device__ __forceinline__ void load_dims(float (&v)[D / 32], const unsigned char* row, int lane) {
  constexpr int DPL = D / 32, EB = CacheFmt<C>::EB;
#pragma unroll
  for (int e = 0; e < DPL / 2; ++e) {
    const unsigned char* at = row + (lane * DPL + 2 * e) * EB;
    const float2 f = CacheFmt<C>::pair(EB == 1 ? *reinterpret_cast<const uint16_t*>(at)
                                               : *reinterpret_cast<const uint32_t*>(at));
    v[2 * e] = f.x;
    v[2 * e + 1] = f.y;
  }
}

template <typename T, typename C, int D>
__global__ void __launch_bounds__(128) pkv_scored_row_kernel(const DecodeParams p, const ScoreParams sc, int block_size) {
  pdl_begin();
  constexpr int DPL = D / 32, EB = CacheFmt<C>::EB;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = blockIdx.y, s = blockIdx.z;
  const int i = blockIdx.x * 4 + warp;
  const bool reporter = blockIdx.x == 0 && h == 0 && threadIdx.x == 0;
  const int ctx = clamp_context(p, s, reporter);
  int q0 = 0;
  const int q_len = scored_query_len(sc, s, ctx, q0);
  if (q_len < 0 && reporter) atomicOr(p.err, PKV_DEVERR_QUERY);
  if (i >= q_len) return;
  const int t = q0 + i, pos = ctx - q_len + i, g = h / p.group;
  const size_t row = (size_t)t * p.num_heads + h;
  int lo, hi;
  scored_span(sc, t, pos, ctx, lo, hi);
  const float slope = sc.slopes ? sc.slopes[h] * 1.4426950408889634f : 0.f;
  float q[DPL], acc[DPL], m = -INFINITY, l = 0.f;
  load_dims<D, T>(q, static_cast<const unsigned char*>(p.query) + row * D * 2, lane);
#pragma unroll
  for (int e = 0; e < DPL; ++e) acc[e] = 0.f;
  for (int j = lo; j < hi; ++j) {
    const int phys = p.block_tables[(size_t)s * p.max_blocks_per_seq + j / block_size];
    if ((unsigned)phys >= (unsigned)p.num_blocks) {
      if (lane == 0) atomicOr(p.err, PKV_DEVERR_BLOCK_ID);
      continue;
    }
    const size_t at = (((size_t)phys * p.num_kv_heads + g) * block_size + j % block_size) * D * EB;
    float k[DPL], v[DPL], d = 0.f;
    load_dims<D, C>(k, p.key_cache + at, lane);
    load_dims<D, C>(v, p.value_cache + at, lane);
#pragma unroll
    for (int e = 0; e < DPL; ++e) d = fmaf(q[e], k[e], d);
    const float x = score_value(sc, warp_sum(d), p.scale_log2) - slope * fabsf((float)(pos - j));
    const float mn = fmaxf(m, x), ms = mn == -INFINITY ? 0.f : mn;
    const float f = fast_exp2(m - ms), w = fast_exp2(x - ms);
    l = fmaf(l, f, w);
#pragma unroll
    for (int e = 0; e < DPL; ++e) acc[e] = fmaf(acc[e], f, w * v[e]);
    m = mn;
  }
  const float inv = l != 0.f ? p.v_scale / l : 0.f;
  uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<T*>(p.out) + row * D + lane * DPL);
#pragma unroll
  for (int e = 0; e < DPL / 2; ++e) dst[e] = Elem<T>::pack2(acc[2 * e] * inv, acc[2 * e + 1] * inv);
}

// Everything a call passes, under the header's names.
struct ScoredCall {
  void* out;
  const void *query, *key_cache, *value_cache;
  const int32_t* block_tables;
  int32_t max_blocks_per_seq;
  const int32_t *context_lens, *query_start_loc;  // query_start_loc null: one query token per sequence
  int32_t num_seqs, num_query_tokens, max_query_len, max_context_len;
  float scale, softcap;
  const float* alibi_slopes;
  int32_t window;
  const int32_t *key_begin, *key_end;
  int32_t block_size, num_heads, num_kv_heads, head_dim, num_blocks;
  pkv_dtype_t dtype;
  bool fp8;
  float k_scale, v_scale;
  int32_t partition_size;
  void* workspace;
  size_t workspace_bytes;
  cudaStream_t stream;
};

bool aligned(const void* ptr, uintptr_t n) { return (reinterpret_cast<uintptr_t>(ptr) & (n - 1)) == 0; }

pkv_status_t scored_impl(const ScoredCall& c, bool decode) {
  set_last_error_message("");
  if (c.num_seqs < 0 || c.num_query_tokens < 0 || c.max_query_len < 0)
    return fail(PKV_ERR_INVALID_ARG, "num_seqs, num_query_tokens and max_query_len must be >= 0");
  if (c.dtype != PKV_F16 && c.dtype != PKV_BF16) return fail(PKV_ERR_INVALID_ARG, "unknown dtype %d", (int)c.dtype);
  if (c.num_heads <= 0 || c.num_kv_heads <= 0 || c.num_heads % c.num_kv_heads)
    return fail(PKV_ERR_INVALID_ARG, "num_heads (%d) must be a positive multiple of num_kv_heads (%d)", c.num_heads,
                c.num_kv_heads);
  if (c.num_blocks <= 0 || c.max_blocks_per_seq <= 0)
    return fail(PKV_ERR_INVALID_ARG, "num_blocks and max_blocks_per_seq must be > 0");
  if (c.head_dim != 64 && c.head_dim != 128)
    return fail(PKV_ERR_UNSUPPORTED, "head_dim %d (supported: 64, 128)", c.head_dim);
  if (c.block_size != 8 && c.block_size != 16 && c.block_size != 32)
    return fail(PKV_ERR_UNSUPPORTED, "block_size %d (supported: 8, 16, 32)", c.block_size);
  if (!isfinite(c.scale)) return fail(PKV_ERR_INVALID_ARG, "scale is not finite");
  if (!(isfinite(c.softcap) && c.softcap >= 0.f))
    return fail(PKV_ERR_INVALID_ARG, "softcap must be finite and >= 0 (0: no cap)");
  if (c.softcap > 0.f && !isfinite(c.scale / c.softcap))
    return fail(PKV_ERR_INVALID_ARG, "scale / softcap is not finite");
  if (c.window < 0) return fail(PKV_ERR_INVALID_ARG, "window must be >= 0 (0: no window)");
  if (c.fp8 && !(isfinite(c.k_scale) && isfinite(c.v_scale) && c.k_scale > 0.f && c.v_scale > 0.f))
    return fail(PKV_ERR_INVALID_ARG, "k_scale and v_scale must be finite and > 0");
  if (c.fp8 && c.head_dim != 128)
    return fail(PKV_ERR_UNSUPPORTED, "scored attention over an FP8 pool needs head_dim 128 (got %d)", c.head_dim);
  if (c.max_context_len < 0) return fail(PKV_ERR_INVALID_ARG, "max_context_len < 0");
  if ((long long)c.max_context_len > (long long)c.max_blocks_per_seq * c.block_size)
    return fail(PKV_ERR_INVALID_ARG, "max_context_len %d exceeds max_blocks_per_seq * block_size = %lld",
                c.max_context_len, (long long)c.max_blocks_per_seq * c.block_size);
  if (!decode && c.max_query_len > c.max_context_len)
    return fail(PKV_ERR_INVALID_ARG, "max_query_len %d exceeds max_context_len %d", c.max_query_len,
                c.max_context_len);
  if (c.num_seqs > 65535 || c.num_heads > 65535)
    return fail(PKV_ERR_UNSUPPORTED, "num_seqs and num_heads must be <= 65535");
  if ((long long)c.num_blocks * c.num_kv_heads * c.block_size >= (1LL << 31))
    return fail(PKV_ERR_UNSUPPORTED, "pool rows num_blocks * num_kv_heads * block_size must be < 2^31");
  if ((long long)c.num_query_tokens * c.num_heads >= (1LL << 31))
    return fail(PKV_ERR_UNSUPPORTED, "num_query_tokens * num_heads must be < 2^31");
  if (c.num_seqs == 0 || c.num_query_tokens == 0 || c.max_query_len == 0) return PKV_OK;
  if (!c.out || !c.query || !c.key_cache || !c.value_cache || !c.block_tables || !c.context_lens ||
      (!decode && !c.query_start_loc))
    return fail(PKV_ERR_INVALID_ARG, "null pointer argument");
  if (!aligned(c.out, 16) || !aligned(c.query, 16) || !aligned(c.key_cache, 16) || !aligned(c.value_cache, 16))
    return fail(PKV_ERR_INVALID_ARG, "out, query and caches must be 16-byte aligned");

  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  DecodeParams p{};
  p.err = device_error_word(dev);
  if (!p.err) return fail(PKV_ERR_CUDA, "device error word unavailable on device %d", dev);
  const float scale = c.fp8 ? c.scale * c.k_scale : c.scale;  // of a product of the stored values
  p.out = c.out;
  p.query = c.query;
  p.key_cache = static_cast<const unsigned char*>(c.key_cache);
  p.value_cache = static_cast<const unsigned char*>(c.value_cache);
  p.block_tables = c.block_tables;
  p.context_lens = c.context_lens;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.v_scale = c.fp8 ? c.v_scale : 1.f;
  p.max_blocks_per_seq = c.max_blocks_per_seq;
  p.num_heads = c.num_heads;
  p.num_kv_heads = c.num_kv_heads;
  p.group = c.num_heads / c.num_kv_heads;
  p.num_blocks = c.num_blocks;
  p.ctx_limit = c.max_context_len;
  ScoreParams sc{};
  sc.slopes = c.alibi_slopes;
  sc.key_begin = c.key_begin;
  sc.key_end = c.key_end;
  sc.query_start_loc = decode ? nullptr : c.query_start_loc;
  sc.window = c.window;
  sc.num_query_tokens = c.num_query_tokens;
  sc.max_query_len = c.max_query_len;
  if (c.softcap > 0.f) {
    sc.cap_in = scale / c.softcap;
    sc.cap_out = c.softcap * 1.4426950408889634f;
  }
  const dim3 grid((unsigned)((c.max_query_len + 3) / 4), (unsigned)c.num_heads, (unsigned)c.num_seqs);
  auto run = [&](auto kern) { return launch_kernel(kern, grid, dim3(128), 0, c.stream, p, sc, (int)c.block_size); };
  using F = __half;
  using B = __nv_bfloat16;
  using E = __nv_fp8_e4m3;
  if (c.fp8)
    e = c.dtype == PKV_F16 ? run(pkv_scored_row_kernel<F, E, 128>) : run(pkv_scored_row_kernel<B, E, 128>);
  else if (c.head_dim == 128)
    e = c.dtype == PKV_F16 ? run(pkv_scored_row_kernel<F, F, 128>) : run(pkv_scored_row_kernel<B, B, 128>);
  else
    e = c.dtype == PKV_F16 ? run(pkv_scored_row_kernel<F, F, 64>) : run(pkv_scored_row_kernel<B, B, 64>);
  if (e != cudaSuccess) return cuda_fail(e, "scored attention launch");
  return PKV_OK;
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" {

size_t paged_attention_scored_workspace_size(int32_t num_query_tokens, int32_t num_heads, int32_t num_kv_heads,
                                             int32_t head_dim, int32_t block_size, int32_t max_query_len,
                                             int32_t max_context_len, int32_t window, int32_t partition_size) {
  (void)num_query_tokens, (void)num_heads, (void)num_kv_heads, (void)head_dim, (void)block_size;
  (void)max_query_len, (void)max_context_len, (void)window, (void)partition_size;
  return 0;
}

pkv_status_t paged_attention_decode_scored(void* out, const void* query, const void* key_cache,
                                           const void* value_cache, const int32_t* block_tables,
                                           int32_t max_blocks_per_seq, const int32_t* context_lens, int32_t num_seqs,
                                           int32_t max_context_len, float scale, float softcap,
                                           const float* alibi_slopes, int32_t window, const int32_t* key_begin,
                                           int32_t block_size, int32_t num_heads, int32_t num_kv_heads,
                                           int32_t head_dim, int32_t num_blocks, pkv_dtype_t dtype,
                                           int32_t partition_size, void* workspace, size_t workspace_bytes,
                                           cudaStream_t stream) {
  return scored_impl({out, query, key_cache, value_cache, block_tables, max_blocks_per_seq, context_lens, nullptr,
                      num_seqs, num_seqs, 1, max_context_len, scale, softcap, alibi_slopes, window, key_begin, nullptr,
                      block_size, num_heads, num_kv_heads, head_dim, num_blocks, dtype, false, 1.f, 1.f,
                      partition_size, workspace, workspace_bytes, stream},
                     true);
}

pkv_status_t paged_attention_decode_scored_fp8(void* out, const void* query, const void* key_cache,
                                               const void* value_cache, const int32_t* block_tables,
                                               int32_t max_blocks_per_seq, const int32_t* context_lens,
                                               int32_t num_seqs, int32_t max_context_len, float scale, float softcap,
                                               const float* alibi_slopes, int32_t window, const int32_t* key_begin,
                                               int32_t block_size, int32_t num_heads, int32_t num_kv_heads,
                                               int32_t head_dim, int32_t num_blocks, pkv_dtype_t dtype, float k_scale,
                                               float v_scale, int32_t partition_size, void* workspace,
                                               size_t workspace_bytes, cudaStream_t stream) {
  return scored_impl({out, query, key_cache, value_cache, block_tables, max_blocks_per_seq, context_lens, nullptr,
                      num_seqs, num_seqs, 1, max_context_len, scale, softcap, alibi_slopes, window, key_begin, nullptr,
                      block_size, num_heads, num_kv_heads, head_dim, num_blocks, dtype, true, k_scale, v_scale,
                      partition_size, workspace, workspace_bytes, stream},
                     true);
}

pkv_status_t paged_attention_multi_query_scored(
    void* out, const void* query, const void* key_cache, const void* value_cache, const int32_t* block_tables,
    int32_t max_blocks_per_seq, const int32_t* context_lens, const int32_t* query_start_loc, int32_t num_seqs,
    int32_t num_query_tokens, int32_t max_query_len, int32_t max_context_len, float scale, float softcap,
    const float* alibi_slopes, int32_t window, const int32_t* key_begin, const int32_t* key_end, int32_t block_size,
    int32_t num_heads, int32_t num_kv_heads, int32_t head_dim, int32_t num_blocks, pkv_dtype_t dtype,
    int32_t partition_size, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  return scored_impl({out, query, key_cache, value_cache, block_tables, max_blocks_per_seq, context_lens,
                      query_start_loc, num_seqs, num_query_tokens, max_query_len, max_context_len, scale, softcap,
                      alibi_slopes, window, key_begin, key_end, block_size, num_heads, num_kv_heads, head_dim,
                      num_blocks, dtype, false, 1.f, 1.f, partition_size, workspace, workspace_bytes, stream},
                     false);
}

pkv_status_t paged_attention_multi_query_scored_fp8(
    void* out, const void* query, const void* key_cache, const void* value_cache, const int32_t* block_tables,
    int32_t max_blocks_per_seq, const int32_t* context_lens, const int32_t* query_start_loc, int32_t num_seqs,
    int32_t num_query_tokens, int32_t max_query_len, int32_t max_context_len, float scale, float softcap,
    const float* alibi_slopes, int32_t window, const int32_t* key_begin, const int32_t* key_end, int32_t block_size,
    int32_t num_heads, int32_t num_kv_heads, int32_t head_dim, int32_t num_blocks, pkv_dtype_t dtype, float k_scale,
    float v_scale, int32_t partition_size, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  return scored_impl({out, query, key_cache, value_cache, block_tables, max_blocks_per_seq, context_lens,
                      query_start_loc, num_seqs, num_query_tokens, max_query_len, max_context_len, scale, softcap,
                      alibi_slopes, window, key_begin, key_end, block_size, num_heads, num_kv_heads, head_dim,
                      num_blocks, dtype, true, k_scale, v_scale, partition_size, workspace, workspace_bytes, stream},
                     false);
}

}  // extern "C"
