// Scored paged attention: the entry points (argument checks, the plan of a call, dispatch) and the reduce kernel.
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "paged_kv.h"
#include "pkv_internal.h"
#include "pkv_reduce.cuh"
#include "pkv_scored.cuh"

namespace pkv {
namespace {

// Merge of the partials of rows that span several partitions: a CTA takes 4 heads (a warp each) of
// kReduceTokens query tokens of a sequence. Each row's first and last partition follow from its interval.
constexpr int kReduceTokens = 8;
constexpr int kTreeReduceCtas = 4864;  // two waves of CTAs of four warps
template <typename T, int D>
__global__ void __launch_bounds__(32 * kReduceRows)
    pkv_scored_reduce_kernel(const DecodeParams p, const ScoreParams sc, int block_size) {
  pdl_begin();
  const int s = blockIdx.x, h = blockIdx.y * kReduceRows + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (h >= p.num_heads) return;
  const int c = p.context_lens[s];
  const int ctx = c < 0 ? 0 : (c > p.ctx_limit ? p.ctx_limit : c);
  int q0 = 0;
  const int q_len = scored_query_len(sc, s, ctx, q0);
  const int base = scored_base(sc, ctx, q_len, block_size);
  for (int i = blockIdx.z * kReduceTokens; i < min(q_len, (int)(blockIdx.z + 1) * kReduceTokens); ++i) {
    int lo, hi;
    scored_span(sc, q0 + i, ctx - q_len + i, ctx, lo, hi);
    const RowParts parts = row_parts(lo, hi, base, p.partition_size);
    if (parts.direct()) continue;  // written by the attention kernel
    const size_t row = (size_t)(q0 + i) * p.num_heads + h;
    const size_t at = row * p.max_partitions + parts.first;
    float mp, lp;
    float o_early[kReduceEarly][D / 32];
    reduce_load_row<D>(p.part_o, p.part_m, p.part_l, at, p.max_partitions - parts.first, lane, mp, lp, o_early);
    reduce_combine_row<T, D>(static_cast<T*>(p.out), p.part_o, p.part_m, p.part_l, at, row,
                             parts.last - parts.first + 1, mp, lp, o_early, lane);
  }
}

// The same for drafted trees: a warp per (query token, head), per_cta query tokens of a sequence a CTA, so that few
// rows of many partitions (one long context) still fill the GPU; eight partials in flight.
template <typename T, int D>
__global__ void __launch_bounds__(32 * kReduceRows)
    pkv_tree_reduce_kernel(const DecodeParams p, const ScoreParams sc, int per_cta) {
  pdl_begin();
  constexpr int DPL = D / 32, BATCH = 8;
  const int s = blockIdx.x, h = blockIdx.y * kReduceRows + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (h >= p.num_heads) return;
  const int c = p.context_lens[s];
  const int ctx = c < 0 ? 0 : (c > p.ctx_limit ? p.ctx_limit : c);
  int q0 = 0;
  const int q_len = scored_query_len(sc, s, ctx, q0);
  const int first = (int)blockIdx.z * per_cta;
  for (int i = first; i < min(q_len, first + per_cta); ++i) {
    int lo, hi;
    scored_span<true>(sc, q0 + i, 0, ctx, lo, hi);
    const RowParts parts = row_parts(lo, hi, 0, p.partition_size);
    if (parts.direct()) continue;  // written by the attention kernel
    const size_t row = (size_t)(q0 + i) * p.num_heads + h, at = row * p.max_partitions + parts.first;
    const int np = parts.last - parts.first + 1;
    float M = -INFINITY;
    for (int k = lane; k < np; k += 32) M = fmaxf(M, p.part_m[at + k]);
    M = warp_max(M);
    float acc[DPL], W = 0.f;
#pragma unroll
    for (int e = 0; e < DPL; ++e) acc[e] = 0.f;
    for (int k0 = 0; k0 < np; k0 += 32) {
      float w = 0.f;  // lane k: the weight of partial k0 + k
      if (k0 + lane < np) {
        const float m = p.part_m[at + k0 + lane];
        w = m == -INFINITY ? 0.f : p.part_l[at + k0 + lane] * fast_exp2(m - M);
      }
      W += w;
      for (int k = 0; k < min(32, np - k0); k += BATCH) {
        float o[BATCH][DPL];
#pragma unroll
        for (int b = 0; b < BATCH; ++b)
#pragma unroll
          for (int e = 0; e < DPL; e += 2) {
            const float2 v = k0 + k + b < np ? *reinterpret_cast<const float2*>(p.part_o + (at + k0 + k + b) * D +
                                                                                lane * DPL + e)
                                             : make_float2(0.f, 0.f);
            o[b][e] = v.x;
            o[b][e + 1] = v.y;
          }
#pragma unroll
        for (int b = 0; b < BATCH; ++b) {
          const float wb = __shfl_sync(kFull, w, k + b);
#pragma unroll
          for (int e = 0; e < DPL; ++e) acc[e] = fmaf(wb, o[b][e], acc[e]);
        }
      }
    }
    W = warp_sum(W);
    const float inv = W > 0.f ? 1.f / W : 0.f;
    uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<T*>(p.out) + row * D + lane * DPL);
#pragma unroll
    for (int e = 0; e < DPL / 2; ++e) dst[e] = Elem<T>::pack2(acc[2 * e] * inv, acc[2 * e + 1] * inv);
  }
}

// How a call runs: partitions of P tokens, np per sequence, and what workspace that needs.
struct ScoredPlan {
  bool tensor;      // the tensor-memory tile, 256 rows a CTA (else the 8-column one)
  int row_tiles;    // row tiles per kv head
  int P, np;
  size_t partials;  // bytes
};

// Rows per kv head (query tokens times heads) from which the tensor-memory tile runs. Measured, us a call, 8-column
// and tensor tile, 64 contexts of 1500 to 4096 tokens with a cap:
//   decode, 2 kv heads    16-bit pool: 24 rows 61, 84; 32 rows 75, 89; 40 rows 89, 90; 48 rows 104, 91
//                         E4M3: 24 rows 58, 98; 32 rows 75, 116; 40 rows 90, 118; 48 rows 104, 117; 64 rows 133, 119
//   multi-query, 4 heads  16-bit pool: 16 rows 150, 209; 24 rows 202, 209; 32 rows 262, 232
//   a kv head, 8 of them  E4M3: 24 rows 200, 279; 32 rows 259, 349; 48 rows 373, 351
int tensor_rows(bool fp8, int max_query_len) { return fp8 ? 41 : max_query_len > 1 ? 25 : 33; }
// Partition sizes as in paged_attention_decode. A small batch is split further: up to three CTAs an SM (tensor
// tile: one), as long as a partition keeps 512 (384) tokens. Measured, us a call: one context of 16384 tokens, 32/8
// heads, 2048-token partitions 31.4, 1024 20.3, 512 19.1, 256 23.4; 16 contexts of 2000 to 4096, 48 heads on one kv
// head (tensor tile), 2048-token partitions 36.7, 1024 24.9, 512 22.0, 384 23.9, 256 27.6, 128 39.0.
constexpr int kScoredPartition = 1024, kScoredPartitionLong = 2048, kScoredLong = 8192;
constexpr int kScoredFill = 456, kScoredFillTensor = 152, kScoredMin = 512, kScoredMinTensor = 384;

constexpr long long kScoredMaxItems = 1ll << 27;  // half a second of empty ones

// The tokens that a sequence's partitions must cover: its context, or what a window leaves visible to its
// query tokens (from the start of the first visible block).
long long scored_span_bound(int block_size, int max_query_len, int max_context_len, int window) {
  const long long w = (long long)window + max_query_len - 1 + block_size - 1;
  return window > 0 && w < max_context_len ? w : max_context_len;
}

ScoredPlan scored_plan(bool fp8, int num_query_tokens, int num_heads, int num_kv_heads, int head_dim, int block_size,
                       int max_query_len, int max_context_len, int window, int partition_size,
                       size_t workspace_bytes = SIZE_MAX) {
  ScoredPlan pl{};
  const long long rows = (long long)max_query_len * (num_heads / num_kv_heads);
  pl.tensor = rows >= tensor_rows(fp8, max_query_len);
  pl.row_tiles = (int)(pl.tensor ? (rows + 255) / 256 : (rows + 7) / 8);
  const long long span = scored_span_bound(block_size, max_query_len, max_context_len, window);
  if (partition_size) {
    pl.P = partition_size;
  } else {
    // The nearest number of partitions of the usual size (tensor tile: one), of equal length; more, down to
    // kScoredMin(Tensor) tokens each, where the CTAs would not fill the GPU.
    // (the batch has at least num_query_tokens / max_query_len sequences)
    const long long seqs = max_query_len > 0 ? ((long long)num_query_tokens + max_query_len - 1) / max_query_len : 0;
    const long long ctas = seqs * num_kv_heads * pl.row_tiles;
    const int p0 = span > kScoredLong ? kScoredPartitionLong : kScoredPartition;
    long long n = pl.tensor ? 1 : span > p0 ? (span + p0 / 2) / p0 : 1;
    const long long fill = ctas > 0 ? ((pl.tensor ? kScoredFillTensor : kScoredFill) + ctas - 1) / ctas : 1;
    const long long most = span / (pl.tensor ? kScoredMinTensor : kScoredMin);
    // (as far as the workspace goes: one that fits a larger batch fits a smaller one, which is split further)
    const size_t one = (size_t)num_query_tokens * num_heads * (head_dim + 2) * sizeof(float);
    const long long room = one ? (long long)(workspace_bytes / one < (1u << 30) ? workspace_bytes / one : 1u << 30) : 1;
    long long more = fill < most ? fill : most;
    if (more > room) more = room;
    if (n < more) n = more;
    long long P = ((span + n - 1) / n + block_size - 1) / block_size * block_size;
    if (!pl.tensor && P > (long long)kMaxPartitionBlocks * block_size) P = (long long)kMaxPartitionBlocks * block_size;
    pl.P = P < block_size ? block_size : (int)P;
  }
  const long long np = (span + pl.P - 1) / pl.P;
  pl.np = np < 1 ? 1 : (int)np;
  pl.partials = pl.np > 1 ? (size_t)num_query_tokens * num_heads * pl.np * (head_dim + 2) * sizeof(float) : 0;
  return pl;
}

// Tree attention: the tensor-memory tile (128 rows a CTA) from the second 8-column tile on. Measured, us a call, 8-column
// and tensor tile, 64 contexts of 1000 to 3000 tokens, 32/8 heads: 16-bit pool 8 rows 93, 95; 12 rows 109, 93; 16 rows
// 115, 96; head_dim 64: 8 rows 56, 69; 12 rows 91, 73; E4M3: 8 rows 62, 88; 12 rows 101, 88; 32 rows 195, 92; 4 contexts
// of 9001 to 32768, 40 heads: 8 rows 295, 304; 24 rows 537, 385.
constexpr int kTreeTensorRows = 9, kTreeRowTile = 128;
constexpr int kTreeSms = 152;
// What a call takes in n equal partitions a sequence, us, if every context is of max_context_len: rounds of CTAs, each a
// partition's 64-token tiles and an item's start and end, then the partials' way through memory and the reduce kernel.
// (Measured per tile and item: 16-bit 0.75 and 3, E4M3 0.51 and 6; head_dim 64 about half a tile. A cap, which costs an
// E4M3 tile another 0.15, shorter contexts than the longest and their order are not in it.) One long context of 32768
// tokens, 32/8 heads: 12 to 19 partitions 35 to 37, 10 38, 8 42; 4 contexts of 16384, 40 heads: 4 220, 6 217, 12 229; 64
// contexts to 2048, 32/8 heads: 1 62, 2 90.
float tree_cost(bool fp8, int head_dim, long long items, long long rows, long long span, long long n) {
  const float tile = head_dim == 64 ? 0.4f : fp8 ? 0.51f : 0.75f, item = fp8 ? 6.f : 3.f;
  const long long tiles = (span + n * 64 - 1) / (n * 64), rounds = (items * n + kTreeSms - 1) / kTreeSms;
  const float bytes = n > 1 ? (float)rows * n * (head_dim + 2) * 8 : 0.f;
  return (float)rounds * (tiles * tile + item) + (n > 1 ? 6.f + bytes / 4.5e6f : 0.f);
}

ScoredPlan tree_plan(bool fp8, int num_query_tokens, int num_heads, int num_kv_heads, int head_dim, int block_size,
                     int max_query_len, int max_context_len, int partition_size, size_t workspace_bytes = SIZE_MAX) {
  const long long rows = (long long)max_query_len * (num_heads / num_kv_heads);
  if (rows < kTreeTensorRows)
    return scored_plan(fp8, num_query_tokens, num_heads, num_kv_heads, head_dim, block_size, max_query_len,
                       max_context_len, 0, partition_size, workspace_bytes);
  ScoredPlan pl{};
  pl.tensor = true;
  pl.row_tiles = (int)((rows + kTreeRowTile - 1) / kTreeRowTile);
  const long long span = max_context_len;
  const size_t one = (size_t)num_query_tokens * num_heads * (head_dim + 2) * sizeof(float);
  if (partition_size) {
    pl.P = partition_size;
  } else {
    // (the batch has at least num_query_tokens / max_query_len sequences; partitions of at least 256 tokens)
    const long long seqs = ((long long)num_query_tokens + max_query_len - 1) / max_query_len;
    const long long items = seqs * num_kv_heads * pl.row_tiles;
    long long most = span / 256 < 64 ? span / 256 : 64, n = 1;
    if (one && workspace_bytes / one < (size_t)most) most = (long long)(workspace_bytes / one);
    float best = INFINITY;
    for (long long k = 1; k <= (most > 1 ? most : 1); ++k) {
      const float cost = tree_cost(fp8, head_dim, items, (long long)num_query_tokens * num_heads, span, k);
      if (cost < best) {
        best = cost;
        n = k;
      }
    }
    const long long P = ((span + n - 1) / n + block_size - 1) / block_size * block_size;
    pl.P = P < block_size ? block_size : (int)P;
  }
  const long long np = (span + pl.P - 1) / pl.P;
  pl.np = np < 1 ? 1 : (int)np;
  pl.partials = pl.np > 1 ? one * pl.np : 0;
  return pl;
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
  bool tree = false;  // the query tokens are nodes of a tree; no distance bias, window or key_end then
  const int32_t* tree_mask = nullptr;
  int32_t mask_words = 0;
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
  // (2 log2(e) softcap must not overflow, nor scale / softcap -- over an FP8 pool times a row's power of two -- lose
  // the scores among subnormal numbers: a product of up to 2^15 * 448 * 128 times their step 2^-149 and softcap)
  if (!(c.softcap >= 0.f && c.softcap <= 1e30f))
    return fail(PKV_ERR_INVALID_ARG, "softcap must be in [0, 1e30] (0: no cap)");
  if (c.window < 0) return fail(PKV_ERR_INVALID_ARG, "window must be >= 0 (0: no window)");
  if (c.fp8 && !(isfinite(c.k_scale) && isfinite(c.v_scale) && c.k_scale > 0.f && c.v_scale > 0.f))
    return fail(PKV_ERR_INVALID_ARG, "k_scale and v_scale must be finite and > 0");
  const float scale = c.fp8 ? c.scale * c.k_scale : c.scale;  // of a product of the stored values
  if (!isfinite(scale * 1.4426950408889634f) || (c.softcap > 0.f && !isfinite(scale / c.softcap)))
    return fail(PKV_ERR_INVALID_ARG, "scale (times k_scale) or its quotient by softcap is not finite");
  if (c.fp8 && c.head_dim != 128)
    return fail(PKV_ERR_UNSUPPORTED, "scored attention over an FP8 pool needs head_dim 128 (got %d)", c.head_dim);
  if (c.max_context_len < 0) return fail(PKV_ERR_INVALID_ARG, "max_context_len < 0");
  if ((long long)c.max_context_len > (long long)c.max_blocks_per_seq * c.block_size)
    return fail(PKV_ERR_INVALID_ARG, "max_context_len %d exceeds max_blocks_per_seq * block_size = %lld",
                c.max_context_len, (long long)c.max_blocks_per_seq * c.block_size);
  if (!decode && c.max_query_len > c.max_context_len)
    return fail(PKV_ERR_INVALID_ARG, "max_query_len %d exceeds max_context_len %d", c.max_query_len,
                c.max_context_len);
  if (c.tree && (long long)c.mask_words * 32 < c.max_query_len)
    return fail(PKV_ERR_INVALID_ARG, "mask_words %d: fewer bits than max_query_len %d", c.mask_words, c.max_query_len);
  if (c.partition_size < 0) return fail(PKV_ERR_INVALID_ARG, "partition_size < 0");
  if (c.partition_size && (c.partition_size % c.block_size || c.partition_size > kMaxPartitionBlocks * c.block_size))
    return fail(PKV_ERR_UNSUPPORTED, "partition_size %d must be a multiple of block_size in [%d, %d]",
                c.partition_size, c.block_size, kMaxPartitionBlocks * c.block_size);
  if (c.num_seqs > 65535 || c.num_heads > 65535)
    return fail(PKV_ERR_UNSUPPORTED, "num_seqs and num_heads must be <= 65535");
  if (c.max_query_len > 65535 * kReduceTokens)
    return fail(PKV_ERR_UNSUPPORTED, "max_query_len must be <= %d", 65535 * kReduceTokens);
  if (c.max_context_len > 1 << 30) return fail(PKV_ERR_UNSUPPORTED, "max_context_len must be <= 2^30");
  if ((long long)c.num_blocks * c.num_kv_heads * c.block_size >= (1LL << 31))
    return fail(PKV_ERR_UNSUPPORTED, "pool rows num_blocks * num_kv_heads * block_size must be < 2^31");
  if ((long long)c.num_query_tokens * c.num_heads >= (1LL << 31))
    return fail(PKV_ERR_UNSUPPORTED, "num_query_tokens * num_heads must be < 2^31");
  const size_t room = c.workspace ? c.workspace_bytes : 0;
  const ScoredPlan pl =
      c.tree ? tree_plan(c.fp8, c.num_query_tokens, c.num_heads, c.num_kv_heads, c.head_dim, c.block_size,
                         c.max_query_len, c.max_context_len, c.partition_size, room)
             : scored_plan(c.fp8, c.num_query_tokens, c.num_heads, c.num_kv_heads, c.head_dim, c.block_size,
                           c.max_query_len, c.max_context_len, c.window, c.partition_size, room);
  if ((long long)pl.np * pl.row_tiles >= (1LL << 31))
    return fail(PKV_ERR_UNSUPPORTED, "partitions * row tiles must be < 2^31");
  // A CTA of the tensor tile looks through the grid for rows, some 0.6 us an empty place (measured: 65536 places for 64
  // sequences of one token, 257 us on 152 SMs): the limit keeps a call without work to half a second.
  if (pl.tensor && (long long)pl.np * pl.row_tiles * c.num_kv_heads * c.num_seqs > kScoredMaxItems)
    return fail(PKV_ERR_UNSUPPORTED,
                "num_seqs * num_kv_heads * partitions (%d) * row tiles (%d, of max_query_len) must be <= 2^27", pl.np,
                pl.row_tiles);
  if (c.num_seqs == 0 || c.num_query_tokens == 0 || c.max_query_len == 0) return PKV_OK;
  if (!c.out || !c.query || !c.key_cache || !c.value_cache || !c.block_tables || !c.context_lens ||
      (!decode && !c.query_start_loc) || (c.tree && !c.tree_mask))
    return fail(PKV_ERR_INVALID_ARG, "null pointer argument");
  if (!aligned(c.out, 16) || !aligned(c.query, 16) || !aligned(c.key_cache, 16) || !aligned(c.value_cache, 16))
    return fail(PKV_ERR_INVALID_ARG, "out, query and caches must be 16-byte aligned");
  if (pl.partials) {
    if (!c.workspace) return fail(PKV_ERR_WORKSPACE, "workspace of %zu bytes required", pl.partials);
    if (c.workspace_bytes < pl.partials)
      return fail(PKV_ERR_WORKSPACE, "workspace of %zu bytes < %zu required", c.workspace_bytes, pl.partials);
    if (!aligned(c.workspace, 16)) return fail(PKV_ERR_WORKSPACE, "workspace must be 16-byte aligned");
  }

  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  DecodeParams p{};
  p.err = device_error_word(dev);
  if (!p.err) return fail(PKV_ERR_CUDA, "device error word unavailable on device %d", dev);
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
  p.partition_size = pl.P;
  p.max_partitions = pl.np;
  if (pl.partials) {
    const size_t n = (size_t)c.num_query_tokens * c.num_heads * pl.np;
    p.part_o = static_cast<float*>(c.workspace);
    p.part_m = p.part_o + n * c.head_dim;
    p.part_l = p.part_m + n;
  }
  ScoreParams sc{};
  sc.slopes = c.alibi_slopes;
  sc.key_begin = c.key_begin;
  sc.key_end = c.key_end;
  sc.query_start_loc = decode ? nullptr : c.query_start_loc;
  sc.window = c.window;
  sc.num_query_tokens = c.num_query_tokens;
  sc.max_query_len = c.max_query_len;
  sc.row_tiles = pl.row_tiles;
  sc.tree_mask = reinterpret_cast<const uint32_t*>(c.tree_mask);
  sc.mask_words = c.mask_words;
  // (a batch of which every CTA takes but one item starts all of them at once)
  if (c.tree && pl.tensor && c.num_seqs <= kTreeSortSeqs &&
      (long long)pl.np * pl.row_tiles * c.num_kv_heads * c.num_seqs > kTreeSms)
    sc.sort_seqs = c.num_seqs;
  if (c.softcap > 0.f) {
    sc.cap_in = scale / c.softcap;
    sc.cap_out = c.softcap * 1.4426950408889634f;
  }
  CUtensorMap kmap, vmap;
  memset(&kmap, 0, sizeof kmap);
  memset(&vmap, 0, sizeof vmap);
  const long long pool_rows = (long long)c.num_blocks * c.num_kv_heads * c.block_size;
  const pkv_dtype_t cache_dtype = c.fp8 ? PKV_FP8_E4M3 : c.dtype;
  const bool one_copy = !c.fp8 && c.head_dim == 128 && (pl.tensor || tile_one_copy());
  if (c.fp8 && pl.tensor ? !make_pool_map_fp8_rows(&kmap, c.key_cache, pool_rows, c.block_size) ||
                               !make_pool_map_fp8_rows(&vmap, c.value_cache, pool_rows, c.block_size)
      : one_copy ? !make_pool_map_tc(&kmap, c.key_cache, pool_rows, c.block_size, c.dtype) ||
                     !make_pool_map_tc(&vmap, c.value_cache, pool_rows, c.block_size, c.dtype)
               : !make_pool_map(&kmap, c.key_cache, pool_rows, c.head_dim, c.block_size, cache_dtype) ||
                     !make_pool_map(&vmap, c.value_cache, pool_rows, c.head_dim, c.block_size, cache_dtype))
    return fail(PKV_ERR_CUDA, "cuTensorMapEncodeTiled failed for the KV pool");
  const bool f16 = c.dtype == PKV_F16;
  if (c.tree)
    e = !pl.tensor ? tree_cols(p, sc, kmap, vmap, f16, c.fp8, c.head_dim, c.block_size, c.num_seqs, c.stream)
        : f16      ? tree_tc_f16(p, sc, kmap, vmap, c.fp8, c.head_dim, c.block_size, c.num_seqs, c.stream)
                   : tree_tc_bf16(p, sc, kmap, vmap, c.fp8, c.head_dim, c.block_size, c.num_seqs, c.stream);
  else if (pl.tensor)
    e = c.fp8 ? scored_tc_fp8(p, sc, kmap, vmap, f16, c.block_size, c.num_seqs, c.stream)
        : f16 ? scored_tc_f16(p, sc, kmap, vmap, c.head_dim, c.block_size, c.num_seqs, c.stream)
              : scored_tc_bf16(p, sc, kmap, vmap, c.head_dim, c.block_size, c.num_seqs, c.stream);
  else
    e = c.fp8 ? scored_cols_fp8(p, sc, kmap, vmap, f16, c.block_size, c.num_seqs, c.stream)
              : scored_cols_16(p, sc, kmap, vmap, f16, c.head_dim, c.block_size, c.num_seqs, c.stream);
  if (e != cudaSuccess) return cuda_fail(e, "scored attention launch");
  if (pl.np > 1) {
    const unsigned head_groups = (unsigned)((c.num_heads + kReduceRows - 1) / kReduceRows);
    // (trees: up to kTreeReduceCtas CTAs before a CTA takes several query tokens)
    const long long ctas = (long long)c.num_seqs * head_groups * c.max_query_len;
    const int per_cta = c.tree ? (int)(ctas > 8ll * kTreeReduceCtas ? 8 : (ctas + kTreeReduceCtas - 1) / kTreeReduceCtas)
                               : kReduceTokens;
    const dim3 grid((unsigned)c.num_seqs, head_groups, (unsigned)((c.max_query_len + per_cta - 1) / per_cta));
    auto scored = [&](auto kern) {
      return launch_kernel(kern, grid, dim3(32 * kReduceRows), 0, c.stream, p, sc, (int)c.block_size);
    };
    auto tree = [&](auto kern) {
      return launch_kernel(kern, grid, dim3(32 * kReduceRows), 0, c.stream, p, sc, per_cta);
    };
    if (c.tree && c.head_dim == 128)
      e = f16 ? tree(pkv_tree_reduce_kernel<__half, 128>) : tree(pkv_tree_reduce_kernel<__nv_bfloat16, 128>);
    else if (c.tree)
      e = f16 ? tree(pkv_tree_reduce_kernel<__half, 64>) : tree(pkv_tree_reduce_kernel<__nv_bfloat16, 64>);
    else if (c.head_dim == 128)
      e = f16 ? scored(pkv_scored_reduce_kernel<__half, 128>) : scored(pkv_scored_reduce_kernel<__nv_bfloat16, 128>);
    else
      e = f16 ? scored(pkv_scored_reduce_kernel<__half, 64>) : scored(pkv_scored_reduce_kernel<__nv_bfloat16, 64>);
    if (e != cudaSuccess) return cuda_fail(e, "scored reduce launch");
  }
  return PKV_OK;
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" {

size_t paged_attention_scored_workspace_size(int32_t num_query_tokens, int32_t num_heads, int32_t num_kv_heads,
                                             int32_t head_dim, int32_t block_size, int32_t max_query_len,
                                             int32_t max_context_len, int32_t window, int32_t partition_size) {
  if (num_query_tokens <= 0 || num_heads <= 0 || num_kv_heads <= 0 || num_heads % num_kv_heads || head_dim <= 0 ||
      block_size <= 0 || max_query_len <= 0 || max_context_len < 0 || window < 0 || partition_size < 0)
    return 0;
  size_t bytes = 0;  // for either type of pool
  for (bool fp8 : {false, true}) {
    const size_t n = scored_plan(fp8, num_query_tokens, num_heads, num_kv_heads, head_dim, block_size, max_query_len,
                                 max_context_len, window, partition_size)
                         .partials;
    if (n > bytes) bytes = n;
  }
  return bytes;
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

size_t paged_attention_tree_workspace_size(int32_t num_query_tokens, int32_t num_heads, int32_t num_kv_heads,
                                           int32_t head_dim, int32_t block_size, int32_t max_query_len,
                                           int32_t max_context_len, int32_t partition_size) {
  if (num_query_tokens <= 0 || num_heads <= 0 || num_kv_heads <= 0 || num_heads % num_kv_heads || head_dim <= 0 ||
      block_size <= 0 || max_query_len <= 0 || max_context_len < 0 || partition_size < 0)
    return 0;
  size_t bytes = 0;  // for either type of pool
  for (bool fp8 : {false, true}) {
    const size_t n = tree_plan(fp8, num_query_tokens, num_heads, num_kv_heads, head_dim, block_size, max_query_len,
                               max_context_len, partition_size)
                         .partials;
    if (n > bytes) bytes = n;
  }
  return bytes;
}

pkv_status_t paged_attention_tree(void* out, const void* query, const void* key_cache, const void* value_cache,
                                  const int32_t* block_tables, int32_t max_blocks_per_seq,
                                  const int32_t* context_lens, const int32_t* query_start_loc, int32_t num_seqs,
                                  int32_t num_query_tokens, int32_t max_query_len, int32_t max_context_len,
                                  const int32_t* tree_mask, int32_t mask_words, float scale, float softcap,
                                  const int32_t* key_begin, int32_t block_size, int32_t num_heads,
                                  int32_t num_kv_heads, int32_t head_dim, int32_t num_blocks, pkv_dtype_t dtype,
                                  int32_t partition_size, void* workspace, size_t workspace_bytes,
                                  cudaStream_t stream) {
  return scored_impl({out, query, key_cache, value_cache, block_tables, max_blocks_per_seq, context_lens,
                      query_start_loc, num_seqs, num_query_tokens, max_query_len, max_context_len, scale, softcap,
                      nullptr, 0, key_begin, nullptr, block_size, num_heads, num_kv_heads, head_dim, num_blocks, dtype,
                      false, 1.f, 1.f, partition_size, workspace, workspace_bytes, stream, true, tree_mask, mask_words},
                     false);
}

pkv_status_t paged_attention_tree_fp8(void* out, const void* query, const void* key_cache, const void* value_cache,
                                      const int32_t* block_tables, int32_t max_blocks_per_seq,
                                      const int32_t* context_lens, const int32_t* query_start_loc, int32_t num_seqs,
                                      int32_t num_query_tokens, int32_t max_query_len, int32_t max_context_len,
                                      const int32_t* tree_mask, int32_t mask_words, float scale, float softcap,
                                      const int32_t* key_begin, int32_t block_size, int32_t num_heads,
                                      int32_t num_kv_heads, int32_t head_dim, int32_t num_blocks, pkv_dtype_t dtype,
                                      float k_scale, float v_scale, int32_t partition_size, void* workspace,
                                      size_t workspace_bytes, cudaStream_t stream) {
  return scored_impl({out, query, key_cache, value_cache, block_tables, max_blocks_per_seq, context_lens,
                      query_start_loc, num_seqs, num_query_tokens, max_query_len, max_context_len, scale, softcap,
                      nullptr, 0, key_begin, nullptr, block_size, num_heads, num_kv_heads, head_dim, num_blocks, dtype,
                      true, k_scale, v_scale, partition_size, workspace, workspace_bytes, stream, true, tree_mask,
                      mask_words},
                     false);
}

}  // extern "C"
