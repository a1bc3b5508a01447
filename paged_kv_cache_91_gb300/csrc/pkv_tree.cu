// The passes around the attention of a drafted tree: paged_kv_tree_layout (masks and positions from the parents) and
// paged_kv_compact_accepted (the accepted rows of every layer move up behind the committed ones). One launch each;
// bound by latency, and the moves of many layers by HBM.
#include <stdint.h>

#include "paged_kv.h"
#include "pkv_common.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

bool overlap(const void* a, size_t n, const void* b, size_t m) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return n && m && x < y + m && y < x + n;
}
bool aligned(const void* ptr, uintptr_t n) { return (reinterpret_cast<uintptr_t>(ptr) & (n - 1)) == 0; }

// Sequence s's q_len and first row q0; -1 for bad offsets, or more query tokens than context.
__device__ __forceinline__ int tree_len(const int32_t* query_start_loc, int s, int ctx, int num_query_tokens,
                                        int max_query_len, int& q0) {
  q0 = query_start_loc[s];
  const int q1 = query_start_loc[s + 1];
  // (compared without a difference that could overflow)
  if (q0 < 0 || q1 < q0 || q1 > num_query_tokens || q1 - q0 > max_query_len || q1 - q0 > ctx) return -1;
  return q1 - q0;
}

struct LayoutParams {
  const int32_t *parents, *query_start_loc, *context_lens;
  uint32_t* tree_mask;
  int32_t* positions;
  unsigned* err;
  int num_query_tokens, max_query_len, mask_words;
};

constexpr int kLayoutWarps = 8;
constexpr int kLayoutNodes = 32;  // per CTA
constexpr int kMaxTree = 1024;

// A CTA takes kLayoutNodes nodes of a tree, a warp one at a time: it walks up to the root through the parents in
// shared memory, and lane w keeps the mask's word w. Latency: 8 trees of up to 16 nodes 1.8 us replayed from a graph; 512
// of up to 64 6.4 us and a chain of 64 nodes 7.3, since a warp takes four nodes one after the other and every ancestor is a
// load that waits for the one before (a chain of 1024 nodes 108 us, 64 of them 500).
__global__ void __launch_bounds__(kLayoutWarps * 32) pkv_tree_layout_kernel(const LayoutParams p) {
  pdl_begin();
  __shared__ int16_t up[kMaxTree];
  const int s = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ctx = p.context_lens[s];
  int q0;
  const int n = tree_len(p.query_start_loc, s, ctx, p.num_query_tokens, p.max_query_len, q0);
  if (n < 0) {
    if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(p.err, PKV_DEVERR_QUERY);
    return;
  }
  const int first = blockIdx.x * kLayoutNodes, last = min(n, first + kLayoutNodes);
  if (first >= n) return;
  for (int i = threadIdx.x; i < last; i += kLayoutWarps * 32) {  // (ancestors come before)
    int parent = p.parents[q0 + i];
    if (parent >= i) {
      if (i >= first) atomicOr(p.err, PKV_DEVERR_QUERY);
      parent = -1;
    }
    up[i] = (int16_t)max(parent, -1);
  }
  __syncthreads();
  for (int i = first + warp; i < last; i += kLayoutWarps) {
    uint32_t word = 0;
    int depth = -1;
    for (int a = i; a >= 0; a = up[a]) {
      if ((a >> 5) == lane) word |= 1u << (a & 31);
      ++depth;
    }
    uint32_t* row = p.tree_mask + (size_t)(q0 + i) * p.mask_words;
    for (int w = lane; w < p.mask_words; w += 32) row[w] = w < 32 ? word : 0u;
    if (lane == 0) p.positions[q0 + i] = ctx - n + depth;
  }
}

struct CompactParams {
  unsigned char *key_cache, *value_cache;
  const int32_t *block_tables, *context_lens, *query_start_loc, *accepted, *num_accepted;
  unsigned* err;
  long long layer_bytes;
  int max_blocks_per_seq, max_accepted;
  int pairs;  // layers * kv heads
  int num_kv_heads, block_size, num_blocks;
};

constexpr int kCompactWarps = 8;
constexpr int kCompactPairs = 4;   // (layer, kv head) pairs a warp
constexpr int kCompactChunk = 64;  // accepted tokens at a time
constexpr int kCompactUnroll = 2;  // rows of each pair that a lane has in flight

// A CTA takes a sequence and kCompactWarps * kCompactPairs (layer, kv head) pairs of it. It works out where each
// accepted row lies and goes to once, for all of them; then each warp moves its pairs' rows, ROW / 16 lanes a row, half
// of the warp's K and half V. The path increases, so a row's source is never before its destination: rows taken in
// order, read before the ones behind them are written, are safe in place.
//
// Bound by latency: what does not depend on one another loads together (the path with the lengths that say how much of
// it counts), and a warp's pairs are in flight at once. 128 sequences, 32 layers of 8 heads, E4M3, some 7 rows each:
// 11.0 us a call replayed from a graph (8.6 at the copy rate).
template <int ROW>
__global__ void __launch_bounds__(kCompactWarps * 32) pkv_compact_kernel(const CompactParams p) {
  pdl_begin();
  __shared__ int s_src[kCompactChunk], s_dst[kCompactChunk];  // pool rows of head 0; src -1: not moved
  const int s = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x;
  const int B = p.block_size;
  const int32_t* path = p.accepted + (size_t)s * p.max_accepted;
  const int n = p.num_accepted[s], ctx = p.context_lens[s];
  const int q0 = p.query_start_loc[s], q1 = p.query_start_loc[s + 1];
  int u0 = tid < p.max_accepted ? path[tid] : 0;  // (its first entries, in bounds however long it is)
  int before = tid > 0 && tid < p.max_accepted ? path[tid - 1] : -1;
  if (n == 0) return;
  const bool too_long = (long long)ctx > (long long)p.max_blocks_per_seq * B;
  // (compared without a difference that could overflow)
  const bool fine = q0 >= 0 && q1 >= q0 && q1 - q0 <= ctx && n > 0 && n <= p.max_accepted && n <= q1 - q0 && !too_long;
  const int q_len = q1 - q0;
  bool good = true;
  if (fine)
    for (int i = tid; i < n; i += kCompactWarps * 32) {
      const int u = i == tid ? u0 : path[i], prev = i == tid ? before : path[i - 1];
      good = good && u > prev && u < q_len;
    }
  if (!fine || !__syncthreads_and(good)) {
    if (blockIdx.x == 0 && tid == 0) atomicOr(p.err, too_long ? PKV_DEVERR_CONTEXT : PKV_DEVERR_QUERY);
    return;
  }
  const int c0 = ctx - q_len;
  const int32_t* table = p.block_tables + (size_t)s * p.max_blocks_per_seq;
  constexpr int LPR = ROW / 16, RPS = 16 / LPR;  // lanes a row; rows of K, and of V, at a time
  unsigned char* cache = lane < 16 ? p.key_cache : p.value_cache;
  const int r0 = (lane & 15) / LPR, c = lane % LPR;
  unsigned char* pool[kCompactPairs];  // this lane's piece of row 0 of each pair's head; null: no such pair
#pragma unroll
  for (int k = 0; k < kCompactPairs; ++k) {
    const int pair = (blockIdx.x * kCompactPairs + k) * kCompactWarps + warp;
    const int layer = pair / p.num_kv_heads, h = pair - layer * p.num_kv_heads;
    pool[k] = pair < p.pairs ? cache + layer * p.layer_bytes + (size_t)h * B * ROW + c * 16 : nullptr;
  }
  for (int i0 = 0; i0 < n; i0 += kCompactChunk) {
    const int m = min(kCompactChunk, n - i0);
    if (tid < m) {
      const int i = i0 + tid, from = c0 + (i0 ? path[i] : u0), to = c0 + i;
      int src = -1, dst = 0;
      if (from != to) {
        const int a = table[from / B], b = table[to / B];
        if ((unsigned)a < (unsigned)p.num_blocks && (unsigned)b < (unsigned)p.num_blocks) {
          src = a * p.num_kv_heads * B + from % B;  // (the pool's rows number less than 2^31)
          dst = b * p.num_kv_heads * B + to % B;
        } else if (blockIdx.x == 0) {
          atomicOr(p.err, PKV_DEVERR_BLOCK_ID);
        }
      }
      s_src[tid] = src;
      s_dst[tid] = dst;
    }
    __syncthreads();
    for (int i = 0; i < m; i += RPS * kCompactUnroll) {
      int src[kCompactUnroll], dst[kCompactUnroll];
      uint4 x[kCompactPairs][kCompactUnroll];
#pragma unroll
      for (int u = 0; u < kCompactUnroll; ++u) {
        const int r = i + u * RPS + r0;
        src[u] = r < m ? s_src[r] : -1;
        dst[u] = r < m ? s_dst[r] : 0;
      }
#pragma unroll
      for (int k = 0; k < kCompactPairs; ++k)
#pragma unroll
        for (int u = 0; u < kCompactUnroll; ++u)
          if (pool[k] && src[u] >= 0) x[k][u] = *reinterpret_cast<const uint4*>(pool[k] + (size_t)src[u] * ROW);
      __syncwarp();  // what is read here is read before other lanes write
#pragma unroll
      for (int k = 0; k < kCompactPairs; ++k)
#pragma unroll
        for (int u = 0; u < kCompactUnroll; ++u)
          if (pool[k] && src[u] >= 0) *reinterpret_cast<uint4*>(pool[k] + (size_t)dst[u] * ROW) = x[k][u];
      __syncwarp();  // (a row that is written here is not read again: sources lie behind)
    }
    __syncthreads();  // the places may be written again
  }
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" {

pkv_status_t paged_kv_tree_layout(const int32_t* parents, const int32_t* query_start_loc, const int32_t* context_lens,
                                  int32_t num_seqs, int32_t num_query_tokens, int32_t max_query_len,
                                  int32_t* tree_mask, int32_t mask_words, int32_t* positions, cudaStream_t stream) {
  set_last_error_message("");
  if (num_seqs < 0 || num_query_tokens < 0 || max_query_len < 0 || mask_words < 0)
    return fail(PKV_ERR_INVALID_ARG, "num_seqs, num_query_tokens, max_query_len and mask_words must be >= 0");
  if ((long long)mask_words * 32 < max_query_len)
    return fail(PKV_ERR_INVALID_ARG, "mask_words %d: fewer bits than max_query_len %d", mask_words, max_query_len);
  if (max_query_len > kMaxTree) return fail(PKV_ERR_UNSUPPORTED, "max_query_len must be <= %d", kMaxTree);
  if (num_seqs > 65535) return fail(PKV_ERR_UNSUPPORTED, "num_seqs must be <= 65535");
  if (num_seqs == 0 || num_query_tokens == 0 || max_query_len == 0) return PKV_OK;
  if (!parents || !query_start_loc || !context_lens || !tree_mask || !positions)
    return fail(PKV_ERR_INVALID_ARG, "null pointer argument");
  const size_t rows = (size_t)num_query_tokens * 4, seqs = (size_t)num_seqs * 4, mask = rows * (size_t)mask_words;
  const void* read[] = {parents, query_start_loc, context_lens};
  const size_t read_bytes[] = {rows, seqs + 4, seqs};
  for (int i = 0; i < 3; ++i)
    if (overlap(tree_mask, mask, read[i], read_bytes[i]) || overlap(positions, rows, read[i], read_bytes[i]))
      return fail(PKV_ERR_INVALID_ARG, "tree_mask and positions must not overlap the inputs");
  if (overlap(tree_mask, mask, positions, rows))
    return fail(PKV_ERR_INVALID_ARG, "tree_mask must not overlap positions");
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  LayoutParams p{};
  p.parents = parents;
  p.query_start_loc = query_start_loc;
  p.context_lens = context_lens;
  p.tree_mask = reinterpret_cast<uint32_t*>(tree_mask);
  p.positions = positions;
  p.err = device_error_word(dev);
  if (!p.err) return fail(PKV_ERR_CUDA, "device error word unavailable on device %d", dev);
  p.num_query_tokens = num_query_tokens;
  p.max_query_len = max_query_len;
  p.mask_words = mask_words;
  const dim3 grid((unsigned)((max_query_len + kLayoutNodes - 1) / kLayoutNodes), (unsigned)num_seqs);
  e = launch_kernel(pkv_tree_layout_kernel, grid, dim3(kLayoutWarps * 32), 0, stream, p);
  if (e != cudaSuccess) return cuda_fail(e, "paged_kv_tree_layout launch");
  return PKV_OK;
}

pkv_status_t paged_kv_compact_accepted(void* key_cache, void* value_cache, int32_t num_layers,
                                       const int32_t* block_tables, int32_t max_blocks_per_seq,
                                       const int32_t* context_lens, const int32_t* query_start_loc, int32_t num_seqs,
                                       const int32_t* accepted, int32_t max_accepted, const int32_t* num_accepted,
                                       int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                                       int32_t num_blocks, pkv_dtype_t dtype, cudaStream_t stream) {
  set_last_error_message("");
  if (num_seqs < 0 || max_accepted < 0 || num_layers < 0)
    return fail(PKV_ERR_INVALID_ARG, "num_layers, num_seqs and max_accepted must be >= 0");
  if (dtype != PKV_F16 && dtype != PKV_BF16 && dtype != PKV_FP8_E4M3)
    return fail(PKV_ERR_INVALID_ARG, "unknown dtype %d", (int)dtype);
  if (num_kv_heads <= 0 || num_blocks <= 0 || max_blocks_per_seq <= 0)
    return fail(PKV_ERR_INVALID_ARG, "num_kv_heads, num_blocks and max_blocks_per_seq must be > 0");
  if (head_dim != 64 && head_dim != 128)
    return fail(PKV_ERR_UNSUPPORTED, "head_dim %d (supported: 64, 128)", head_dim);
  if (block_size != 8 && block_size != 16 && block_size != 32)
    return fail(PKV_ERR_UNSUPPORTED, "block_size %d (supported: 8, 16, 32)", block_size);
  if (num_seqs > 65535) return fail(PKV_ERR_UNSUPPORTED, "num_seqs must be <= 65535");
  if ((long long)num_blocks * num_kv_heads * block_size >= (1LL << 31))
    return fail(PKV_ERR_UNSUPPORTED, "pool rows num_blocks * num_kv_heads * block_size must be < 2^31");
  const long long pairs = (long long)num_layers * num_kv_heads;
  if (pairs >= (1LL << 30)) return fail(PKV_ERR_UNSUPPORTED, "num_layers * num_kv_heads must be < 2^30");
  if (num_seqs == 0 || max_accepted == 0 || num_layers == 0) return PKV_OK;
  if (!key_cache || !value_cache || !block_tables || !context_lens || !query_start_loc || !accepted || !num_accepted)
    return fail(PKV_ERR_INVALID_ARG, "null pointer argument");
  if (!aligned(key_cache, 16) || !aligned(value_cache, 16))
    return fail(PKV_ERR_INVALID_ARG, "caches must be 16-byte aligned");
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  const int row = head_dim * (dtype == PKV_FP8_E4M3 ? 1 : 2);
  CompactParams p{};
  p.key_cache = static_cast<unsigned char*>(key_cache);
  p.value_cache = static_cast<unsigned char*>(value_cache);
  p.block_tables = block_tables;
  p.context_lens = context_lens;
  p.query_start_loc = query_start_loc;
  p.accepted = accepted;
  p.num_accepted = num_accepted;
  p.err = device_error_word(dev);
  if (!p.err) return fail(PKV_ERR_CUDA, "device error word unavailable on device %d", dev);
  p.layer_bytes = (long long)num_blocks * num_kv_heads * block_size * row;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.max_accepted = max_accepted;
  p.pairs = (int)pairs;
  p.num_kv_heads = num_kv_heads;
  p.block_size = block_size;
  p.num_blocks = num_blocks;
  constexpr int per_cta = kCompactWarps * kCompactPairs;
  const dim3 grid((unsigned)((pairs + per_cta - 1) / per_cta), (unsigned)num_seqs);
  auto run = [&](auto kern) { return launch_kernel(kern, grid, dim3(kCompactWarps * 32), 0, stream, p); };
  e = row == 256 ? run(pkv_compact_kernel<256>) : row == 128 ? run(pkv_compact_kernel<128>) : run(pkv_compact_kernel<64>);
  if (e != cudaSuccess) return cuda_fail(e, "paged_kv_compact_accepted launch");
  return PKV_OK;
}

}  // extern "C"
