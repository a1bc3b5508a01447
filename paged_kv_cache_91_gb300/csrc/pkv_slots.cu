// Block tables and slot maps on the GPU: paged_kv_reserve_slots gives the next step's tokens their slots and
// takes the new blocks from a free stack, paged_kv_release_blocks puts finished sequences' blocks back. Both
// are one launch each, so that a step (reserve, cache write, attention, release) needs no host round trip and
// can be captured in a graph.
//
// Both are prefix sums over the sequences followed by independent writes. A CTA does not wait for another
// one: each computes the sums that its own part needs from the request lengths, which stay in L2 (8 bytes per
// sequence), instead of a second launch or a look-back. Bound by launch and memory latency.
#include <stdint.h>

#include "paged_kv.h"
#include "pkv_common.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr int kSlotThreads = 512;
constexpr int kSlotItems = 4;                             // sequences per thread and round
constexpr int kSlotChunk = kSlotThreads * kSlotItems;     // sequences per round
constexpr int kSlotTokens = 1024;                         // tokens per CTA

struct TwoSums {
  long long a, b;
};

// Exclusive sums of v over the CTA's threads, and the total. `ws`: one entry per warp.
__device__ __forceinline__ TwoSums block_exclusive(TwoSums v, TwoSums* ws, TwoSums& total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  TwoSums x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long a = __shfl_up_sync(kFull, x.a, o), b = __shfl_up_sync(kFull, x.b, o);
    if (lane >= o) {
      x.a += a;
      x.b += b;
    }
  }
  if (lane == 31) ws[warp] = x;
  __syncthreads();
  TwoSums before = {0, 0};
  total = {0, 0};
#pragma unroll
  for (int w = 0; w < kSlotThreads / 32; ++w) {
    if (w == warp) before = total;
    total.a += ws[w].a;
    total.b += ws[w].b;
  }
  __syncthreads();  // ws may be written again
  return {before.a + x.a - v.a, before.b + x.b - v.b};
}

struct ReserveParams {
  int32_t* block_tables;
  const int32_t* context_lens;
  const int32_t* new_lens;
  const int32_t* free_blocks;
  const int32_t* num_free;
  int64_t* slot_mapping;
  int32_t* query_start_loc;
  int32_t* context_lens_out;
  int32_t* num_free_out;
  int32_t* granted;
  unsigned* err;
  int num_seqs, max_tokens, max_blocks_per_seq, free_capacity, block_size, num_blocks;
};

// CTA c gives the tokens [c * kSlotTokens, (c + 1) * kSlotTokens) their slots and writes the per-sequence
// outputs of the sequences that start there (the last CTA: of all later ones too, and the totals). It walks
// the sequences in rounds of kSlotChunk, up to its last token.
__global__ void __launch_bounds__(kSlotThreads) pkv_reserve_slots_kernel(const ReserveParams p) {
  pdl_begin();
  __shared__ TwoSums ws[kSlotThreads / 32];
  __shared__ int32_t s_start[kSlotChunk];  // first token of each sequence of the round
  __shared__ int32_t s_ctx[kSlotChunk];    // its context before the step
  __shared__ int32_t s_take[kSlotChunk];   // new blocks taken before it; -1: no slots (refused)
  __shared__ int s_max[kSlotThreads / 32];
  const int tid = threadIdx.x;
  const bool last = blockIdx.x == gridDim.x - 1;
  const long long t0 = (long long)blockIdx.x * kSlotTokens;
  const long long t1 = last ? (long long)p.max_tokens : t0 + kSlotTokens;
  const int B = p.block_size;
  const long long limit = (long long)p.max_blocks_per_seq * B;
  int nfree = p.num_free[0];
  if (nfree < 0 || nfree > p.free_capacity) {
    if (last && tid == 0) atomicOr(p.err, PKV_DEVERR_BLOCK_ID);
    nfree = nfree < 0 ? 0 : p.free_capacity;
  }
  long long tok = 0, taken = 0;  // tokens and new blocks of the rounds before
  int used = 0;                  // new blocks of the granted sequences seen by this thread
  for (int s0 = 0; s0 < p.num_seqs; s0 += kSlotChunk) {
    int ctx[kSlotItems], add[kSlotItems], need[kSlotItems];
    bool bad[kSlotItems];
    TwoSums mine = {0, 0};
#pragma unroll
    for (int k = 0; k < kSlotItems; ++k) {
      const int s = s0 + tid * kSlotItems + k;
      ctx[k] = s < p.num_seqs ? p.context_lens[s] : 0;
      add[k] = s < p.num_seqs ? p.new_lens[s] : 0;
    }
#pragma unroll
    for (int k = 0; k < kSlotItems; ++k) {
      bad[k] = ctx[k] < 0 || add[k] < 0 || (long long)ctx[k] + add[k] > limit;
      if (add[k] < 0) add[k] = 0;
      // (within the limit, ctx + add + B - 1 fits 32 bits: the host bounds max_blocks_per_seq * block_size)
      need[k] = bad[k] ? 0 : (ctx[k] + add[k] + B - 1) / B - (ctx[k] + B - 1) / B;
      mine.a += add[k];
      mine.b += need[k];
    }
    TwoSums total;
    TwoSums at = block_exclusive(mine, ws, total);
    at.a += tok;
    at.b += taken;
#pragma unroll
    for (int k = 0; k < kSlotItems; ++k) {
      const int i = tid * kSlotItems + k, s = s0 + i;
      const bool over = add[k] > 0 && at.a + add[k] > p.max_tokens;  // (no tokens: none past max_tokens)
      const bool ok = !bad[k] && !over && (need[k] == 0 || at.b + need[k] <= nfree);
      s_start[i] = (int)min(at.a, (long long)p.max_tokens);
      s_ctx[i] = ctx[k];
      s_take[i] = ok ? (need[k] ? (int)at.b : 0) : -1;  // (past nfree only where no block is needed)
      if (s < p.num_seqs && at.a >= t0 && (at.a < t1 || last)) {
        p.query_start_loc[s] = s_start[i];
        p.context_lens_out[s] = ok ? ctx[k] + add[k] : ctx[k];
        p.granted[s] = ok ? 1 : 0;
        if (bad[k]) atomicOr(p.err, PKV_DEVERR_CONTEXT);
        if (over) atomicOr(p.err, PKV_DEVERR_QUERY);
      }
      // the blocks are handed out in order, so the last granted sequence's sum is the number taken
      if (ok && need[k] > 0) used = (int)(at.b + need[k]);
      at.a += add[k];
      at.b += need[k];
    }
    __syncthreads();
    // this round's tokens of the CTA
    const int n = min(kSlotChunk, p.num_seqs - s0);
    const long long r0 = max(t0, tok), r1 = min(t1, tok + total.a);
    for (long long t = r0 + tid; t < r1; t += kSlotThreads) {
      int lo = 0, hi = n;  // the last sequence that starts at or before t (it has tokens: the next starts after t)
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_start[mid] <= t) lo = mid; else hi = mid;
      }
      long long slot = -1;
      if (s_take[lo] >= 0) {
        const int pos = s_ctx[lo] + (int)(t - s_start[lo]);
        const int col = pos / B, off = pos - col * B;
        const int have = (s_ctx[lo] + B - 1) / B;
        int32_t* entry = p.block_tables + (size_t)(s0 + lo) * p.max_blocks_per_seq + col;
        int phys;
        if (col >= have) {
          phys = p.free_blocks[nfree - 1 - (s_take[lo] + col - have)];
          if ((unsigned)phys >= (unsigned)p.num_blocks) phys = -1;
          if (off == 0) *entry = phys;
        } else {
          phys = *entry;
        }
        if ((unsigned)phys < (unsigned)p.num_blocks)
          slot = (long long)phys * B + off;
        else
          atomicOr(p.err, PKV_DEVERR_BLOCK_ID);
      }
      p.slot_mapping[t] = slot;
    }
    tok += total.a;
    taken += total.b;
    if (tok >= t1 && !last) break;
    __syncthreads();  // the round's arrays may be written again
  }
  for (long long t = max(t0, tok) + tid; t < t1; t += kSlotThreads) p.slot_mapping[t] = -1;  // padding
  if (last) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) used = max(used, __shfl_xor_sync(kFull, used, o));
    if ((tid & 31) == 0) s_max[tid >> 5] = used;
    __syncthreads();
    if (tid == 0) {
      for (int w = 1; w < kSlotThreads / 32; ++w) used = max(used, s_max[w]);
      p.num_free_out[0] = nfree - used;
      p.query_start_loc[p.num_seqs] = (int)min(tok, (long long)p.max_tokens);
    }
  }
}

struct ReleaseParams {
  const int32_t* block_tables;
  const int32_t* context_lens;
  const int32_t* finished;
  int32_t* free_blocks;
  const int32_t* num_free;
  int32_t* context_lens_out;
  int32_t* num_free_out;
  unsigned* err;
  int num_seqs, per_cta, max_blocks_per_seq, free_capacity, block_size, num_blocks;
};

constexpr int kReleaseSeqs = kSlotThreads;  // most sequences per CTA

// CTA c pushes the blocks of the finished ones among sequences [c * per_cta, (c + 1) * per_cta), in order; it
// sums the block counts of the sequences before its own itself.
__global__ void __launch_bounds__(kSlotThreads) pkv_release_blocks_kernel(const ReleaseParams p) {
  pdl_begin();
  __shared__ TwoSums ws[kSlotThreads / 32];
  __shared__ int32_t s_at[kReleaseSeqs + 1];  // where each of the CTA's sequences starts among the CTA's blocks (< 2^31)
  const int tid = threadIdx.x;
  const int s0 = blockIdx.x * p.per_cta, n = min(p.per_cta, p.num_seqs - s0);
  const long long limit = (long long)p.max_blocks_per_seq * p.block_size;
  auto blocks = [&](int s) -> int {
    if (!p.finished[s]) return 0;
    long long c = p.context_lens[s];
    c = c < 0 ? 0 : (c > limit ? limit : c);
    return (int)((c + p.block_size - 1) / p.block_size);
  };
  int nfree = p.num_free[0];
  if (nfree < 0 || nfree > p.free_capacity) {
    if (blockIdx.x == 0 && tid == 0) atomicOr(p.err, PKV_DEVERR_BLOCK_ID);
    nfree = nfree < 0 ? 0 : p.free_capacity;
  }
  // a: blocks before the CTA's sequences, b: blocks of its own, one sequence per thread
  TwoSums v = {0, 0}, total;
  for (int s = tid; s < s0; s += kSlotThreads) v.a += blocks(s);
  if (tid < n) {
    const int c = p.context_lens[s0 + tid];
    const bool gone = p.finished[s0 + tid] != 0;
    if (gone && (c < 0 || c > limit)) atomicOr(p.err, PKV_DEVERR_CONTEXT);
    p.context_lens_out[s0 + tid] = gone ? 0 : c;
    v.b = blocks(s0 + tid);
  }
  const TwoSums at = block_exclusive(v, ws, total);
  if (tid < n) s_at[tid] = (int)at.b;
  if (tid == 0) s_at[n] = (int)total.b;
  __syncthreads();
  for (int e = tid; e < (int)total.b; e += kSlotThreads) {
    int lo = 0, hi = n;  // the last sequence that starts at or before e
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s_at[mid] <= e) lo = mid; else hi = mid;
    }
    int id = p.block_tables[(size_t)(s0 + lo) * p.max_blocks_per_seq + (e - s_at[lo])];
    const long long to = nfree + total.a + e;
    if ((unsigned)id >= (unsigned)p.num_blocks) {
      atomicOr(p.err, PKV_DEVERR_BLOCK_ID);
      id = -1;
    }
    if (to < p.free_capacity)
      p.free_blocks[to] = id;
    else
      atomicOr(p.err, PKV_DEVERR_BLOCK_ID);
  }
  if (blockIdx.x == gridDim.x - 1 && tid == 0)
    p.num_free_out[0] = (int)min(nfree + total.a + total.b, (long long)p.free_capacity);
}

// A device array of a call. (A null or empty one overlaps nothing.)
struct Span {
  const char* name;
  const void* at;
  size_t bytes;
};
bool overlap(const Span& a, const Span& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.at), y = reinterpret_cast<uintptr_t>(b.at);
  return a.bytes && b.bytes && x < y + b.bytes && y < x + a.bytes;
}
// Every CTA reads the inputs for itself while others write: an array that is written shares no byte with another one
// of the call, read or written.
template <int NW, int NR>
pkv_status_t check_apart(const Span (&written)[NW], const Span (&read)[NR]) {
  for (int i = 0; i < NW; ++i) {
    for (int j = 0; j < i; ++j)
      if (overlap(written[i], written[j]))
        return fail(PKV_ERR_INVALID_ARG, "%s must not overlap %s", written[i].name, written[j].name);
    for (const Span& in : read)
      if (overlap(written[i], in)) return fail(PKV_ERR_INVALID_ARG, "%s must not overlap %s", written[i].name, in.name);
  }
  return PKV_OK;
}

// The checks that both calls share. (An empty batch launches too: its totals are outputs.)
pkv_status_t check_common(int32_t num_seqs, int32_t max_blocks_per_seq, int32_t free_capacity, int32_t block_size,
                          int32_t num_blocks) {
  if (num_seqs < 0) return fail(PKV_ERR_INVALID_ARG, "num_seqs < 0");
  if (num_blocks <= 0 || max_blocks_per_seq <= 0)
    return fail(PKV_ERR_INVALID_ARG, "num_blocks and max_blocks_per_seq must be > 0");
  if (free_capacity < 0) return fail(PKV_ERR_INVALID_ARG, "free_capacity < 0");
  if (block_size != 8 && block_size != 16 && block_size != 32)
    return fail(PKV_ERR_UNSUPPORTED, "block_size %d (supported: 8, 16, 32)", block_size);
  if (num_seqs > 65535) return fail(PKV_ERR_UNSUPPORTED, "num_seqs must be <= 65535");
  if ((long long)max_blocks_per_seq * block_size >= (1LL << 31) - 64)
    return fail(PKV_ERR_UNSUPPORTED, "max_blocks_per_seq * block_size must be < 2^31 - 64");
  return PKV_OK;
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" {

pkv_status_t paged_kv_reserve_slots(int32_t* block_tables, int32_t max_blocks_per_seq, const int32_t* context_lens,
                                    const int32_t* new_lens, const int32_t* free_blocks, int32_t free_capacity,
                                    const int32_t* num_free, int64_t* slot_mapping, int32_t max_tokens,
                                    int32_t* query_start_loc, int32_t* context_lens_out, int32_t* num_free_out,
                                    int32_t* granted, int32_t num_seqs, int32_t block_size, int32_t num_blocks,
                                    cudaStream_t stream) {
  set_last_error_message("");
  const pkv_status_t st = check_common(num_seqs, max_blocks_per_seq, free_capacity, block_size, num_blocks);
  if (st != PKV_OK) return st;
  if (max_tokens < 0) return fail(PKV_ERR_INVALID_ARG, "max_tokens < 0");
  if (!num_free || !query_start_loc || !num_free_out || (max_tokens > 0 && !slot_mapping) ||
      (free_capacity > 0 && !free_blocks) ||
      (num_seqs > 0 && (!block_tables || !context_lens || !new_lens || !context_lens_out || !granted)))
    return fail(PKV_ERR_INVALID_ARG, "null pointer argument");
  const size_t n = (size_t)num_seqs * sizeof(int32_t);
  const Span written[] = {{"block_tables", block_tables, n * (size_t)max_blocks_per_seq},
                          {"slot_mapping", slot_mapping, (size_t)max_tokens * sizeof(int64_t)},
                          {"query_start_loc", query_start_loc, n + sizeof(int32_t)},
                          {"context_lens_out", context_lens_out, n},
                          {"num_free_out", num_free_out, sizeof(int32_t)},
                          {"granted", granted, n}};
  const Span read[] = {{"context_lens", context_lens, n},
                       {"new_lens", new_lens, n},
                       {"free_blocks", free_blocks, (size_t)free_capacity * sizeof(int32_t)},
                       {"num_free", num_free, sizeof(int32_t)}};
  const pkv_status_t apart = check_apart(written, read);
  if (apart != PKV_OK) return apart;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  ReserveParams p{};
  p.block_tables = block_tables;
  p.context_lens = context_lens;
  p.new_lens = new_lens;
  p.free_blocks = free_blocks;
  p.num_free = num_free;
  p.slot_mapping = slot_mapping;
  p.query_start_loc = query_start_loc;
  p.context_lens_out = context_lens_out;
  p.num_free_out = num_free_out;
  p.granted = granted;
  p.err = device_error_word(dev);
  if (!p.err) return fail(PKV_ERR_CUDA, "device error word unavailable on device %d", dev);
  p.num_seqs = num_seqs;
  p.max_tokens = max_tokens;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.free_capacity = free_capacity;
  p.block_size = block_size;
  p.num_blocks = num_blocks;
  const unsigned grid = max_tokens > 0 ? (unsigned)((max_tokens - 1) / kSlotTokens + 1) : 1u;
  e = launch_kernel(pkv_reserve_slots_kernel, dim3(grid), dim3(kSlotThreads), 0, stream, p);
  if (e != cudaSuccess) return cuda_fail(e, "paged_kv_reserve_slots launch");
  return PKV_OK;
}

pkv_status_t paged_kv_release_blocks(const int32_t* block_tables, int32_t max_blocks_per_seq,
                                     const int32_t* context_lens, const int32_t* finished, int32_t* free_blocks,
                                     int32_t free_capacity, const int32_t* num_free, int32_t* context_lens_out,
                                     int32_t* num_free_out, int32_t num_seqs, int32_t block_size, int32_t num_blocks,
                                     cudaStream_t stream) {
  set_last_error_message("");
  const pkv_status_t st = check_common(num_seqs, max_blocks_per_seq, free_capacity, block_size, num_blocks);
  if (st != PKV_OK) return st;
  if (!num_free || !num_free_out || (free_capacity > 0 && !free_blocks) ||
      (num_seqs > 0 && (!block_tables || !context_lens || !finished || !context_lens_out)))
    return fail(PKV_ERR_INVALID_ARG, "null pointer argument");
  const size_t n = (size_t)num_seqs * sizeof(int32_t);
  const Span written[] = {{"free_blocks", free_blocks, (size_t)free_capacity * sizeof(int32_t)},
                          {"context_lens_out", context_lens_out, n},
                          {"num_free_out", num_free_out, sizeof(int32_t)}};
  const Span read[] = {{"block_tables", block_tables, n * (size_t)max_blocks_per_seq},
                       {"context_lens", context_lens, n},
                       {"finished", finished, n},
                       {"num_free", num_free, sizeof(int32_t)}};
  const pkv_status_t apart = check_apart(written, read);
  if (apart != PKV_OK) return apart;
  const int per_cta = num_seqs > 304 ? (num_seqs + 303) / 304 : 1;  // about two CTAs per SM (at most 216 sequences each)
  if ((long long)per_cta * max_blocks_per_seq >= 1LL << 31)
    return fail(PKV_ERR_UNSUPPORTED, "max_blocks_per_seq times %d sequences must be < 2^31", per_cta);
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  ReleaseParams p{};
  p.block_tables = block_tables;
  p.context_lens = context_lens;
  p.finished = finished;
  p.free_blocks = free_blocks;
  p.num_free = num_free;
  p.context_lens_out = context_lens_out;
  p.num_free_out = num_free_out;
  p.err = device_error_word(dev);
  if (!p.err) return fail(PKV_ERR_CUDA, "device error word unavailable on device %d", dev);
  p.num_seqs = num_seqs;
  p.per_cta = per_cta;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.free_capacity = free_capacity;
  p.block_size = block_size;
  p.num_blocks = num_blocks;
  const unsigned grid = num_seqs > 0 ? (unsigned)((num_seqs + p.per_cta - 1) / p.per_cta) : 1u;
  e = launch_kernel(pkv_release_blocks_kernel, dim3(grid), dim3(kSlotThreads), 0, stream, p);
  if (e != cudaSuccess) return cuda_fail(e, "paged_kv_release_blocks launch");
  return PKV_OK;
}

}  // extern "C"
