// Scored paged attention: attention over the paged pool whose scores are capped by a tanh and biased by
// distance, and whose query tokens each see an interval of key positions. What the kernels share: the rules
// of a launch, the visible interval of a query token, and a score's value.
//
// Query token t of a sequence with context n sits at position p. With x_j = scale * dot(q, K_j):
//   x_j <- softcap * tanh(x_j / softcap)   (softcap > 0)
//   x_j <- x_j - slope_h * |p - j|         (alibi_slopes)
//   visible: j in [lo, hi), lo = max(0, key_begin[t], p - window + 1), hi = min(n, key_end[t] or p + 1)
// A token with an empty interval gives zeros. Scores live in the base-2 domain: the kernels work with
// x_j * log2(e) and exp2.
#pragma once

#include "pkv_common.cuh"

namespace pkv {

struct ScoreParams {
  const float* slopes = nullptr;        // [num_heads], or null: no distance bias
  const int32_t* key_begin = nullptr;   // [query tokens], or null: 0
  const int32_t* key_end = nullptr;     // [query tokens], or null: p + 1
  const int32_t* query_start_loc = nullptr;  // [num_seqs + 1], or null: query token s is sequence s's only one
  int window = 0;                       // keys p - window + 1 .. are visible; 0: no window
  int num_query_tokens = 0;             // host bound on query_start_loc entries
  int max_query_len = 1;                // host bound on every q_len
  float cap_in = 0.f;                   // scale / softcap
  float cap_out = 0.f;                  // softcap * log2(e); 0: no cap
  int row_tiles = 1;                    // row tiles per (partition, kv head, sequence)
  const uint32_t* tree_mask = nullptr;  // [query tokens][mask_words], of the kernels for trees (TREE)
  int mask_words = 0;
  int sort_seqs = 0;                    // tree, tensor-memory tile: num_seqs to take them longest first, else 0
};

constexpr int kTreeSortSeqs = 128;  // sequences that a CTA of the tree's tensor-memory tile can sort

__device__ __forceinline__ float fast_rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// tanh(z): below 1 an odd polynomial, a minimax fit of tanh(z) / z in z^2 on [0, 1] (relative error 5e-8);
// above, 1 - 2 / (e^(2 z) + 1), whose cancellation costs nothing there (|tanh| > 0.76). tanh.approx has a
// relative error of 2^-11, which at a cap of 50 would move a score by up to 0.02.
__device__ __forceinline__ float score_tanh(float z) {
  const float u = z * z;
  float q = 0.0010410216f;
  q = fmaf(q, u, -0.00620337599f);
  q = fmaf(q, u, 0.0202899769f);
  q = fmaf(q, u, -0.0534570277f);
  q = fmaf(q, u, 0.13325204f);
  q = fmaf(q, u, -0.333328391f);
  q = fmaf(q, u, 0.99999995f);
  const float e = fast_exp2(z * 2.8853900817779268f);  // e^(2z): infinity gives 1, 0 gives -1
  const float far = 1.f - __fdividef(2.f, e + 1.f);
  return u < 1.f ? q * z : far;
}

// q_len of sequence s with (clamped) context ctx and its first query row q0; -1 if query_start_loc is
// inconsistent with the bounds or the context. Without query_start_loc: one query token per sequence.
__device__ __forceinline__ int scored_query_len(const ScoreParams& sc, int s, int ctx, int& q0) {
  if (!sc.query_start_loc) {
    q0 = s;
    return 1;
  }
  q0 = sc.query_start_loc[s];
  const int q1 = sc.query_start_loc[s + 1];
  // (compared without a difference that could overflow)
  if (q0 < 0 || q1 < q0 || q1 > sc.num_query_tokens || q1 - q0 > sc.max_query_len || q1 - q0 > ctx) return -1;
  return q1 - q0;
}

// The n lowest bits (all from 32 on, none for n <= 0).
__device__ __forceinline__ uint32_t low_bits(int n) {
  return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u;
}

// The visible keys [lo, hi) of query token t at position p in a context of ctx tokens (hi >= lo). TREE: the query
// tokens are nodes of a tree, the context's last q_len positions; of those a token sees the ones in its mask, so that
// its interval ends with the context.
template <bool TREE = false>
__device__ __forceinline__ void scored_span(const ScoreParams& sc, int t, int p, int ctx, int& lo, int& hi) {
  if constexpr (TREE) {
    lo = sc.key_begin ? max(0, sc.key_begin[t]) : 0;
    hi = max(ctx, lo);
    return;
  }
  lo = sc.window > 0 && p >= sc.window ? p - sc.window + 1 : 0;
  if (sc.key_begin) lo = max(lo, sc.key_begin[t]);
  hi = p + 1;
  if (sc.key_end) hi = min(sc.key_end[t], ctx);
  hi = max(hi, lo);
}

// TREE: bit i says whether query token t sees the key of its sequence's node u + i; the keys before node 0 are
// committed ones, which it does.
__device__ __forceinline__ uint32_t tree_bits(const ScoreParams& sc, int t, int u) {
  if (u <= -32) return 0xffffffffu;
  const uint32_t* words = sc.tree_mask + (size_t)t * sc.mask_words;
  const int w = u >> 5;  // (rounded down: -1 for u < 0)
  const uint32_t a = w < 0 ? 0xffffffffu : w < sc.mask_words ? words[w] : 0u;
  const uint32_t b = w + 1 < sc.mask_words ? words[w + 1] : 0u;
  return __funnelshift_r(a, b, u & 31);
}

// Whether one of the tokens ta .. tb of a sequence (its context ctx tokens, its first query row q0) sees a key of
// the block that starts at place at. Asked only of a block with a bad id: an error if it is seen, else nothing.
template <bool TREE, int BS>
__device__ __noinline__ bool block_seen(const ScoreParams& sc, int q0, int q_len, int ctx, int ta, int tb, int at) {
  for (int t = ta; t <= tb; ++t) {
    int lo, hi;
    scored_span<TREE>(sc, q0 + t, ctx - q_len + t, ctx, lo, hi);
    uint32_t see = low_bits(min(hi - at, BS)) & ~low_bits(lo - at);
    if constexpr (TREE) {
      if (see) see &= tree_bits(sc, q0 + t, at - (ctx - q_len));
    }
    if (see) return true;
  }
  return false;
}

// A sequence's partitions: partition k holds the positions [base + k P, base + (k + 1) P), where base is the
// start of the block of the first position that the window leaves visible to any of its query tokens (0
// without a window). So a window costs as many partitions as it spans, wherever it lies in the context.
__device__ __forceinline__ int scored_base(const ScoreParams& sc, int ctx, int q_len, int block_size) {
  const int p0 = ctx - q_len;  // position of the first query token
  return sc.window > 0 && p0 >= sc.window ? (p0 - sc.window + 1) / block_size * block_size : 0;
}

// The partitions first .. last of a row that sees [lo, hi) (lo >= base); last < first: it sees nothing. A row
// of at most one partition is written to the output directly, by partition 0 if it is empty.
struct RowParts {
  int first, last;
  __device__ __forceinline__ bool direct() const { return last <= first; }
  __device__ __forceinline__ bool in(int part) const {
    return last < first ? part == 0 : first <= part && part <= last;
  }
};
__device__ __forceinline__ RowParts row_parts(int lo, int hi, int base, int P) {
  if (hi <= lo) return {0, -1};
  return {(lo - base) / P, (hi - 1 - base) / P};
}

// The SM's clock in steps of 2^kWorkClock, which a warp at long work stores as a sign of it for those that wait.
constexpr int kWorkClock = 10;
__device__ __forceinline__ unsigned work_clock() { return (unsigned)((unsigned long long)clock64() >> kWorkClock); }

// This lane's D / 32 dims of a stored row (16-bit or E4M3 codes).
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

// One row over the keys [a, b) on one warp: (m, l) and the output normalised by l. Lane t scores key t of 32, then
// the lanes hold D / 32 dims each for their weighted values. The tiles multiply every key of a tile with every row,
// a masked one with weight 0, and 0 times a NaN or infinite value is NaN: a row that such a value may have reached
// is computed again here, where a masked key is not touched. pos: the row's position; TREE: that of node 0 (there is
// no distance bias). sign: where to leave a sign of work every 32 keys; or null.
template <typename T, typename C, int D, bool TREE = false>
__device__ __noinline__ void scored_row(const DecodeParams& p, const ScoreParams& sc, size_t row, int s, int h,
                                        int pos, int a, int b, int block_size, int lane, float& m, float& l,
                                        float (&o)[D / 32], volatile int* sign = nullptr) {
  constexpr int DPL = D / 32, EB = CacheFmt<C>::EB, EPP = 16 / EB;
  const int g = h / p.group;
  const float slope = sc.slopes ? sc.slopes[h] * 1.4426950408889634f : 0.f;
  const unsigned char* q = static_cast<const unsigned char*>(p.query) + row * D * 2;
#pragma unroll
  for (int e = 0; e < DPL; ++e) o[e] = 0.f;
  m = -INFINITY;
  l = 0.f;
  for (int j0 = a; j0 < b; j0 += 32) {
    if (sign && lane == 0) *sign = (int)work_clock();
    const int j = j0 + lane;
    const int phys = j < b ? p.block_tables[(size_t)s * p.max_blocks_per_seq + j / block_size] : -1;
    bool ok = (unsigned)phys < (unsigned)p.num_blocks;  // (a bad id is reported by the tile)
    if constexpr (TREE) {
      if (ok && j >= pos) ok = tree_bits(sc, (int)(row / p.num_heads), j - pos) & 1u;
    }
    const size_t at = ok ? (((size_t)phys * p.num_kv_heads + g) * block_size + j % block_size) * D * EB : 0;
    float d = 0.f;
    if (ok) {
#pragma unroll 4
      for (int c = 0; c < D / EPP; ++c) {
        const uint4 k4 = *reinterpret_cast<const uint4*>(p.key_cache + at + c * 16);
        const uint32_t kw[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
        for (int e = 0; e < EPP / 2; ++e) {
          const float2 kf = CacheFmt<C>::pair(EB == 1 ? kw[e / 2] >> (16 * (e & 1)) : kw[e & 3]);
          const float2 qf = Elem<T>::to_float2(*reinterpret_cast<const uint32_t*>(q + (c * EPP + 2 * e) * 2));
          d = fmaf(qf.x, kf.x, d);
          d = fmaf(qf.y, kf.y, d);
        }
      }
    }
    const float x = ok ? (sc.cap_out != 0.f ? sc.cap_out * score_tanh(d * sc.cap_in) : d * p.scale_log2) -
                             slope * fabsf((float)(pos - j))
                       : -INFINITY;
    const float mn = fmaxf(m, warp_max(x)), ms = mn == -INFINITY ? 0.f : mn;
    const float f = fast_exp2(m - ms), w = ok ? fast_exp2(x - ms) : 0.f;
    l = fmaf(l, f, warp_sum(w));
    m = mn;
#pragma unroll
    for (int e = 0; e < DPL; ++e) o[e] *= f;
    const unsigned in = __ballot_sync(kFull, ok);
#pragma unroll 4
    for (int t = 0; t < 32; ++t) {
      const float wt = __shfl_sync(kFull, w, t);
      const size_t vt = __shfl_sync(kFull, (unsigned long long)at, t);
      if ((in >> t) & 1u) {
        float v[DPL];
        load_dims<D, C>(v, p.value_cache + vt, lane);
#pragma unroll
        for (int e = 0; e < DPL; ++e) o[e] = fmaf(wt, v[e], o[e]);
      }
    }
  }
  const float inv = l != 0.f ? p.v_scale / l : 0.f;
#pragma unroll
  for (int e = 0; e < DPL; ++e) o[e] *= inv;
  if (l != l) m = 0.f;  // (a partial with m = -inf would be left out of the merge)
}

// The first and the last key of [a, b) whose value row of kv head g holds a NaN or an infinity (first > last: none),
// on one warp. sign as in scored_row, every 1024 keys.
template <typename C, int D>
__device__ __noinline__ void bad_values(const DecodeParams& p, int s, int g, int a, int b, int block_size, int lane,
                                        int& first, int& last, volatile int* sign) {
  constexpr int EB = CacheFmt<C>::EB, CH = D * EB / 16, KPI = 32 / CH;  // pieces of a row, keys per load
  first = INT32_MAX;
  last = -1;
#pragma unroll 4
  for (int j0 = a; j0 < b; j0 += KPI) {
    if (((j0 - a) & 1023) == 0 && lane == 0) *sign = (int)work_clock();
    const int j = j0 + lane / CH;
    if (j >= b) continue;
    const int phys = p.block_tables[(size_t)s * p.max_blocks_per_seq + j / block_size];
    if ((unsigned)phys >= (unsigned)p.num_blocks) continue;
    const uint4 v4 = *reinterpret_cast<const uint4*>(
        p.value_cache + (((size_t)phys * p.num_kv_heads + g) * block_size + j % block_size) * D * EB + lane % CH * 16);
    const uint32_t v[4] = {v4.x, v4.y, v4.z, v4.w};
    bool bad = false;
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int k = 0; k < 2 / EB; ++k) {
        const float2 f = CacheFmt<C>::pair(v[e] >> (16 * k));
        bad = bad || !(fabsf(f.x) < INFINITY) || !(fabsf(f.y) < INFINITY);
      }
    if (bad) {
      first = min(first, j);
      last = max(last, j);
    }
  }
  first = __reduce_min_sync(kFull, first);
  last = __reduce_max_sync(kFull, last);
}

// The row's result of one partition: the output itself, or its partial.
template <typename T, int D>
__device__ __forceinline__ void store_row(const DecodeParams& p, size_t row, int part, bool direct, int lane,
                                          float m, float l, const float (&o)[D / 32]) {
  constexpr int DPL = D / 32;
  if (direct) {
    uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<T*>(p.out) + row * D + lane * DPL);
#pragma unroll
    for (int e = 0; e < DPL / 2; ++e) dst[e] = Elem<T>::pack2(o[2 * e], o[2 * e + 1]);
  } else {
    const size_t at = row * p.max_partitions + part;
    float2* dst = reinterpret_cast<float2*>(p.part_o + at * D + lane * DPL);
#pragma unroll
    for (int e = 0; e < DPL / 2; ++e) dst[e] = make_float2(o[2 * e], o[2 * e + 1]);
    if (lane == 0) {
      p.part_m[at] = m;
      p.part_l[at] = l;
    }
  }
}

}  // namespace pkv
