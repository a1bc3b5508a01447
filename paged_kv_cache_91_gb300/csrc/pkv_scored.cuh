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
  float cap_in = 0.f;                   // scale / softcap (0: no cap)
  float cap_out = 0.f;                  // softcap * log2(e)
};

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

// The score, in the base-2 domain, of a raw product `s` (without scale): sl2 = scale * log2(e).
__device__ __forceinline__ float score_value(const ScoreParams& sc, float s, float sl2) {
  return sc.cap_in != 0.f ? sc.cap_out * score_tanh(s * sc.cap_in) : s * sl2;
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

// The visible keys [lo, hi) of query token t at position p in a context of ctx tokens (hi >= lo).
__device__ __forceinline__ void scored_span(const ScoreParams& sc, int t, int p, int ctx, int& lo, int& hi) {
  lo = sc.window > 0 && p >= sc.window ? p - sc.window + 1 : 0;
  if (sc.key_begin) lo = max(lo, sc.key_begin[t]);
  hi = p + 1;
  if (sc.key_end) hi = min(sc.key_end[t], ctx);
  hi = max(hi, lo);
}

}  // namespace pkv
