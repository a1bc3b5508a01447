// Merge of one output row's split-K partials by log-sum-exp, shared by the reduce kernels of the decode,
// multi-query and scored calls.
#pragma once

#include "pkv_common.cuh"

namespace pkv {

// split-K reduce: merge the partitions' (m_p, l_p, o_p) of one (seq, head) by
// log-sum-exp: out = sum_p w_p o_p / sum_p w_p with w_p = l_p 2^(m_p - max m).
// One warp per output row; lane p holds the weight of partition p (p < 32 per
// round) and each lane merges D/32 dims.

constexpr int kReduceRows = 4;
constexpr int kReduceEarly = 4;  // partitions whose partial outputs are fetched with the first loads

// The first round of loads for output row `row` (partials at base = row * max_partitions):
// this lane's partition (m, l) and the partial outputs of the first kReduceEarly partitions.
// All are in bounds whatever the row's partition count; entries past it are masked later.
template <int D>
__device__ __forceinline__ void reduce_load_row(const float* __restrict__ part_o, const float* __restrict__ part_m,
                                                const float* __restrict__ part_l, size_t base, int max_partitions,
                                                int lane, float& mp, float& lp, float (&o_early)[kReduceEarly][D / 32]) {
  constexpr int DPL = D / 32;
  mp = -INFINITY;
  lp = 0.f;
  if (lane < max_partitions) {
    mp = part_m[base + lane];
    lp = part_l[base + lane];
  }
#pragma unroll
  for (int k = 0; k < kReduceEarly; ++k) {
    if (k < max_partitions) {
      const float* o = part_o + (base + k) * D + lane * DPL;
      if constexpr (DPL == 4) {
        const float4 v = *reinterpret_cast<const float4*>(o);
        o_early[k][0] = v.x; o_early[k][1] = v.y; o_early[k][2] = v.z; o_early[k][3] = v.w;
      } else {
        const float2 v = *reinterpret_cast<const float2*>(o);
        o_early[k][0] = v.x; o_early[k][1] = v.y;
      }
    } else {
#pragma unroll
      for (int e = 0; e < DPL; ++e) o_early[k][e] = 0.f;
    }
  }
}

// Merge the np (> 1) partials of output row `row` into out[row][:], given the first round of loads.
template <typename T, int D>
__device__ __forceinline__ void reduce_combine_row(T* __restrict__ out, const float* __restrict__ part_o,
                                                   const float* __restrict__ part_m,
                                                   const float* __restrict__ part_l, size_t base, size_t row,
                                                   int np, float mp, float lp,
                                                   const float (&o_early)[kReduceEarly][D / 32], int lane) {
  constexpr int DPL = D / 32;
  if (lane >= np) mp = -INFINITY;
  // global max over all partitions (np may exceed 32)
  float M = mp;
  for (int p = 32 + lane; p < np; p += 32) M = fmaxf(M, part_m[base + p]);
  M = warp_max(M);
  float acc[DPL];
#pragma unroll
  for (int e = 0; e < DPL; ++e) acc[e] = 0.f;
  float W = 0.f;
  for (int p0 = 0; p0 < np; p0 += 32) {
    float wp = 0.f;
    if (p0 == 0) {
      wp = mp == -INFINITY ? 0.f : lp * fast_exp2(mp - M);
    } else if (p0 + lane < np) {
      const float m2 = part_m[base + p0 + lane];
      wp = m2 == -INFINITY ? 0.f : part_l[base + p0 + lane] * fast_exp2(m2 - M);
    }
    W += wp;
    const int cnt = np - p0 < 32 ? np - p0 : 32;
    int k = 0;
    if (p0 == 0) {
#pragma unroll
      for (int q = 0; q < kReduceEarly; ++q) {
        const float w = __shfl_sync(kFull, wp, q);
        if (q < cnt) {
#pragma unroll
          for (int e = 0; e < DPL; ++e) acc[e] = fmaf(w, o_early[q][e], acc[e]);
        }
      }
      k = kReduceEarly;
    }
    for (; k < cnt; ++k) {
      const float w = __shfl_sync(kFull, wp, k);
      const float* o = part_o + (base + p0 + k) * D + lane * DPL;
      if constexpr (DPL == 4) {
        const float4 v = *reinterpret_cast<const float4*>(o);
        acc[0] = fmaf(w, v.x, acc[0]);
        acc[1] = fmaf(w, v.y, acc[1]);
        acc[2] = fmaf(w, v.z, acc[2]);
        acc[3] = fmaf(w, v.w, acc[3]);
      } else {
        const float2 v = *reinterpret_cast<const float2*>(o);
        acc[0] = fmaf(w, v.x, acc[0]);
        acc[1] = fmaf(w, v.y, acc[1]);
      }
    }
  }
  W = warp_sum(W);
  const float inv = W > 0.f ? 1.f / W : 0.f;
  T* dst = out + row * D + lane * DPL;
  if constexpr (DPL == 4) {
    uint2 v;
    v.x = Elem<T>::pack2(acc[0] * inv, acc[1] * inv);
    v.y = Elem<T>::pack2(acc[2] * inv, acc[3] * inv);
    *reinterpret_cast<uint2*>(dst) = v;
  } else {
    *reinterpret_cast<uint32_t*>(dst) = Elem<T>::pack2(acc[0] * inv, acc[1] * inv);
  }
}

}  // namespace pkv
