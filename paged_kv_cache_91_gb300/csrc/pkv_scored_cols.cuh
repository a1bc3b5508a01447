// Scored paged attention with few rows per kv head: 8 (query token, head) rows per CTA in the n = 8 dimension
// of the warp MMAs, the CTA's warps splitting the partition's blocks (pkv_scored_tile.cuh). Row r of a (sequence,
// kv head) is query token r / G, head kvh * G + r % G; decode is the case of one query token, with every group
// size, 1 included.
//
// A tile's products become scores in registers (ScoredRule): some 8 instructions a score beside the 2 * D * 2
// bytes of K and V that up to 8 rows share, so over a 16-bit pool the kernel stays bound by reading them (256
// contexts, 32/8 heads, cap 50, window 1024: 154 us, 6.6 TB/s; 12 contexts of 9001 to 16384 tokens, 40 heads,
// distance biases: 462 us, 7.2 TB/s). An E4M3 pool halves the bytes and the widening of its codes doubles the
// instructions a byte: no unit is full (issue slots 47 %, HBM 71 %), and warps wait for their copies most (128 contexts
// to 4096 tokens, 64/8 heads, cap 30: 121 us, 5.3 TB/s). Only the blocks between the CTA's first and last visible key
// are copied.
#pragma once

#include "pkv_scored.cuh"
#include "pkv_scored_tile.cuh"

namespace pkv {

struct ScoredRule {
  float mul0, mul1;      // of the raw product: scale * log2(e), or scale / softcap
  float cap_out;         // softcap * log2(e), 0: no cap
  bool biased;
  float slope0, slope1;  // times log2(e)
  int lo0, n0, lo1, n1;  // the columns' visible keys [lo, lo + n)
  int pos0, pos1;        // the columns' positions
  int tok_base;          // position of the tile's token 0
  bool whole;            // every column of the warp sees every token of the tile
  __device__ __forceinline__ void operator()(float (&x)[4], int ta, bool va, int tb, bool vb) const {
    const int ja = tok_base + ta, jb = tok_base + tb;
    bool see[4] = {true, true, true, true};
    if (!whole) {
      see[0] = va && (unsigned)(ja - lo0) < (unsigned)n0;
      see[1] = va && (unsigned)(ja - lo1) < (unsigned)n1;
      see[2] = vb && (unsigned)(jb - lo0) < (unsigned)n0;
      see[3] = vb && (unsigned)(jb - lo1) < (unsigned)n1;
    }
    x[0] *= mul0;
    x[1] *= mul1;
    x[2] *= mul0;
    x[3] *= mul1;
    if (cap_out != 0.f) {
      float z = 0.f;  // (of the keys that are seen: the others may hold anything)
#pragma unroll
      for (int e = 0; e < 4; ++e) z = fmaxf(z, see[e] ? fabsf(x[e]) : 0.f);
      if (__all_sync(kFull, z <= 0.5f)) {
        // tanh(z) / z in z^2 on [0, 1/4]: a minimax fit, relative error 6e-7
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float u = x[e] * x[e];
          const float q = fmaf(u, fmaf(u, fmaf(u, -0.0444022226f, 0.131902965f), -0.333263179f), 0.999999456f);
          x[e] = cap_out * (x[e] * q);
        }
      } else {
        // some score is of the cap's size: the cancellation of 1 - 2 / (e^(2 z) + 1) is small beside it, but not beside
        // a small score, which keeps to the polynomial whatever stands beside it
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float u = x[e] * x[e];
          const float q = fmaf(u, fmaf(u, fmaf(u, -0.0444022226f, 0.131902965f), -0.333263179f), 0.999999456f);
          const float far = cap_out - 2.f * cap_out * fast_rcp(fast_exp2(x[e] * 2.8853900817779268f) + 1.f);
          x[e] = fabsf(x[e]) <= 0.5f ? cap_out * (x[e] * q) : far;
        }
      }
    }
    if (biased) {
      x[0] = fmaf(-slope0, fabsf((float)(pos0 - ja)), x[0]);
      x[1] = fmaf(-slope1, fabsf((float)(pos1 - ja)), x[1]);
      x[2] = fmaf(-slope0, fabsf((float)(pos0 - jb)), x[2]);
      x[3] = fmaf(-slope1, fabsf((float)(pos1 - jb)), x[3]);
    }
    if (!whole) {
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = see[e] ? x[e] : -INFINITY;
    }
  }
};

// C: the cache's element type (the tile's T, or E4M3).
template <typename Tile, typename C, int NW, int SPW>
__global__ void __launch_bounds__(NW * 32, Tile::MIN_CTAS)
    pkv_scored_cols_kernel(const __grid_constant__ DecodeParams p, const __grid_constant__ ScoreParams sc,
                           const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
  pdl_begin();
  using T = typename Tile::T;
  constexpr int D = Tile::D, BS = Tile::BS;
  using Sh = MmaShape<D, BS, NW, SPW, Tile::TILE>;
  extern __shared__ __align__(128) unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));

  // the last row tiles first: with a causal limit they see the most keys
  const int part = blockIdx.x / sc.row_tiles, rt = sc.row_tiles - 1 - (int)blockIdx.x % sc.row_tiles;
  const int kvh = blockIdx.y;
  const int s = blockIdx.z;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = p.group, P = p.partition_size;
  const bool reporter = blockIdx.x == 0 && kvh == 0 && threadIdx.x == 0;
  const int ctx = clamp_context(p, s, reporter);
  int q0 = 0;
  const int q_len = scored_query_len(sc, s, ctx, q0);
  if (q_len < 0) {
    if (reporter) atomicOr(p.err, PKV_DEVERR_QUERY);
    return;
  }
  const int R = q_len * G, row0 = rt * 8;
  if (row0 >= R) return;
  const int ncol = min(8, R - row0);
  const int base = scored_base(sc, ctx, q_len, BS);

  // lane / 4: this lane's query column n (rows past ncol repeat the last one and are not stored)
  const int rn = row0 + min(lane >> 2, ncol - 1);
  const int tn = q0 + rn / G, hn = kvh * G + rn % G, pn = ctx - q_len + rn / G;
  int lo, hi;
  scored_span(sc, tn, pn, ctx, lo, hi);
  const RowParts parts = row_parts(lo, hi, base, P);
  // the CTA's keys: from its rows' first to their last visible one, within the partition
  int c0 = hi > lo ? lo : INT32_MAX, c1 = hi > lo ? hi : 0;
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) {
    c0 = min(c0, __shfl_xor_sync(kFull, c0, o));
    c1 = max(c1, __shfl_xor_sync(kFull, c1, o));
  }
  const int tok0 = base + part * P;  // (no overflow: the host bounds contexts by 2^30)
  c0 = max(c0, tok0);
  c1 = min(c1, tok0 + P);
  if (c1 <= c0) {  // no key: partition 0 writes the zeros of rows that see nothing
    if (part == 0 && warp == 0 && parts.last < parts.first && (lane >> 2) < ncol) {
      T* out = static_cast<T*>(p.out) + ((size_t)tn * p.num_heads + hn) * D;
      for (int d = (lane & 3) * 8; d < D; d += 32) *reinterpret_cast<uint4*>(out + d) = make_uint4(0u, 0u, 0u, 0u);
    }
    return;
  }
  const int blk0 = c0 / BS;
  const int nblk = (c1 + BS - 1) / BS - blk0;
  const int nmine = warp < nblk ? (nblk - warp + NW - 1) / NW : 0;  // <= 32: P spans at most 32 NW blocks

  if (threadIdx.x == 0) {
    prefetch_tensormap(&kmap);
    prefetch_tensormap(&vmap);
  }
  int my_phys = -1;
  if (lane < nmine) {
    const int v = p.block_tables[(size_t)s * p.max_blocks_per_seq + blk0 + warp + NW * lane];
    if ((unsigned)v < (unsigned)p.num_blocks) {
      my_phys = v;
    } else {
      atomicOr(p.err, PKV_DEVERR_BLOCK_ID);
    }
  }

  unsigned char* ring = smem + warp * SPW * Sh::STAGE;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Sh::BARS) + warp * SPW;
  if (lane == 0) {
#pragma unroll
    for (int k = 0; k < SPW; ++k) mbar_init(bars + k, 1);
    fence_mbar_init();
  }
  __syncwarp();

  unsigned zeroed = 0;  // stages with value rows zeroed since their last refill
  auto issue = [&](int i) {
    const int phys = __shfl_sync(kFull, my_phys, i);
    if (lane == 0) {
      uint64_t* bar = bars + (i % SPW);
      unsigned char* st = ring + (i % SPW) * Sh::STAGE;
      if (phys >= 0) {
        if (PKV_PROXY_FENCE || ((zeroed >> (i % SPW)) & 1u)) fence_proxy_async_smem();
        mbar_arrive_expect_tx(bar, Sh::STAGE);
        Tile::issue_tiles(st, &kmap, &vmap, (phys * p.num_kv_heads + kvh) * BS, bar);
      } else {
        mbar_arrive(bar);
      }
    }
  };
  const int nfirst = nmine < SPW ? nmine : SPW;
  for (int i = 0; i < nfirst; ++i) issue(i);
  int issued = nfirst;

  const T* qrow =
      (lane >> 2) < ncol ? reinterpret_cast<const T*>(p.query) + ((size_t)tn * p.num_heads + hn) * D : nullptr;
  typename Tile::QB qb;
  float fa = 1.f, fb = 1.f;  // factors of this lane's two columns' products
  if constexpr (Tile::FP8)
    Tile::load_qb_row(qb, qrow, lane, 1.f, fa, fb);  // per-column f16 scaling of a bf16 query
  else
    Tile::load_qb_row(qb, qrow, lane);
  const int j0 = (lane & 3) * 2;  // its two accumulator columns
  ScoredRule rule;
  {
    const float mul = sc.cap_out != 0.f ? sc.cap_in : p.scale_log2;
    const float slope = sc.slopes ? sc.slopes[hn] * 1.4426950408889634f : 0.f;
    rule.cap_out = sc.cap_out;
    rule.biased = sc.slopes != nullptr;
    rule.mul0 = mul * fa;
    rule.mul1 = mul * fb;
    rule.slope0 = __shfl_sync(kFull, slope, 4 * j0);
    rule.slope1 = __shfl_sync(kFull, slope, 4 * j0 + 4);
    rule.pos0 = __shfl_sync(kFull, pn, 4 * j0);
    rule.pos1 = __shfl_sync(kFull, pn, 4 * j0 + 4);
    rule.lo0 = __shfl_sync(kFull, lo, 4 * j0);
    rule.lo1 = __shfl_sync(kFull, lo, 4 * j0 + 4);
    rule.n0 = __shfl_sync(kFull, hi - lo, 4 * j0);
    rule.n1 = __shfl_sync(kFull, hi - lo, 4 * j0 + 4);
  }

  float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
  float acc[Tile::KT][4];
#pragma unroll
  for (int mt = 0; mt < Tile::KT; ++mt) acc[mt][0] = acc[mt][1] = acc[mt][2] = acc[mt][3] = 0.f;

  int failed_at = -1;
  for (int i = 0; i < nmine; ++i) {
    const int phys = __shfl_sync(kFull, my_phys, i);
    const int k = i % SPW;
    const bool ready = __all_sync(kFull, mbar_wait(bars + k, (i / SPW) & 1));
    if (!ready) {
      failed_at = i;
      break;
    }
    if (phys >= 0) {
      unsigned char* Ks = ring + k * Sh::STAGE;
      rule.tok_base = (blk0 + warp + NW * i) * BS;
      const int first = max(0, c0 - rule.tok_base), nvalid = min(BS, c1 - rule.tok_base);
      // (a tile of 8 tokens fills half of the MMA's rows: its other rows are masked)
      rule.whole = BS >= 16 && first == 0 && nvalid == BS &&
                   __all_sync(kFull, lo <= rule.tok_base && rule.tok_base + BS <= hi);
      Tile::fold(Ks, Ks + Sh::TILE, first, nvalid, qb, lane, m0, m1, l0, l1, acc, rule);
      if (first > 0 || nvalid < BS) zeroed |= 1u << k;
    }
    __syncwarp();
    if (i + SPW < nmine) {
      issue(i + SPW);
      zeroed &= ~(1u << k);
      ++issued;
    }
  }

  if (failed_at >= 0) {
    if (lane == 0) atomicOr(p.err, PKV_DEVERR_TIMEOUT);
    for (int j = failed_at; j < issued; ++j) mbar_wait(bars + (j % SPW), (j / SPW) & 1);
    m0 = m1 = -INFINITY;
    l0 = l1 = 0.f;
#pragma unroll
    for (int mt = 0; mt < Tile::KT; ++mt) acc[mt][0] = acc[mt][1] = acc[mt][2] = acc[mt][3] = 0.f;
  }
  Tile::finish(l0, l1);

  // merge the warps: each warp writes [column][D] accumulators, m, l into its own ring slice
  float* red = reinterpret_cast<float*>(ring);
  float* red_m = red + 8 * D;
  float* red_l = red_m + 8;
  Tile::store_acc(red, acc, lane);
  if (lane < 4) {
    red_m[j0] = m0;
    red_m[j0 + 1] = m1;
    red_l[j0] = l0;
    red_l[j0 + 1] = l1;
  }
  __syncthreads();
  constexpr int DPL = D / 32;
  for (int n = warp; n < ncol; n += NW) {  // a warp per row
    const int nlo = __shfl_sync(kFull, lo, 4 * n), nhi = __shfl_sync(kFull, hi, 4 * n);
    const RowParts np = row_parts(nlo, nhi, base, P);
    if (!np.in(part)) continue;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < NW; ++w) M = fmaxf(M, reinterpret_cast<float*>(smem + w * SPW * Sh::STAGE)[8 * D + n]);
    float L = 0.f, o[DPL];
#pragma unroll
    for (int e = 0; e < DPL; ++e) o[e] = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const float* rw = reinterpret_cast<float*>(smem + w * SPW * Sh::STAGE);
      const float mw = rw[8 * D + n];
      const float f = mw == -INFINITY ? 0.f : fast_exp2(mw - M);
      L += rw[8 * D + 8 + n] * f;
#pragma unroll
      for (int e = 0; e < DPL; ++e) o[e] += rw[n * D + lane * DPL + e] * f;
    }
    float inv = L != 0.f ? 1.f / L : 0.f;
    if constexpr (Tile::FP8) inv *= p.v_scale * Tile::UNIT;  // V codes -> values
    bool fine = true;
#pragma unroll
    for (int e = 0; e < DPL; ++e) {
      o[e] *= inv;
      fine = fine && fabsf(o[e]) < INFINITY;
    }
    const int r = row0 + n, h = kvh * G + r % G;
    const size_t row = (size_t)(q0 + r / G) * p.num_heads + h;
    // a non-finite row is a masked key's doing only if it misses some of the keys that the CTA multiplies, and not if
    // its own scores are NaN
    if (!__all_sync(kFull, fine) && L == L && (nlo > c0 || nhi < c1))
      scored_row<T, C, D>(p, sc, row, s, h, ctx - q_len + r / G, max(nlo, tok0), min(nhi, tok0 + P), BS, lane, M, L, o);
    store_row<T, D>(p, row, part, np.direct(), lane, M, L, o);
  }
}

template <typename Tile, typename C, int RING_BYTES = PKV_MMA_RING_BYTES>
cudaError_t launch_scored_cols(const DecodeParams& p, const ScoreParams& sc, const CUtensorMap& kmap,
                               const CUtensorMap& vmap, int num_seqs, cudaStream_t stream) {
  constexpr int NW = kDecodeWarps;
  constexpr int SPW = mma_stages<2 * Tile::TILE, RING_BYTES>();
  using Sh = MmaShape<Tile::D, Tile::BS, NW, SPW, Tile::TILE>;
  auto kern = pkv_scored_cols_kernel<Tile, C, NW, SPW>;
  static bool configured[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64) return cudaErrorInvalidDevice;
  if (!configured[dev]) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::SMEM);
    if (e != cudaSuccess) return e;
    configured[dev] = true;
  }
  const dim3 grid((unsigned)p.max_partitions * (unsigned)sc.row_tiles, (unsigned)p.num_kv_heads, (unsigned)num_seqs);
  return launch_kernel(kern, grid, dim3(NW * 32), Sh::SMEM, stream, p, sc, kmap, vmap);
}

}  // namespace pkv
