// The tiles of the 8-column scored kernel: the layouts, operands and merges of the decode tiles (MmaTile,
// MmaTileE4M3), with a fold() whose scores come from a rule and whose columns may see no token of a tile.
//
// rule(x, ta, va, tb, vb) turns a lane's four raw products -- column 0 and column 1 with token ta of the tile, then
// with token tb -- into scores in the base-2 domain, -inf where the column does not see the token (va, vb: it is
// among the tile's valid tokens first .. nvalid-1). Value rows of the other tokens are zeroed in shared memory (the
// stage then needs a proxy fence before the copy engine refills it).
#pragma once

#include "pkv_decode_mma.cuh"
#include "pkv_decode_mma_fp8.cuh"

namespace pkv {

template <typename T_, int D_, int BS_>
struct ScoredTile : MmaTile<T_, D_, BS_> {
  using Base = MmaTile<T_, D_, BS_>;
  using T = T_;
  static constexpr int D = D_, BS = BS_, NBOX = Base::NBOX, CH = Base::CH, KT = Base::KT;

  template <typename Rule>
  static __device__ __forceinline__ void fold(unsigned char* Ks, unsigned char* Vs, int first, int nvalid,
                                              const uint32_t (&qb)[KT][2], int lane, float& m0, float& m1,
                                              float& l0, float& l1, float (&acc)[KT][4], const Rule& rule) {
    const int mi = lane >> 3;  // which 8x8 matrix this lane addresses in ldmatrix
    const int r8 = lane & 7;   // row inside that matrix
    const int r0 = lane >> 2;  // accumulator rows r0 and r0 + 8
    if (nvalid < BS) {
      // value rows past the context may hold anything (even NaN): zero them so
      // that their zero weights contribute exactly zero
      const int nz = (BS - nvalid) * (D / 8);
      for (int idx = lane; idx < nz; idx += 32) {
        const int t = nvalid + idx / (D / 8), piece = idx % (D / 8);
        *reinterpret_cast<uint4*>(Vs + swz_offset<BS, NBOX>(t, piece)) = make_uint4(0u, 0u, 0u, 0u);
      }
      __syncwarp();
    }
    if (first > 0) {
      for (int idx = lane; idx < first * (D / 8); idx += 32)
        *reinterpret_cast<uint4*>(Vs + swz_offset<BS, NBOX>(idx / (D / 8), idx % (D / 8))) = make_uint4(0u, 0u, 0u, 0u);
      __syncwarp();
    }
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      if (c * 16 < nvalid && c * 16 + 16 > first) {
        // scores S^T[token][head] for 16 tokens, in two accumulation chains
        float sacc[4] = {0.f, 0.f, 0.f, 0.f};
        {
          float sacc2[4] = {0.f, 0.f, 0.f, 0.f};
          const int rr = r8 + ((mi & 1) << 3);  // A rows 0..15
          const int t = BS >= 16 ? c * 16 + rr : (rr & (BS - 1));
#pragma unroll
          for (int kk = 0; kk < KT; ++kk) {
            uint32_t a[4];
            ldmatrix_x4(a, Ks + swz_offset<BS, NBOX>(t, kk * 2 + (mi >> 1)));
            if (kk & 1) {
              Mma<T>::run(sacc2, a, qb[kk][0], qb[kk][1]);
            } else {
              Mma<T>::run(sacc, a, qb[kk][0], qb[kk][1]);
            }
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) sacc[e] += sacc2[e];
        }
        const int ta = c * 16 + r0, tb = ta + 8;
        const bool va = (BS >= 16 || r0 < BS) && ta < nvalid && ta >= first;
        const bool vb = BS >= 16 && tb < nvalid && tb >= first;
        rule(sacc, ta, va, tb, vb);
        const float x00 = sacc[0], x01 = sacc[1], x10 = sacc[2], x11 = sacc[3];
        // Lazy rescaling: a column's reference m moves (and its state is rescaled) only when one of its
        // scores exceeds m by more than 8, so p = 2^(x - m) <= 2^8. Each lane tests its own scores and the
        // warp votes; the max is reduced across the lanes only when some score does exceed.
        float mx0 = fmaxf(x00, x10), mx1 = fmaxf(x01, x11);
        if (__any_sync(kFull, mx0 > m0 + 8.f || mx1 > m1 + 8.f)) {
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) {
            mx0 = fmaxf(mx0, __shfl_xor_sync(kFull, mx0, o));
            mx1 = fmaxf(mx1, __shfl_xor_sync(kFull, mx1, o));
          }
          const bool up0 = mx0 > m0 + 8.f, up1 = mx1 > m1 + 8.f;
          const float mn0 = up0 ? mx0 : m0, mn1 = up1 ? mx1 : m1;
          // a column that keeps its m may still hold -inf there (it has seen nothing yet): factor 1
          const float al0 = up0 ? fast_exp2(m0 - mn0) : 1.f, al1 = up1 ? fast_exp2(m1 - mn1) : 1.f;
          l0 *= al0;
          l1 *= al1;
#pragma unroll
          for (int mt = 0; mt < KT; ++mt) {
            acc[mt][0] *= al0;
            acc[mt][1] *= al1;
            acc[mt][2] *= al0;
            acc[mt][3] *= al1;
          }
          m0 = mn0;
          m1 = mn1;
        }
        // a column that has seen no token yet keeps m = -inf (all its x are -inf): exponentiate against 0
        const float ms0 = m0 == -INFINITY ? 0.f : m0, ms1 = m1 == -INFINITY ? 0.f : m1;
        const uint32_t pa = Elem<T>::pack2(fast_exp2(x00 - ms0), fast_exp2(x01 - ms1));
        const uint32_t pb = Elem<T>::pack2(fast_exp2(x10 - ms0), fast_exp2(x11 - ms1));
        const float2 fa = Elem<T>::to_float2(pa), fb = Elem<T>::to_float2(pb);
        // l: this lane's rows only (the weights PV multiplies); finish() adds the lanes of a column
        l0 += fa.x + fb.x;
        l1 += fa.y + fb.y;
        // P^T as the B operand of the PV MMA: transpose the 8x8 score fragments
        const uint32_t b0 = movmatrix_trans(pa), b1 = movmatrix_trans(pb);
        {
          const int tr = r8 + ((mi >> 1) << 3);  // stored V rows 0..15
          const int t = BS >= 16 ? c * 16 + tr : (tr & (BS - 1));
#pragma unroll
          for (int mt = 0; mt < KT; ++mt) {
            uint32_t a[4];
            ldmatrix_x4_trans(a, Vs + swz_offset<BS, NBOX>(t, mt * 2 + (mi & 1)));
            Mma<T>::run(acc[mt], a, b0, b1);
          }
        }
      }
    }
  }
};

template <typename T_, int D_, int BS_>
struct ScoredTileE4M3 : MmaTileE4M3<T_, D_, BS_> {
  using Base = MmaTileE4M3<T_, D_, BS_>;
  using T = T_;
  using QB = typename Base::QB;
  static constexpr int D = D_, BS = BS_, CH = Base::CH, KT = Base::KT;
  static __device__ __forceinline__ int off(int t, int c) { return Base::off(t, c); }

  template <typename Rule>
  static __device__ __forceinline__ void fold(unsigned char* Ks, unsigned char* Vs, int first, int nvalid,
                                              const QB& qb, int lane, float& m0, float& m1, float& l0, float& l1,
                                              float (&acc)[KT][4], const Rule& rule) {
    const int g = lane >> 2, qd = lane & 3;
    if (nvalid < BS) {
      // value rows past the context may hold anything (NaN codes too): zero them
      // so that their zero weights contribute exactly zero
      const int nz = (BS - nvalid) * 8;
      for (int idx = lane; idx < nz; idx += 32)
        *reinterpret_cast<uint4*>(Vs + (nvalid + idx / 8) * 128 + (idx % 8) * 16) = make_uint4(0u, 0u, 0u, 0u);
      __syncwarp();
    }
    if (first > 0) {
      for (int idx = lane; idx < first * 8; idx += 32)
        *reinterpret_cast<uint4*>(Vs + (idx / 8) * 128 + (idx % 8) * 16) = make_uint4(0u, 0u, 0u, 0u);
      __syncwarp();
    }
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      if (c * 16 < nvalid && c * 16 + 16 > first) {
        // K rows of this lane: c*16 + g and + 8 (with BS = 8 the second aliases the first; masked)
        const int ta = c * 16 + g, tb = BS >= 16 ? ta + 8 : ta;
        const uint4 ka0 = *reinterpret_cast<const uint4*>(Ks + off(ta, 2 * qd));
        const uint4 ka1 = *reinterpret_cast<const uint4*>(Ks + off(ta, 2 * qd + 1));
        const uint4 kb0 = *reinterpret_cast<const uint4*>(Ks + off(tb, 2 * qd));
        const uint4 kb1 = *reinterpret_cast<const uint4*>(Ks + off(tb, 2 * qd + 1));
        const uint32_t wa[8] = {ka0.x, ka0.y, ka0.z, ka0.w, ka1.x, ka1.y, ka1.z, ka1.w};
        const uint32_t wb[8] = {kb0.x, kb0.y, kb0.z, kb0.w, kb1.x, kb1.y, kb1.z, kb1.w};
        float sacc[4] = {0.f, 0.f, 0.f, 0.f}, sacc2[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < KT; ++j) {
          uint32_t a[4];  // rows g, g + 8 at positions 2qd.. (dims +0, +1) and 2qd+8.. (dims +2, +3)
          e4m3x4_to_f16x2(wa[j], a[0], a[2]);
          e4m3x4_to_f16x2(wb[j], a[1], a[3]);
          if (j & 1) {
            Mma<__half>::run(sacc2, a, qb[j][0], qb[j][1]);
          } else {
            Mma<__half>::run(sacc, a, qb[j][0], qb[j][1]);
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) sacc[e] += sacc2[e];
        const bool va = ta < nvalid && ta >= first;
        const bool vb = BS >= 16 && ta + 8 < nvalid && ta + 8 >= first;
        rule(sacc, ta, va, ta + 8, vb);
        const float x00 = sacc[0], x01 = sacc[1], x10 = sacc[2], x11 = sacc[3];
        // Lazy rescaling: a column's reference m moves (and its state is rescaled)
        // only when a score exceeds it by more than 8, so p = 2^(x - m) <= 2^8. Each
        // lane tests its own scores and the warp votes; the max is reduced across
        // the lanes only when some score does exceed.
        float mx0 = fmaxf(x00, x10), mx1 = fmaxf(x01, x11);
        if (__any_sync(kFull, mx0 > m0 + 8.f || mx1 > m1 + 8.f)) {
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) {
            mx0 = fmaxf(mx0, __shfl_xor_sync(kFull, mx0, o));
            mx1 = fmaxf(mx1, __shfl_xor_sync(kFull, mx1, o));
          }
          const bool up0 = mx0 > m0 + 8.f, up1 = mx1 > m1 + 8.f;
          const float mn0 = up0 ? mx0 : m0, mn1 = up1 ? mx1 : m1;
          float al0 = fast_exp2(m0 - mn0), al1 = fast_exp2(m1 - mn1);
          {  // a column that keeps its m may still hold -inf there
            if (!up0) al0 = 1.f;
            if (!up1) al1 = 1.f;
          }
          l0 *= al0;
          l1 *= al1;
#pragma unroll
          for (int mt = 0; mt < KT; ++mt) {
            acc[mt][0] *= al0;
            acc[mt][1] *= al1;
            acc[mt][2] *= al0;
            acc[mt][3] *= al1;
          }
          m0 = mn0;
          m1 = mn1;
        }
        float r0 = m0, r1 = m1;  // exponentials against the reference
        {  // a column that has seen nothing yet: against 0 (its x are all -inf)
          if (r0 == -INFINITY) r0 = 0.f;
          if (r1 == -INFINITY) r1 = 0.f;
        }
        const uint32_t pa = Elem<__half>::pack2(fast_exp2(x00 - r0), fast_exp2(x01 - r1));
        const uint32_t pb = Elem<__half>::pack2(fast_exp2(x10 - r0), fast_exp2(x11 - r1));
        const float2 fa = Elem<__half>::to_float2(pa), fb = Elem<__half>::to_float2(pb);
        // l: this lane's rows only; finish() adds the lanes of a column
        l0 += fa.x + fb.x;
        l1 += fa.y + fb.y;
        // P^T as the B operand of the PV MMA: transpose the 8x8 score fragments
        const uint32_t b0 = movmatrix_trans(pa), b1 = movmatrix_trans(pb);
        // V: chunk g (dims 16g .. 16g+15) of token rows 2qd, 2qd+1, 2qd+8, 2qd+9
        // (with BS = 8 the last two alias the first two; their weights are zero)
        const int v0 = c * 16 + 2 * qd, v8 = BS >= 16 ? v0 + 8 : v0;
        const uint4 X0 = *reinterpret_cast<const uint4*>(Vs + off(v0, g));
        const uint4 X1 = *reinterpret_cast<const uint4*>(Vs + off(v0 + 1, g));
        const uint4 X8 = *reinterpret_cast<const uint4*>(Vs + off(v8, g));
        const uint4 X9 = *reinterpret_cast<const uint4*>(Vs + off(v8 + 1, g));
        const uint32_t x0[4] = {X0.x, X0.y, X0.z, X0.w}, x1[4] = {X1.x, X1.y, X1.z, X1.w};
        const uint32_t x8[4] = {X8.x, X8.y, X8.z, X8.w}, x9[4] = {X9.x, X9.y, X9.z, X9.w};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          // byte b of word w is dim 16g + 4w + b. For the token rows (r, r'):
          // lo = [r.b0, r'.b0, r.b1, r'.b1] and hi = [r.b2, r'.b2, r.b3, r'.b3], so
          // each 16-bit half pairs the two rows at one dim
          const uint32_t lo01 = prmt(x0[w], x1[w], 0x5140), hi01 = prmt(x0[w], x1[w], 0x7362);
          const uint32_t lo89 = prmt(x8[w], x9[w], 0x5140), hi89 = prmt(x8[w], x9[w], 0x7362);
          // m-tile 2w: dims 16g + 4w (row g) and + 1 (row g + 8); m-tile 2w + 1: + 2 and + 3
          uint32_t ae[4], ao[4];
          e4m3x4_to_f16x2(lo01, ae[0], ae[1]);
          e4m3x4_to_f16x2(lo89, ae[2], ae[3]);
          e4m3x4_to_f16x2(hi01, ao[0], ao[1]);
          e4m3x4_to_f16x2(hi89, ao[2], ao[3]);
          Mma<__half>::run(acc[2 * w], ae, b0, b1);
          Mma<__half>::run(acc[2 * w + 1], ao, b0, b1);
        }
      }
    }
  }
};

}  // namespace pkv
