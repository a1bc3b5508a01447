// Scored paged attention with many rows per kv head, on the fifth-generation tensor cores (tcgen05).
//
// One CTA per SM takes up to 256 (query token, head) rows of a (partition, kv head, sequence) -- row r is query
// token r / G, head kvh * G + r % G -- and walks the keys that any of them sees in tiles of 128 tokens
// (128 / block_size pool blocks). Its two streams of 128 rows each compute, tile by tile,
//   S = Q . K^T        M 128, N 64, K = head_dim       -> tensor memory (fp32)
//   P = exp2(score(S) - m)   one thread per row, 16-bit, over S's columns
//   O += P . V         M 128, N = head_dim, K 64       A from tensor memory
// in halves of 64 keys, each half with its own columns for S and P: while the threads work on one half, the
// other's PV and then its next S run. (With whole tiles, S, P and PV of a stream ran one after the other:
// a causal prompt of 8192 tokens, 32/8 heads, took 562 us against 485, with cap 50 675 against 556.)
// The streams share every K and V tile (read once per 256 rows), and one's products run while the other's
// threads exponentiate. A CTA with at most 128 rows gives both streams the same rows: stream w then takes every
// second tile, and their (m, l, O) are merged at the end.
//
// What bounds it: per 256 x 128 scores the tensor cores need about 2048 cycles (head_dim 128) and the shared
// memory port as many (Q and K twice, V twice, the copies once); the exponentials take 1 special-function
// operation a score and the scores 4 to 8 fp32 operations (cap), which is of the same size. So the streams
// overlap the two, and a score is kept to few instructions: tiles that every row sees whole skip the masks,
// and the tanh is a polynomial where the tile's scores stay well below the cap.
//
// Warps: 0-3 and 4-7 the streams' rows; 8 and 9 issue a stream's MMAs (one thread each); 10 and 11 copy the
// blocks of K and V tiles, half of each tile a warp (a copy takes about 100 cycles to issue), into a ring of
// tile slots in the order K0 V0 K1 V1 ...; FP8 pool: 12-15 widen a tile's codes to f16 in place.
// Every wait is bounded: a copy or MMA that does not complete makes the CTA stop, set PKV_DEVERR_TIMEOUT and
// write zeros.
#pragma once

#include <type_traits>

#include "pkv_mq_tc.cuh"
#include "pkv_scored.cuh"

namespace pkv {

// Pairs of fp32 values in one 64-bit register pair: one instruction for two operations.
using f32x2 = unsigned long long;
__device__ __forceinline__ f32x2 pair2(float lo, float hi) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpair2(f32x2 v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// The largest of 64 values held as pairs, and of their negatives (four chains of three-way maxima).
__device__ __forceinline__ float max64(const f32x2 (&x)[32]) {
  float m[4], a, b;
#pragma unroll
  for (int u = 0; u < 32; ++u) {
    unpair2(x[u], a, b);
    m[u & 3] = u < 4 ? fmaxf(a, b) : max3(m[u & 3], a, b);
  }
  return max3(fmaxf(m[0], m[1]), m[2], m[3]);
}
__device__ __forceinline__ float max64neg(const f32x2 (&x)[32]) {
  float m[4], a, b;
#pragma unroll
  for (int u = 0; u < 32; ++u) {
    unpair2(x[u], a, b);
    m[u & 3] = u < 4 ? fmaxf(-a, -b) : max3(m[u & 3], -a, -b);
  }
  return max3(fmaxf(m[0], m[1]), m[2], m[3]);
}

// The 64 weights 2^e(u) (pairs) in 16 bits into pw; returns the sum of the fp32 weights before that rounding,
// which moves the result by at most the rounding unit times the row's largest |v|.
template <typename TP, typename E>
__device__ __forceinline__ float weights64(uint32_t (&pw)[32], E e) {
  f32x2 ls[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
  for (int u = 0; u < 32; ++u) {
    float a, b;
    unpair2(e(u), a, b);
    a = fast_exp2(a);
    b = fast_exp2(b);
    pw[u] = Elem<TP>::pack2(a, b);
    ls[u & 3] = add2(ls[u & 3], pair2(a, b));
  }
  float a, b;
  unpair2(add2(add2(ls[0], ls[1]), add2(ls[2], ls[3])), a, b);
  return a + b;
}

template <typename T, int D, int BS, bool F8>
struct ScoredTcShape {
  static constexpr int ROWS = 128;           // rows per stream (M)
  static constexpr int NT = 128;             // tokens per tile
  static constexpr int NBT = NT / BS;        // pool blocks per tile
  static constexpr int DH = D / 64;          // 128-byte halves of a 16-bit row
  static constexpr int ATOM = DH * 1024;     // 8 tokens: their columns 0..63, then 64..127
  static constexpr int TILE = NT / 8 * ATOM; // bytes of a K or V tile slot
  static constexpr int QT = DH * ROWS * 128; // bytes of a stream's Q
  static constexpr int NS = D == 128 ? 5 : 8;  // tile slots
  static constexpr int HALF = TILE / 2;      // FP8 pool: a tile's codes land in its slot's upper half
  static constexpr int OFF_RING = 2 * QT;
  static constexpr int OFF_BARS = OFF_RING + NS * TILE;
  // barriers: full[8], empty[8], raw[8] per slot; per stream q_full, fin; per stream and half s_full, p_full, pv_done
  static constexpr int NBARS = 24 + 16;
  static constexpr int OFF_MISC = OFF_BARS + NBARS * 8;  // tensor-memory base, abort flag, key range, row state
  static constexpr int OFF_ML = OFF_MISC + 16;           // stream 1's (m, l) in a CTA of shared rows
  static constexpr int SMEM = OFF_ML + 2 * ROWS * 4;
  static constexpr int S_COL = 0, O_COL = 256;  // tensor memory: stream w's S at 128 w, its O at 256 + 128 w
  static constexpr int TMEM_COLS = 512;
  static constexpr int MMA_WARP = 8, COPY_WARP = 10, WIDEN_WARP = 12;
  static constexpr int THREADS = (F8 ? 16 : 12) * 32;
  static_assert(SMEM <= 232448 - 1024, "one CTA's shared memory");
  static_assert(NBT >= 4 && NBT <= 16, "blocks per tile");
  static_assert(!F8 || D == 128, "an FP8 pool: head_dim 128");
  static_assert(2 * ROWS * D * 2 <= NS * TILE, "the merge of the streams stages one O in the ring");
};

// Whether every thread of the four widening warps says yes.
__device__ __forceinline__ bool widen_agree(bool yes) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.and.pred q, 1, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(yes ? 1u : 0u)
      : "memory");
  return r != 0;
}

// x -= slope |d0 - t| for the half's 64 keys t.
__device__ __forceinline__ void add_bias(f32x2 (&x)[32], float slope, int d0) {
  const float d = (float)d0;
#pragma unroll
  for (int u = 0; u < 32; ++u) {
    float a, b;
    unpair2(x[u], a, b);
    x[u] = pair2(fmaf(-slope, fabsf(d - (float)(2 * u)), a), fmaf(-slope, fabsf(d - (float)(2 * u + 1)), b));
  }
}

// FP8 pool: a widening warp's 32 tokens (4 atoms) of a tile. The whole tile is read into registers (all four
// warps, then a barrier) before anything is written, because the f16 atoms overwrite the codes. Lane (t = lane
// / 4, q = lane % 4) takes codes 32 q .. of token 8 a + t; the orders keep 8-lane phases on distinct banks.
__device__ __forceinline__ void scored_widen(unsigned char* slot, int half, int w, int lane) {
  const unsigned char* src = slot + half + w * 32 * 128;
  const int t8 = lane >> 2, q = lane & 3;
  const int h0 = (t8 & 1) * 16, h1 = 16 - h0;
  uint4 c[4][2];
#pragma unroll
  for (int a = 0; a < 4; ++a) {
    const unsigned char* row = src + (8 * a + t8) * 128 + 32 * q;
    const uint4 x = *reinterpret_cast<const uint4*>(row + h0);
    const uint4 y = *reinterpret_cast<const uint4*>(row + h1);
    c[a][0] = h0 ? y : x;
    c[a][1] = h0 ? x : y;
  }
  asm volatile("bar.sync 1, 128;" ::: "memory");  // the four widening warps
#pragma unroll
  for (int a = 0; a < 4; ++a) {
    const uint32_t x[8] = {c[a][0].x, c[a][0].y, c[a][0].z, c[a][0].w, c[a][1].x, c[a][1].y, c[a][1].z, c[a][1].w};
    unsigned char* row = slot + (4 * w + a) * 2048 + (q >> 1) * 1024 + t8 * 128;
    const bool rot = (q >> 1) != 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int kk = rot ? (k ^ 2) : k;
      uint32_t h[4];
      e4m3x4_to_f16x2(rot ? x[2 * (k ^ 2)] : x[2 * k], h[0], h[1]);
      e4m3x4_to_f16x2(rot ? x[2 * (k ^ 2) + 1] : x[2 * k + 1], h[2], h[3]);
      *reinterpret_cast<uint4*>(row + ((((q & 1) * 4 + kk) ^ t8) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
    }
  }
}

template <typename T, int D, int BS, bool F8, bool CAP, bool BIAS>
__global__ void __launch_bounds__(F8 ? 512 : 384, 1)
    pkv_scored_tc_kernel(const __grid_constant__ DecodeParams p, const __grid_constant__ ScoreParams sc,
                         const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
  pdl_begin();
  using Sh = ScoredTcShape<T, D, BS, F8>;
  using TP = typename std::conditional<F8, __half, T>::type;  // the MMAs' type
  using C = typename std::conditional<F8, __nv_fp8_e4m3, T>::type;  // the cache's
  constexpr int NT = Sh::NT, NBT = Sh::NBT, NS = Sh::NS, ROWS = Sh::ROWS;
  extern __shared__ __align__(1024) unsigned char smem[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Sh::OFF_BARS);
  uint64_t *full = bars, *empty = bars + 8, *raw = bars + 16;
  uint64_t* q_full = bars + 24;   // [stream]
  uint64_t* fin = bars + 26;      // [stream]: everything issued
  uint64_t* s_full = bars + 28;   // [stream][half]
  uint64_t* p_full = bars + 32;   // [stream][half]
  uint64_t* pv_done = bars + 36;  // [stream][half]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Sh::OFF_MISC);
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* range = reinterpret_cast<int*>(tmem_slot + 2);  // first visible key, end of the visible keys
  auto slot = [&](int it) { return smem + Sh::OFF_RING + (it % NS) * Sh::TILE; };

  // the last row tiles first: with a causal limit they see the most keys
  const int part = blockIdx.x / sc.row_tiles, rt = sc.row_tiles - 1 - (int)blockIdx.x % sc.row_tiles;
  const int kvh = blockIdx.y;
  const int s = sc.order ? sc.order[blockIdx.z] : (int)blockIdx.z;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = p.group, P = p.partition_size;
  const bool reporter = blockIdx.x == 0 && kvh == 0 && threadIdx.x == 0;
  if (smem_u32(smem) & 1023u) {  // not expected on any supported GPU; nothing is written
    if (threadIdx.x == 0) atomicOr(p.err, PKV_DEVERR_LAYOUT);
    return;
  }
  const int ctx = clamp_context(p, s, reporter);
  int q0 = 0;
  const int q_len = scored_query_len(sc, s, ctx, q0);
  if (q_len < 0) {
    if (reporter) atomicOr(p.err, PKV_DEVERR_QUERY);
    return;
  }
  const long long R = (long long)q_len * G, row0 = (long long)rt * 2 * ROWS;
  if (row0 >= R) return;
  const int nrows = (int)min((long long)2 * ROWS, R - row0);
  const bool shared_rows = nrows <= ROWS;  // both streams take the same rows
  const int base = scored_base(sc, ctx, q_len, BS);
  const int tok0 = base + part * P;

  // the streams' rows: warps 0-7, thread row = its tensor-memory lane
  const int w = warp >> 2;  // (stream, for warps 0-7)
  const int row = 32 * (warp & 3) + lane;
  const int rr = (shared_rows ? 0 : w * ROWS) + row;  // row within the CTA
  const bool active = warp < 8 && rr < nrows;
  const int ti = active ? (int)((row0 + rr) / G) : 0;  // query token within the sequence
  const int h = kvh * G + (active ? (int)((row0 + rr) % G) : 0);
  const int pos = ctx - q_len + ti;
  int lo = 0, hi = 0;
  if (active) scored_span(sc, q0 + ti, pos, ctx, lo, hi);
  const RowParts parts = row_parts(lo, hi, base, P);

  // the CTA's keys: from its rows' first to their last visible one, within the partition
  int c0, c1;
  if (!sc.key_begin && !sc.key_end) {  // the first row's first, the last row's last
    int unused;
    scored_span(sc, 0, ctx - q_len + (int)(row0 / G), ctx, c0, unused);
    scored_span(sc, 0, ctx - q_len + (int)((row0 + nrows - 1) / G), ctx, unused, c1);
  } else {
    if (threadIdx.x == 0) {
      range[0] = INT32_MAX;
      range[1] = 0;
    }
    __syncthreads();
    if (warp < 8) {
      int a = hi > lo ? lo : INT32_MAX, b = hi > lo ? hi : 0;
      a = __reduce_min_sync(kFull, a);
      b = __reduce_max_sync(kFull, b);
      if (lane == 0) {
        atomicMin(range, a);
        atomicMax(range + 1, b);
      }
    }
    __syncthreads();
    c0 = range[0];
    c1 = range[1];
  }
  c0 = max(c0, tok0);
  c1 = min(c1, tok0 + P);
  T* out_row = static_cast<T*>(p.out) + ((size_t)(q0 + ti) * p.num_heads + h) * D;
  if (c1 <= c0) {  // no key: partition 0 writes the zeros of rows that see nothing
    if (part == 0 && active && parts.last < parts.first)
      for (int d = 0; d < D; d += 8) *reinterpret_cast<uint4*>(out_row + d) = make_uint4(0u, 0u, 0u, 0u);
    return;
  }
  const int blk0 = c0 / BS, nblk = (c1 + BS - 1) / BS - blk0;
  const int ntile = (nblk + NBT - 1) / NBT;
  const int32_t* table = p.block_tables + (size_t)s * p.max_blocks_per_seq + blk0;
  const int step = shared_rows ? 2 : 1;                  // a stream's tiles: first, first + step, ...
  auto first_tile = [&](int stream) { return shared_rows ? stream : 0; };

  if (threadIdx.x == 0) {
    prefetch_tensormap(&kmap);
    prefetch_tensormap(&vmap);
    for (int k = 0; k < NS; ++k) {
      mbar_init(full + k, F8 ? 4 : 2);
      mbar_init(empty + k, shared_rows ? 1 : 2);
      mbar_init(raw + k, 2);
    }
    for (int k = 0; k < 2; ++k) {
      mbar_init(q_full + k, ROWS);
      mbar_init(fin + k, 1);
      for (int hf = 0; hf < 2; ++hf) {
        mbar_init(s_full + 2 * k + hf, 1);
        mbar_init(p_full + 2 * k + hf, ROWS);
        mbar_init(pv_done + 2 * k + hf, 1);
      }
    }
    fence_mbar_init();
    *abort = 0;
  }
  if (warp == Sh::MMA_WARP) tc::alloc(tmem_slot, Sh::TMEM_COLS);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tbase = *tmem_slot;

  if (warp == Sh::COPY_WARP || warp == Sh::COPY_WARP + 1) {
    // ---- copies: this warp's half of the blocks of item it = 2 j (K tile j) and 2 j + 1 (V tile j)
    constexpr int NH = NBT / 2;
    const int at = (warp - Sh::COPY_WARP) * NH + (lane & (NH - 1));  // lane < NH: block of the tile
    uint64_t* landed = F8 ? raw : full;
    auto load_id = [&](int j) { return lane < NH && j * NBT + at < nblk ? table[j * NBT + at] : -1; };
    int next = load_id(0);
    int it = 0;
    bool ok = true;
    for (int j = 0; ok && j < ntile; ++j) {
      int id = next;
      if (j + 1 < ntile) next = load_id(j + 1);
      if (lane < NH && j * NBT + at < nblk && (unsigned)id >= (unsigned)p.num_blocks) {
        atomicOr(p.err, PKV_DEVERR_BLOCK_ID);
        id = -1;
      }
      const int n = __popc(__ballot_sync(kFull, id >= 0));
      const int y = (id * p.num_kv_heads + kvh) * BS;  // first pool row of the block
#pragma unroll
      for (int kv = 0; kv < 2; ++kv, ++it) {
        uint64_t* bar = landed + it % NS;
        if (it >= NS) ok = __all_sync(kFull, tc_wait(empty + it % NS, (it / NS - 1) & 1, abort));
        if (!ok) break;
        if (lane == 0) {
          fence_proxy_async_smem();  // generic stores into the slot (zeroed rows, widened codes): before the copies
          mbar_arrive_expect_tx(bar, n * BS * (F8 ? 128 : D * 2));
        }
        __syncwarp();
        if (id >= 0) {
          if constexpr (F8)
            tma_load_2d(slot(it) + Sh::HALF + at * BS * 128, kv ? &vmap : &kmap, 0, y, bar);
          else if constexpr (Sh::DH == 2)
            tma_load_4d(slot(it) + at * (BS / 8) * Sh::ATOM, kv ? &vmap : &kmap, 0, 0, 0, y / 8, bar);
          else
            tma_load_2d(slot(it) + at * (BS / 8) * Sh::ATOM, kv ? &vmap : &kmap, 0, y, bar);
        }
      }
    }
    // no copy may still be landing when the CTA leaves
    if (lane == 0)
      for (int k = it > NS ? it - NS : 0; k < it; ++k) mbar_wait(landed + k % NS, (k / NS) & 1);
  } else if (F8 && warp >= Sh::WIDEN_WARP) {
    // ---- FP8 pool: widen each item's codes once they have landed
    for (int it = 0; it < 2 * ntile; ++it) {
      // (agreed among the four warps, which meet at barriers: all go on, or all leave)
      if (!widen_agree(tc_wait(raw + it % NS, (it / NS) & 1, abort))) break;
      if constexpr (F8) scored_widen(slot(it), Sh::HALF, warp - Sh::WIDEN_WARP, lane);
      fence_proxy_async_smem();  // generic stores, read by the MMAs
      __syncwarp();
      if (lane == 0) mbar_arrive(full + it % NS);
    }
  } else if (warp == Sh::MMA_WARP || warp == Sh::MMA_WARP + 1) {
    // ---- MMA issue: one thread per stream, in the order S S | PV S | PV S | ... by halves of a tile
    if (lane == 0) {
      const int st = warp - Sh::MMA_WARP;
      constexpr bool BF = std::is_same<TP, __nv_bfloat16>::value;
      constexpr uint32_t IDESC_S = tc::idesc_f16(BF, ROWS, NT / 2, false, false);
      constexpr uint32_t IDESC_O = tc::idesc_f16(BF, ROWS, D, false, true);
      const uint32_t q_addr = smem_u32(smem) + (shared_rows ? 0 : st * Sh::QT);
      const uint32_t scol = tbase + Sh::S_COL + st * NT, ocol = tbase + Sh::O_COL + st * 128;
      // S of tile j's half hf (64 keys: 8 atoms of K) into that half's columns, which the caller knows are free
      auto issue_s = [&](int j, int hf) {
        const int ik = 2 * j;
        if (hf == 0 && !tc_wait(full + ik % NS, (ik / NS) & 1, abort)) return false;
        tc::fence_after_sync();
        const uint32_t k_addr = smem_u32(slot(ik)) + hf * 8 * Sh::ATOM;
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          tc::mma_f16(scol + hf * 64, tc::desc_sw128(q_addr + (k / 4) * (ROWS * 128) + (k % 4) * 32, 16, 1024),
                      tc::desc_sw128(k_addr + (k / 4) * 1024 + (k % 4) * 32, 16, Sh::ATOM), IDESC_S, k > 0);
        tc::commit(s_full + 2 * st + hf);
        if (hf) tc::commit(empty + ik % NS);
        return true;
      };
      bool ok = shared_rows ? tc_wait(q_full, 0, abort) && tc_wait(q_full + 1, 0, abort) : tc_wait(q_full + st, 0, abort);
      int j = first_tile(st), n = 0;
      if (j < ntile) ok = ok && issue_s(j, 0) && issue_s(j, 1);
      for (; ok && j < ntile; j += step, ++n) {
        const int iv = 2 * j + 1;
        const uint32_t v_addr = smem_u32(slot(iv));
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          ok = ok && tc_wait(p_full + 2 * st + hf, n & 1, abort) &&
               (hf > 0 || tc_wait(full + iv % NS, (iv / NS) & 1, abort));
          if (!ok) break;
          tc::fence_after_sync();
#pragma unroll
          for (int k = 0; k < 4; ++k)  // 16 keys each: 8 columns of P, two atoms of V
            tc::mma_f16_ta(ocol, scol + hf * 64 + k * 8,
                           tc::desc_sw128(v_addr + (hf * 4 + k) * 2 * Sh::ATOM, 1024, Sh::ATOM), IDESC_O,
                           n > 0 || hf > 0 || k > 0);
          tc::commit(pv_done + 2 * st + hf);
          if (hf) tc::commit(empty + iv % NS);
          // the next tile's S goes where this half's P is: not before its PV has read it
          if (j + step < ntile) ok = tc_wait(pv_done + 2 * st + hf, n & 1, abort) && issue_s(j + step, hf);
        }
      }
      tc::commit(fin + st);  // every MMA issued above has completed once this arrives
      mbar_wait(fin + st, 0);
    }
    __syncwarp();
  } else if (warp < 8) {
    // ---- rows
    float qscale = 1.f;  // FP8 pool, bf16 query: the 2^-k the row was scaled by
    unsigned char* Qs = smem + (shared_rows ? 0 : w * Sh::QT);
    // (row tile rt of 256 rows: stream w's rows are tile 2 rt + w of 128 rows)
    const int rt128 = 2 * rt + (shared_rows ? 0 : w);
    if constexpr (F8 && std::is_same<T, __nv_bfloat16>::value) {
      // (in a CTA of shared rows both streams need the factor; both store the same Q)
      qscale = mq_tc_fetch_q_bf16_as_f16<D, ROWS>(Qs, row, reinterpret_cast<const __nv_bfloat16*>(p.query), q0, kvh,
                                                  rt128, q_len, G, p.num_heads);
    } else if (!shared_rows || w == 0) {
      mq_tc_fetch_q<T, D, ROWS>(Qs, row, reinterpret_cast<const T*>(p.query), q0, kvh, rt128, q_len, G, p.num_heads);
      cp_async_wait_all();
    }
    fence_proxy_async_smem();  // generic-proxy writes, read by the S MMAs
    mbar_arrive(q_full + w);
    const float sl2 = p.scale_log2 * qscale;
    const float cap_in = sc.cap_in * qscale, cap_out = sc.cap_out;
    const float slope = BIAS ? sc.slopes[h] * 1.4426950408889634f : 0.f;
    // cap_out * tanh(x * cap_in) = x (c0 + c1 x^2 + c2 x^4 + c3 x^6) while |x * cap_in| <= 1/2: a minimax fit of
    // tanh(z) / z in z^2 on [0, 1/4], relative error 6e-7. (Not for factors whose powers leave fp32's range.)
    f32x2 cc[4];
    float near2 = -1.f;  // the largest x^2 that it is for
    {
      const float z2 = cap_in * cap_in;
      float c = cap_out * cap_in;
      const float fit[4] = {0.999999456f, -0.333263179f, 0.131902965f, -0.0444022226f};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        cc[k] = pair2(c * fit[k], c * fit[k]);
        c *= z2;
      }
      if (z2 < 1e6f && z2 > 1e-18f) near2 = 0.25f / z2;
    }
    const int t_first = blk0 * BS;
    const uint32_t scol = tc::taddr(tbase, 32 * (warp & 3), Sh::S_COL + w * NT);
    const uint32_t ocol = tc::taddr(tbase, 32 * (warp & 3), Sh::O_COL + w * 128);
    // which blocks of a tile were copied: lane b < NBT holds block b's test (the copying warps' own)
    auto load_ok = [&](int j) {
      const int b = j * NBT + (lane & (NBT - 1));
      return b < nblk ? (unsigned)table[b] < (unsigned)p.num_blocks : false;
    };
    constexpr uint32_t all = NBT == 32 ? 0xffffffffu : (1u << NBT) - 1u;
    float m_ref = -INFINITY, l = 0.f;
    bool ok = true;
    int n = 0;
    bool next = first_tile(w) < ntile && load_ok(first_tile(w));
    for (int j = first_tile(w); j < ntile; j += step, ++n) {
      const uint32_t blocks = __ballot_sync(kFull, next) & all;
      if (j + step < ntile) next = load_ok(j + step);
      const int tb = t_first + j * NT;  // position of the tile's first token
      const bool edge = blocks != all || tb < c0 || tb + NT > c1;  // V rows outside the CTA's keys, or not copied
#pragma unroll 1
      for (int hf = 0; hf < 2; ++hf) {
        const int th = tb + hf * 64;
        // (tensor-memory accesses are warp-wide: a warp leaves the loop as a whole)
        ok = __all_sync(kFull, tc_wait(s_full + 2 * w + hf, n & 1, abort));
        if (!ok) break;
        tc::fence_after_sync();
        uint32_t sr[2][32];
        tc::ld32(scol + hf * 64, sr[0]);
        tc::ld32(scol + hf * 64 + 32, sr[1]);
        tc::wait_ld();
        f32x2 x[32];  // keys 2 u and 2 u + 1 of the half
#pragma unroll
        for (int u = 0; u < 32; ++u)
          x[u] = pair2(__uint_as_float(sr[u >> 4][(2 * u) & 31]), __uint_as_float(sr[u >> 4][(2 * u + 1) & 31]));
        const bool whole = !edge && th >= lo && th + 64 <= hi;
        float f = 1.f;      // factor of what the row holds
        bool resc = false;  // O's row holds terms to rescale
        // The reference m moves, and the row is rescaled, only when a score exceeds it by more than 8, so
        // weights are at most 2^8. A row that has seen nothing yet exponentiates against 0 (its scores are
        // -inf, or NaN, which must stay).
        auto reference = [&](float mx) {
          const bool move = mx > m_ref + 8.f;
          resc = move && m_ref != -INFINITY;
          f = resc ? fast_exp2(m_ref - mx) : 1.f;
          if (move) m_ref = mx;
          return m_ref == -INFINITY ? 0.f : -m_ref;
        };
        uint32_t pw[32];  // P row as 16-bit pairs
        float lsum;       // its sum
        bool near = false;
        float top = 0.f;
        if constexpr (CAP) {
          top = max64(x);
          const float bottom = -max64neg(x);
          near = __all_sync(kFull, fmaxf(top * top, bottom * bottom) <= near2);  // the warp's scores: at most half the cap
          if (cap_in < 0.f) top = bottom;
        }
        if (!BIAS && __all_sync(kFull, whole) && (CAP ? near : sl2 >= 0.f)) {
          if constexpr (CAP) {
            const f32x2 t = pair2(top, top), t2 = mul2(t, t);
            float mx, unused;
            unpair2(mul2(t, fma2(t2, fma2(t2, fma2(t2, cc[3], cc[2]), cc[1]), cc[0])), mx, unused);
            const float nm = reference(mx);
            const f32x2 sub = pair2(nm, nm);
            lsum = weights64<TP>(pw, [&](int u) {
              const f32x2 sq = mul2(x[u], x[u]);
              return fma2(x[u], fma2(sq, fma2(sq, fma2(sq, cc[3], cc[2]), cc[1]), cc[0]), sub);
            });
          } else {
            const float nm = reference(max64(x) * sl2);
            const f32x2 mul = pair2(sl2, sl2), sub = pair2(nm, nm);
            lsum = weights64<TP>(pw, [&](int u) { return fma2(x[u], mul, sub); });
          }
        } else {
          if constexpr (CAP) {
            if (near) {
#pragma unroll
              for (int u = 0; u < 32; ++u) {
                const f32x2 sq = mul2(x[u], x[u]);
                x[u] = mul2(x[u], fma2(sq, fma2(sq, fma2(sq, cc[3], cc[2]), cc[1]), cc[0]));
              }
            } else {
#pragma unroll
              for (int u = 0; u < 32; ++u) {
                float v0, v1;
                unpair2(x[u], v0, v1);
                x[u] = pair2(cap_out * score_tanh(v0 * cap_in), cap_out * score_tanh(v1 * cap_in));
              }
            }
            if constexpr (BIAS) add_bias(x, slope, pos - th);
          } else if (BIAS && __all_sync(kFull, pos >= th + 63)) {
            // keys up to the token's own position: -slope (p - j) is linear in j, four chains of steps of 8
            const f32x2 mul = pair2(sl2, sl2), step8 = pair2(8.f * slope, 8.f * slope);
            const float d = (float)(th - pos);
            f32x2 bias[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) bias[k] = pair2(slope * (d + 2 * k), slope * (d + 2 * k + 1));
#pragma unroll
            for (int u = 0; u < 32; ++u) {
              x[u] = fma2(x[u], mul, bias[u & 3]);
              if (u < 28) bias[u & 3] = add2(bias[u & 3], step8);
            }
          } else {
            const f32x2 mul = pair2(sl2, sl2);
#pragma unroll
            for (int u = 0; u < 32; ++u) x[u] = mul2(x[u], mul);
            if constexpr (BIAS) add_bias(x, slope, pos - th);
          }
          if (!whole) {
            const uint32_t hb = blocks >> (hf * (NBT / 2));
            const int a = lo - th;
            const unsigned len = (unsigned)(hi - lo);
#pragma unroll
            for (int u = 0; u < 32; ++u) {
              float v0, v1;
              unpair2(x[u], v0, v1);
              const bool there = (hb >> (2 * u / BS)) & 1u;
              x[u] = pair2(there && (unsigned)(2 * u - a) < len ? v0 : -INFINITY,
                           there && (unsigned)(2 * u + 1 - a) < len ? v1 : -INFINITY);
            }
          }
          const float nm = reference(max64(x));
          const f32x2 sub = pair2(nm, nm);
          lsum = weights64<TP>(pw, [&](int u) { return add2(x[u], sub); });
        }
        if (__any_sync(kFull, resc)) {  // the whole warp moves its rows' O (factor 1 for rows that keep theirs)
          // the half two before is done (its P's columns hold this S); the one before may still be multiplied
          // (a row that moves has seen keys, so there is one)
          ok = __all_sync(kFull, hf ? tc_wait(pv_done + 2 * w, n & 1, abort)
                                    : n == 0 || tc_wait(pv_done + 2 * w + 1, (n - 1) & 1, abort));
          if (!ok) break;
          tc::fence_after_sync();
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            tc::ld32(ocol + c * 32, o);
            tc::wait_ld();
#pragma unroll
            for (int u = 0; u < 32; ++u) o[u] = __float_as_uint(__uint_as_float(o[u]) * f);
            tc::st32(ocol + c * 32, o);
          }
        }
        l = l * f + lsum;
        tc::st32(scol + hf * 64, pw);  // P over S
        tc::wait_st();
        // V rows that were not copied, or lie outside the CTA's keys, may hold anything (NaN): zero them once
        // V has landed, since P = 0 times NaN is NaN in the MMA
        if (edge && hf == 0) {
          const int iv = 2 * j + 1;
          ok = __all_sync(kFull, tc_wait(full + iv % NS, (iv / NS) & 1, abort));
          if (!ok) break;
          unsigned char* vs = slot(iv);
          for (int i = threadIdx.x & 127; i < NT * 8 * Sh::DH; i += 128) {
            const int t = i / (8 * Sh::DH), c = i % (8 * Sh::DH);
            if (!((blocks >> (t / BS)) & 1u) || tb + t >= c1 || tb + t < c0)
              *reinterpret_cast<uint4*>(vs + (t / 8) * Sh::ATOM + (c / 8) * 1024 + tc::sw128(t % 8, c % 8)) =
                  make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();  // the zeros precede the PV's reads
        }
        tc::fence_before_sync();
        mbar_arrive(p_full + 2 * w + hf);
      }
      if (!ok) break;
    }
    // ---- epilogue: O / l
    if (ok && n > 0)
      ok = __all_sync(kFull, tc_wait(pv_done + 2 * w, (n - 1) & 1, abort) &&
                                 tc_wait(pv_done + 2 * w + 1, (n - 1) & 1, abort));
    tc::fence_after_sync();
    float f0 = 1.f, f1 = 0.f;  // factors of this stream's O and of the other's (shared rows)
    float* stage = reinterpret_cast<float*>(smem + Sh::OFF_RING);  // [D][128]: the other stream's O
    float* ml = reinterpret_cast<float*>(smem + Sh::OFF_ML);
    if (shared_rows) {
      // stream 1 hands its (m, l, O) over; every slot has been read, for both streams' PV are done
      asm volatile("bar.sync 2, 256;" ::: "memory");
      if (w == 1) {
        ml[row] = ok && n > 0 ? m_ref : -INFINITY;
        ml[ROWS + row] = ok && n > 0 ? l : 0.f;
        if (ok && n > 0) {
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            tc::ld32(ocol + c * 32, o);
            tc::wait_ld();
#pragma unroll
            for (int u = 0; u < 32; ++u) stage[(c * 32 + u) * ROWS + row] = __uint_as_float(o[u]);
          }
        } else {
          for (int d = 0; d < D; ++d) stage[d * ROWS + row] = 0.f;
        }
      }
      asm volatile("bar.sync 2, 256;" ::: "memory");
      if (w == 0) {
        const float m1 = ml[row], l1 = ml[ROWS + row];
        const float M = fmaxf(m_ref, m1), Ms = M == -INFINITY ? 0.f : M;
        f0 = m_ref == -INFINITY ? (l == 0.f ? 0.f : 1.f) : fast_exp2(m_ref - Ms);
        f1 = m1 == -INFINITY ? (l1 == 0.f ? 0.f : 1.f) : fast_exp2(m1 - Ms);
        l = l * f0 + l1 * f1;
        m_ref = M;
      }
    }
    ok = ok && !*abort;
    if (!shared_rows || w == 0) {
      const bool mine = active && parts.in(part), direct = parts.direct();
      const size_t orow = (size_t)(q0 + ti) * p.num_heads + h;
      // 1 / l (FP8 pool: times the value of one V code)
      const float inv = ok && l != 0.f ? (F8 ? p.v_scale : 1.f) / l : 0.f;
      bool fine = true;
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        tc::ld32(ocol + c * 32, o);
        tc::wait_ld();
        float v[32];
#pragma unroll
        for (int u = 0; u < 32; ++u) {
          v[u] = __uint_as_float(o[u]);
          if (shared_rows) v[u] = f0 * v[u] + f1 * stage[(c * 32 + u) * ROWS + row];
          v[u] = ok ? v[u] * inv : 0.f;
          fine = fine && fabsf(v[u]) < INFINITY;
        }
        if (!mine) continue;
        if (direct) {
          uint4* dst = reinterpret_cast<uint4*>(out_row + c * 32);
#pragma unroll
          for (int u = 0; u < 4; ++u)
            dst[u] = make_uint4(Elem<T>::pack2(v[8 * u], v[8 * u + 1]), Elem<T>::pack2(v[8 * u + 2], v[8 * u + 3]),
                                Elem<T>::pack2(v[8 * u + 4], v[8 * u + 5]), Elem<T>::pack2(v[8 * u + 6], v[8 * u + 7]));
        } else {
          float4* dst = reinterpret_cast<float4*>(p.part_o + (orow * p.max_partitions + part) * D + c * 32);
#pragma unroll
          for (int u = 0; u < 8; ++u) dst[u] = make_float4(v[4 * u], v[4 * u + 1], v[4 * u + 2], v[4 * u + 3]);
        }
      }
      if (mine && !direct) {
        p.part_m[orow * p.max_partitions + part] = ok ? m_ref : -INFINITY;
        p.part_l[orow * p.max_partitions + part] = ok ? l : 0.f;
      }
      // rows that came out non-finite: again, key by key, on the whole warp
      for (uint32_t redo = __ballot_sync(kFull, mine && !fine); redo; redo &= redo - 1) {
        const int src = __ffs(redo) - 1;
        const int rlo = __shfl_sync(kFull, lo, src), rhi = __shfl_sync(kFull, hi, src);
        const int rpos = __shfl_sync(kFull, pos, src), rh = __shfl_sync(kFull, h, src);
        const int rti = __shfl_sync(kFull, ti, src);
        const bool rdirect = __shfl_sync(kFull, (int)direct, src);
        const size_t at = (size_t)(q0 + rti) * p.num_heads + rh;
        float m, ll, o[D / 32];
        scored_row<T, C, D>(p, sc, at, s, rh, rpos, max(rlo, tok0), min(rhi, tok0 + P), BS, lane, m, ll, o);
        store_row<T, D>(p, at, part, rdirect, lane, m, ll, o);
      }
    }
  }

  tc::fence_before_sync();
  __syncthreads();
  if (*abort && threadIdx.x == 0) atomicOr(p.err, PKV_DEVERR_TIMEOUT);
  if (warp == Sh::MMA_WARP) {
    tc::fence_after_sync();
    tc::dealloc(tbase, Sh::TMEM_COLS);
  }
}

template <typename T, int D, int BS, bool F8, bool CAP, bool BIAS>
cudaError_t launch_scored_tc_mode(const DecodeParams& p, const ScoreParams& sc, const CUtensorMap& kmap,
                             const CUtensorMap& vmap, int num_seqs, cudaStream_t stream) {
  using Sh = ScoredTcShape<T, D, BS, F8>;
  auto kern = pkv_scored_tc_kernel<T, D, BS, F8, CAP, BIAS>;
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
  return launch_kernel(kern, grid, dim3(Sh::THREADS), Sh::SMEM, stream, p, sc, kmap, vmap);
}

// A kernel for each of the score's forms: the row loop holds 64 scores in registers, and with the forms chosen
// at run time in one kernel the compiler moved them about between the branches: a causal prompt of 8192 tokens,
// 32 heads, took 615 us against 562 (no cap or bias), 782 against 675 (cap).
template <typename T, int D, int BS, bool F8>
cudaError_t launch_scored_tc(const DecodeParams& p, const ScoreParams& sc, const CUtensorMap& kmap,
                             const CUtensorMap& vmap, int num_seqs, cudaStream_t stream) {
  if (sc.cap_out != 0.f)
    return sc.slopes ? launch_scored_tc_mode<T, D, BS, F8, true, true>(p, sc, kmap, vmap, num_seqs, stream)
                     : launch_scored_tc_mode<T, D, BS, F8, true, false>(p, sc, kmap, vmap, num_seqs, stream);
  return sc.slopes ? launch_scored_tc_mode<T, D, BS, F8, false, true>(p, sc, kmap, vmap, num_seqs, stream)
                   : launch_scored_tc_mode<T, D, BS, F8, false, false>(p, sc, kmap, vmap, num_seqs, stream);
}

}  // namespace pkv
