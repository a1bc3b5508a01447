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
// What bounds it: per 256 x 128 scores the tensor cores need about 2048 cycles (head_dim 128), the shared memory
// port 2500 (Q for every half, K and V for both streams, the copies once) and the exponentials 1024; a CTA takes 4000
// without and 4700 with a cap over its tiles (468 and 552 us, 1170 and 1000 TFLOP/s of visible scores, a causal prompt
// of 8192 tokens, 32/8 heads), with no unit saturated: it is the chain from S to P in the row threads. So a score is kept to few
// instructions: tiles that every row sees whole skip the masks, the tanh is a polynomial where the tile's scores
// stay well below the cap, and both are computed on pairs.
//
// A CTA stays and takes one (partition, row tile, kv head, sequence) after the other: when its copies of an item
// are issued it asks the hardware for the next unstarted CTA of the grid and does that one's work too. So the
// copies and first products of an item run under the end of the one before, and tensor memory and barriers are
// set up once: 16384 tokens of packed documents, 760 us with an item a CTA, 726 so. Over an FP8 pool a CTA keeps to
// its own item: the row threads convert a bf16 query themselves at an item's end, and there the next CTA's start
// is the cheaper one (E4M3 chunks with a prefix mask, 242 us staying, 221 not; a causal prompt of 8192 tokens, 567
// and 534).
//
// Warps: 0-3 and 4-7 the streams' rows; 8 and 9 issue a stream's MMAs (one thread each); 10 and 11 copy the
// blocks of K and V tiles, half of each tile a warp (a copy takes about 100 cycles to issue), into a ring of
// tile slots in the order K0 V0 K1 V1 ..., and 10 finds the items; FP8 pool: 12-15 widen a tile's codes to f16
// in place. Every wait is bounded (work_wait): a copy or MMA that does not complete makes the CTA stop, set
// PKV_DEVERR_TIMEOUT and write zeros for the rows of the item at hand. The rows of one that it has already claimed
// for later stay as they were.
#pragma once

#include <type_traits>

#include "pkv_f32x2.cuh"
#include "pkv_mq_tc.cuh"
#include "pkv_scored.cuh"

namespace pkv {

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

// The 64 weights 2^e(u) (pairs) in 16 bits into the tensor-memory columns from pcol on, half of them at a time (the
// registers); returns the sum of the fp32 weights before that rounding. A bf16 weight is off by at most its rounding
// unit, which moves the result by as much times the row's largest |v|. An f16 one (f16 and FP8 pools) below f16's
// normal range is off by up to 2^-25, where the key that gave the reference weighs 1: over n keys another n 2^-25
// times the largest |v|, 0.0005 at 16384 keys.
template <typename TP, typename E>
__device__ __forceinline__ float weights64(uint32_t pcol, E e) {
  f32x2 ls[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t pw[16];
#pragma unroll
    for (int u = 0; u < 16; ++u) {
      float a, b;
      unpair2(e(16 * i + u), a, b);
      a = fast_exp2(a);
      b = fast_exp2(b);
      pw[u] = Elem<TP>::pack2(a, b);
      ls[u & 3] = add2(ls[u & 3], pair2(a, b));
    }
    tc::st16(pcol + 16 * i, pw);
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
  // barriers: full[8], empty[8], raw[8] per slot; per stream q_full, fin; per stream and half s_full, p_full,
  // pv_done; items: info_full[2], info_empty[2], next; q_shared
  static constexpr int NBARS = 24 + 16 + 6;
  static constexpr int OFF_NEXT = (OFF_BARS + NBARS * 8 + 15) / 16 * 16;  // the hardware's answer: the next CTA
  static constexpr int OFF_MISC = OFF_NEXT + 16;                         // tensor-memory base, abort flag, sign of work
  static constexpr int OFF_INFO = OFF_MISC + 16;                         // two items
  static constexpr int OFF_ML = OFF_INFO + 2 * 64;                       // stream 1's (m, l) in an item of shared rows
  static constexpr int SMEM = OFF_ML + 2 * ROWS * 4;
  static constexpr int S_COL = 0, O_COL = 256;  // tensor memory: stream w's S at 128 w, its O at 256 + 128 w
  static constexpr int TMEM_COLS = 512;
  static constexpr int MMA_WARP = 8, COPY_WARP = 10, WIDEN_WARP = 12;
  static constexpr int THREADS = (F8 ? 16 : 12) * 32;
  static_assert(SMEM <= 232448 - 1024, "one CTA's shared memory");
  static_assert(NBT >= 4 && NBT <= 16, "blocks per tile");
  static_assert(!F8 || D == 128, "an FP8 pool: head_dim 128");
};

// tc_wait for a warp that may have to wait while rows are computed again over a whole partition (10.8 us for 32 keys
// of a row, up to 32 rows a warp: a second for 100,000 keys), or while a place of the grid that holds work is looked
// for (0.6 us an empty place; 2^27 of them are half a second if all SMs look). The warps that are at it leave a sign
// of work at abort[1] every few microseconds, and the limit runs from the last one; what they do ends by itself.
// Such waits are those for an item, its Q and its P, and for the place of an item or a tile to be free; a tile on
// its way and MMAs that were issued do not wait for the rows, and the rows wait for tiles only when none of them is
// at such work (they meet at barriers without a limit). OUT_OF_LINE: as a call, where instructions to fetch are what
// a kernel waits for (tree attention over an E4M3 pool with a cap 117 us against 120; over a 16-bit pool 62 against
// 61, scored prompts 746 against 724).
__device__ __forceinline__ bool work_wait_on(uint64_t* bar, uint32_t parity, volatile int* abort) {
  const unsigned t0 = work_clock();
  for (;;) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*abort) return false;
    const unsigned now = work_clock();  // (a sign may be newer)
    if (min((int)(now - t0), (int)(now - (unsigned)abort[1])) > (int)(kWaitLimitCycles >> kWorkClock)) {
      *abort = 1;
      return false;
    }
  }
}
static __device__ __noinline__ bool work_wait_call(uint64_t* bar, uint32_t parity, volatile int* abort) {
  return work_wait_on(bar, parity, abort);
}
template <bool OUT_OF_LINE>
__device__ __forceinline__ bool work_wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
  if (mbar_try_wait(bar, parity)) return true;
  return OUT_OF_LINE ? work_wait_call(bar, parity, abort) : work_wait_on(bar, parity, abort);
}

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

// -inf for the keys 2 u, 2 u + 1 whose bits of see are not set.
__device__ __forceinline__ void mask64(f32x2 (&x)[32], const uint32_t (&see)[2]) {
#pragma unroll
  for (int u = 0; u < 32; ++u) {
    float a, b;
    unpair2(x[u], a, b);
    const uint32_t bits = see[u >> 4];
    x[u] = pair2(bits & (1u << ((2 * u) & 31)) ? a : -INFINITY, bits & (1u << ((2 * u + 1) & 31)) ? b : -INFINITY);
  }
}
// The largest magnitude of the others.
__device__ __forceinline__ float max64_seen(const f32x2 (&x)[32], const uint32_t (&see)[2]) {
  float m = 0.f;
#pragma unroll
  for (int u = 0; u < 32; ++u) {
    float a, b;
    unpair2(x[u], a, b);
    const uint32_t bits = see[u >> 4];
    if (bits & (1u << ((2 * u) & 31))) m = fmaxf(m, fabsf(a));
    if (bits & (1u << ((2 * u + 1) & 31))) m = fmaxf(m, fabsf(b));
  }
  return m;
}

// Each lane of a quad holds four 16-byte units u[0..3] of its row; afterwards lane q holds unit q of the quad's
// rows 0..3, so that the quad stores 64 consecutive bytes of one row at a time.
__device__ __forceinline__ void quad_transpose(uint32_t (&u)[16], int lane) {
#pragma unroll
  for (int d = 1; d <= 2; d <<= 1) {
    const bool up = lane & d;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i & d) continue;
#pragma unroll
      for (int e = 0; e < 4; ++e) {  // units i and i + d
        uint32_t &a = u[4 * i + e], &b = u[4 * (i + d) + e];
        const uint32_t got = __shfl_xor_sync(kFull, up ? a : b, d);
        if (up)
          a = got;
        else
          b = got;
      }
    }
  }
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

// One CTA's work of the grid: the rows of a row tile and their keys [c0, c1).
struct ScoredItem {
  int ntile;  // tiles; 0: no key (rows that see nothing may need their zeros); -1: no more items
  int part, rt, kvh, s;
  int ctx, q0, q_len;
  int c0, c1;
  __device__ __forceinline__ long long row0() const { return (long long)rt * 256; }
  __device__ __forceinline__ int nrows(int G) const { return (int)min(256ll, (long long)q_len * G - row0()); }
};

// The item of CTA (x, y, z) of the grid, on one warp. ntile = -2: nothing to do.
template <int BS, int NT>
__device__ __forceinline__ ScoredItem scored_item(const DecodeParams& p, const ScoreParams& sc, int x, int y, int z,
                                                  int lane) {
  ScoredItem m;
  m.ntile = -2;
  // the last row tiles first: with a causal limit they see the most keys
  m.part = x / sc.row_tiles;
  m.rt = sc.row_tiles - 1 - x % sc.row_tiles;
  m.kvh = y;
  m.s = z;
  const bool reporter = x == 0 && y == 0 && lane == 0;
  m.ctx = clamp_context(p, m.s, reporter);
  m.q0 = 0;
  m.q_len = scored_query_len(sc, m.s, m.ctx, m.q0);
  if (m.q_len < 0) {
    if (reporter) atomicOr(p.err, PKV_DEVERR_QUERY);
    return m;
  }
  const int G = p.group;
  if (m.row0() >= (long long)m.q_len * G) return m;
  // its rows' first and last visible key, within the partition
  const int ta = (int)(m.row0() / G), tb = (int)((m.row0() + m.nrows(G) - 1) / G);
  const int p0 = m.ctx - m.q_len;  // position of the sequence's first query token
  int a = INT32_MAX, b = 0;
  if (!sc.key_begin && !sc.key_end) {  // the first token's first, the last token's last
    int unused;
    scored_span(sc, 0, p0 + ta, m.ctx, a, unused);
    scored_span(sc, 0, p0 + tb, m.ctx, unused, b);
  } else {
    for (int t = ta + lane; t <= tb; t += 32) {
      int lo, hi;
      scored_span(sc, m.q0 + t, p0 + t, m.ctx, lo, hi);
      if (hi > lo) {
        a = min(a, lo);
        b = max(b, hi);
      }
    }
    a = __reduce_min_sync(kFull, a);
    b = __reduce_max_sync(kFull, b);
  }
  const int tok0 = scored_base(sc, m.ctx, m.q_len, BS) + m.part * p.partition_size;
  m.c0 = max(a, tok0);
  m.c1 = min(b, tok0 + p.partition_size);
  if (m.c1 <= m.c0)
    m.ntile = m.part == 0 ? 0 : -2;
  else
    m.ntile = (m.c1 - m.c0 / BS * BS + NT - 1) / NT;
  return m;
}

// Ask for the next unstarted CTA of the grid; the answer lands at `dst` (16 bytes) and completes `bar`.
__device__ __forceinline__ void ask_next_cta(void* dst, uint64_t* bar) {
  mbar_arrive_expect_tx(bar, 16);
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                   smem_u32(dst)),
               "r"(smem_u32(bar))
               : "memory");
}
// The answer: false if there is none left, else its index.
__device__ __forceinline__ bool next_cta(const void* src, int& x, int& y, int& z) {
  uint32_t got, a, b, c;
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b128 r;\n\t"
      "ld.shared.b128 r, [%4];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t"
      "mov.u32 %1, 0;\n\tmov.u32 %2, 0;\n\tmov.u32 %3, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%1, %2, %3, _}, r;\n\t}"
      : "=r"(got), "=r"(a), "=r"(b), "=r"(c)
      : "r"(smem_u32(src))
      : "memory");
  x = (int)a;
  y = (int)b;
  z = (int)c;
  return got != 0;
}

// A stream's warp brings its 32 query rows into Q's A-operand layout (128-byte swizzled rows, columns 64.. in the
// next ROWS x 128 bytes), asynchronously, a row's bytes by neighbouring lanes. Lane l's own row is row l: its
// index in query, or -1 for zeros.
template <typename T, int D, int ROWS>
__device__ __forceinline__ void scored_fetch_q(unsigned char* Qs, int wq, int lane, const T* query, int own) {
  constexpr int CH = D / 8, RPI = 32 / CH;  // 16-byte chunks of a row, rows per instruction
  const int c = lane % CH;
#pragma unroll
  for (int i = 0; i < 32 / RPI; ++i) {
    const int rl = i * RPI + lane / CH;
    const int idx = __shfl_sync(kFull, own, rl);
    const int r = 32 * wq + rl;
    cp_async16(smem_u32(Qs) + r * 128 + (c / 8) * (ROWS * 128) + (((c % 8) ^ (r & 7)) << 4),
               query + (idx < 0 ? 0 : (size_t)idx * D) + c * 8, idx < 0 ? 0u : 16u);
  }
}

// FP8 pool with a bf16 query: the same rows in f16, each multiplied by 2^k so that its largest magnitude lies in
// [2^14, 2^15) (every bf16 value keeps its 8 significant bits unless it lies below 2^-14 of that range, where its
// contribution is far below the fp32 accumulation error). Returns this lane's row's 2^-k. store: write them.
template <int ROWS>
__device__ __forceinline__ float scored_fetch_q_bf16_as_f16(unsigned char* Qs, int wq, int lane,
                                                            const __nv_bfloat16* query, int own, bool store) {
  constexpr int D = 128;
  const int c = lane & 15;
  float mine = 1.f;
  uint4 rows[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int idx = __shfl_sync(kFull, own, 2 * i + (lane >> 4));
    rows[i] = make_uint4(0, 0, 0, 0);
    if (idx >= 0) rows[i] = *reinterpret_cast<const uint4*>(query + (size_t)idx * D + c * 8);
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int rl = 2 * i + (lane >> 4);
    const uint4 v = rows[i];
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
    float amax = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 f = Elem<__nv_bfloat16>::to_float2(w[e]);
      amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
    }
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, o));
    const int ex = static_cast<int>((__float_as_uint(amax) >> 23) & 0xff) - 127;  // floor(log2(amax))
    int k = amax > 0.f ? 14 - ex : 0;
    k = k < -60 ? -60 : (k > 60 ? 60 : k);
    const float pw = __uint_as_float(static_cast<uint32_t>(127 + k) << 23);
    const float inv = __uint_as_float(static_cast<uint32_t>(127 - k) << 23);
    const float i0 = __shfl_sync(kFull, inv, 0), i1 = __shfl_sync(kFull, inv, 16);
    if (lane == 2 * i) mine = i0;
    if (lane == 2 * i + 1) mine = i1;
    if (store) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 f = Elem<__nv_bfloat16>::to_float2(w[e]);
        w[e] = Elem<__half>::pack2(f.x * pw, f.y * pw);
      }
      const int r = 32 * wq + rl;
      *reinterpret_cast<uint4*>(Qs + r * 128 + (c / 8) * (ROWS * 128) + (((c % 8) ^ (r & 7)) << 4)) =
          make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  return mine;
}

// Whether every thread of the two streams' rows says yes.
__device__ __forceinline__ bool rows_agree(bool yes) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.and.pred q, 2, 256, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(yes ? 1u : 0u)
      : "memory");
  return r != 0;
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
  uint64_t* info_full = bars + 40;   // [2]
  uint64_t* info_empty = bars + 42;  // [2]
  uint64_t* next_bar = bars + 44;
  uint64_t* q_shared = bars + 45;  // shared rows' Q, which stream 0 brings
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Sh::OFF_MISC);
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);
  static_assert(sizeof(ScoredItem) <= 64, "an item's place");
  auto info = [&](int k) { return reinterpret_cast<ScoredItem*>(smem + Sh::OFF_INFO + (k & 1) * 64); };
  auto slot = [&](int it) { return smem + Sh::OFF_RING + (it % NS) * Sh::TILE; };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = p.group, P = p.partition_size;
  if (smem_u32(smem) & 1023u) {  // not expected on any supported GPU; nothing is written
    if (threadIdx.x == 0) atomicOr(p.err, PKV_DEVERR_LAYOUT);
    return;
  }
  if (threadIdx.x == 0) {
    prefetch_tensormap(&kmap);
    prefetch_tensormap(&vmap);
    for (int k = 0; k < NS; ++k) {
      mbar_init(full + k, F8 ? 4 : 2);
      mbar_init(empty + k, 2);  // the streams
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
      mbar_init(info_full + k, 1);
      mbar_init(info_empty + k, Sh::THREADS / 32 - 1);  // every warp but the one that finds the items
    }
    mbar_init(next_bar, 1);
    mbar_init(q_shared, ROWS);
    fence_mbar_init();
    abort[0] = 0;
    abort[1] = (int)work_clock();
  }
  if (warp == Sh::MMA_WARP) tc::alloc(tmem_slot, Sh::TMEM_COLS);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tbase = *tmem_slot;

  // Item k, read by a whole warp; its place is then free again. False: none came in time.
  auto wait_item = [&](int k) {
    return __all_sync(kFull, work_wait<false>(info_full + (k & 1), (k >> 1) & 1, abort)) != 0;
  };
  auto free_item = [&](int k) {
    __syncwarp();
    if (lane == 0) mbar_arrive(info_empty + (k & 1));
  };
  auto read_item = [&](int k, ScoredItem& m) {
    if (!wait_item(k)) return false;
    m = *info(k);
    free_item(k);
    return true;
  };
  // A stream's tiles of an item: first, first + step, ...; shared: both streams take the same rows.
  auto shared_rows = [&](const ScoredItem& m) { return m.nrows(G) <= ROWS; };

  if (warp == Sh::COPY_WARP || warp == Sh::COPY_WARP + 1) {
    // ---- copies: this warp's half of the blocks of the ring's items it = 2 j (K tile j) and 2 j + 1 (V tile j)
    constexpr int NH = NBT / 2;
    const int at = (warp - Sh::COPY_WARP) * NH + (lane & (NH - 1));  // lane < NH: block of the tile
    uint64_t* landed = F8 ? raw : full;
    const bool finder = warp == Sh::COPY_WARP;
    ScoredItem m;
    int k = 0, it = 0, asked = 0;
    bool ok = true;
    // The finder's next item with anything to do, published; x, y, z: the first CTA to look at, or have = false.
    auto find = [&](bool have, int x, int y, int z) {
      m.ntile = -2;
      while (ok && m.ntile == -2) {
        if (!have && F8) {  // (FP8 pool: one item a CTA, see above)
          m.ntile = -1;
          break;
        }
        if (!have) {
          if (lane == 0) {
            fence_proxy_async_smem();  // the answer before has been read
            ask_next_cta(smem + Sh::OFF_NEXT, next_bar);
          }
          __syncwarp();
          ok = __all_sync(kFull, tc_wait(next_bar, asked & 1, abort));
          ++asked;
          if (!ok) {  // the answer may not land in a CTA that has left
            mbar_wait(next_bar, (asked - 1) & 1);
            break;
          }
          have = next_cta(smem + Sh::OFF_NEXT, x, y, z);
          __syncwarp();
        }
        if (have)
          m = scored_item<BS, NT>(p, sc, x, y, z, lane);
        else
          m.ntile = -1;  // (nothing is asked again)
        have = false;
        if (m.ntile == -2 && lane == 0) abort[1] = (int)work_clock();
      }
      if (ok && k >= 2) ok = __all_sync(kFull, work_wait<false>(info_empty + (k & 1), ((k >> 1) - 1) & 1, abort));
      if (!ok) return;
      if (lane == 0) {
        *info(k) = m;
        mbar_arrive(info_full + (k & 1));
      }
      __syncwarp();
    };
    if (finder)
      find(true, blockIdx.x, blockIdx.y, blockIdx.z);
    else
      ok = read_item(0, m);
    while (ok && m.ntile >= 0) {
      const int blk0 = m.c0 / BS, nblk = m.ntile > 0 ? (m.c1 + BS - 1) / BS - blk0 : 0;
      const int32_t* table = p.block_tables + (size_t)m.s * p.max_blocks_per_seq + blk0;
      auto load_id = [&](int j) { return lane < NH && j * NBT + at < nblk ? table[j * NBT + at] : -1; };
      int next = load_id(0);
      for (int j = 0; ok && j < m.ntile; ++j) {
        int id = next;
        if (j + 1 < m.ntile) next = load_id(j + 1);
        if (lane < NH && j * NBT + at < nblk && (unsigned)id >= (unsigned)p.num_blocks) {
          const int last = (int)((m.row0() + m.nrows(G) - 1) / G);
          if (block_seen<false, BS>(sc, m.q0, m.q_len, m.ctx, (int)(m.row0() / G), last, (blk0 + j * NBT + at) * BS))
            atomicOr(p.err, PKV_DEVERR_BLOCK_ID);
          id = -1;
        }
        const int n = __popc(__ballot_sync(kFull, id >= 0));
        const int y = (id * p.num_kv_heads + m.kvh) * BS;  // first pool row of the block
#pragma unroll
        for (int kv = 0; kv < 2; ++kv, ++it) {
          uint64_t* bar = landed + it % NS;
          if (it >= NS) ok = __all_sync(kFull, work_wait<false>(empty + it % NS, (it / NS - 1) & 1, abort));
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
      ++k;
      if (!ok) break;
      if (finder)
        find(false, 0, 0, 0);
      else
        ok = read_item(k, m);
    }
    // no copy may still be landing when the CTA leaves
    if (lane == 0)
      for (int i = it > NS ? it - NS : 0; i < it; ++i) mbar_wait(landed + i % NS, (i / NS) & 1);
  } else if (F8 && warp >= Sh::WIDEN_WARP) {
    // ---- FP8 pool: widen each slot's codes once they have landed
    // (agreed among the four warps, which meet at barriers: all go on, or all leave)
    ScoredItem m;
    int it = 0;
    bool ok = true;
    for (int k = 0; ok; ++k) {
      ok = widen_agree(read_item(k, m));
      if (!ok || m.ntile < 0) break;
      for (int i = 0; i < 2 * m.ntile; ++i, ++it) {
        ok = widen_agree(tc_wait(raw + it % NS, (it / NS) & 1, abort));
        if (!ok) break;
        if constexpr (F8) scored_widen(slot(it), Sh::HALF, warp - Sh::WIDEN_WARP, lane);
        fence_proxy_async_smem();  // generic stores, read by the MMAs
        __syncwarp();
        if (lane == 0) mbar_arrive(full + it % NS);
      }
    }
  } else if (warp == Sh::MMA_WARP || warp == Sh::MMA_WARP + 1) {
    // ---- MMA issue: one thread per stream, in the order S S | PV S | PV S | ... by halves of a tile
    const int st = warp - Sh::MMA_WARP;
    constexpr bool BF = std::is_same<TP, __nv_bfloat16>::value;
    constexpr uint32_t IDESC_S = tc::idesc_f16(BF, ROWS, NT / 2, false, false);
    constexpr uint32_t IDESC_O = tc::idesc_f16(BF, ROWS, D, false, true);
    const uint32_t scol = tbase + Sh::S_COL + st * NT, ocol = tbase + Sh::O_COL + st * 128;
    ScoredItem m;
    int tiles = 0, cnt = 0, nq = 0;  // ring tiles of the items before, this stream's tiles, items with keys
    int nshared = 0;                 // of them with shared rows
    bool ok = true;
    for (int k = 0; ok; ++k) {
      ok = read_item(k, m);
      if (!ok || m.ntile < 0) break;
      if (m.ntile == 0) continue;
      const bool shared = shared_rows(m);
      const int first = shared ? st : 0, step = shared ? 2 : 1;
      if (lane == 0) {
        const uint32_t q_addr = smem_u32(smem) + (shared ? 0 : st * Sh::QT);
        // The other stream's tile of shared rows: waited for and freed like one of this stream's. (Every waiter goes
        // through every phase of a barrier: one that left a phase out could not tell the next from the last.)
        auto skip_tile = [&](int j) {
          for (int it = 2 * (tiles + j); it < 2 * (tiles + j) + 2; ++it) {
            if (!tc_wait(full + it % NS, (it / NS) & 1, abort)) return false;
            mbar_arrive(empty + it % NS);
          }
          return true;
        };
        // S of tile j's half hf (64 keys: 8 atoms of K) into that half's columns, which the caller knows are free
        auto issue_s = [&](int j, int hf) {
          const int ik = 2 * (tiles + j);
          if (hf == 0 && !tc_wait(full + ik % NS, (ik / NS) & 1, abort)) return false;
          tc::fence_after_sync();
          const uint32_t k_addr = smem_u32(slot(ik)) + hf * 8 * Sh::ATOM;
#pragma unroll
          for (int u = 0; u < D / 16; ++u)
            tc::mma_f16(scol + hf * 64, tc::desc_sw128(q_addr + (u / 4) * (ROWS * 128) + (u % 4) * 32, 16, 1024),
                        tc::desc_sw128(k_addr + (u / 4) * 1024 + (u % 4) * 32, 16, Sh::ATOM), IDESC_S, u > 0);
          tc::commit(s_full + 2 * st + hf);
          if (hf) {
            tc::commit(empty + ik % NS);
            if (shared && j + 1 < m.ntile) return skip_tile(j + 1);
          }
          return true;
        };
        // a P's columns take the next S: not before its PV has read it
        auto pv_read = [&](int hf) { return cnt == 0 || tc_wait(pv_done + 2 * st + hf, (cnt - 1) & 1, abort); };
        // Shared rows are stream 0's to bring, so stream 1 waits for those too, on a barrier of shared items alone:
        // of q_full[0] it would leave out the other items' phases, and in those the streams may be an item apart.
        ok = work_wait<false>(q_full + st, nq & 1, abort) &&
             (st == 0 || !shared || work_wait<false>(q_shared, nshared++ & 1, abort));
        if (first > 0) ok = ok && skip_tile(0);
        if (first < m.ntile) {
          ok = ok && pv_read(0) && issue_s(first, 0) && pv_read(1) && issue_s(first, 1);
        } else {  // a stream without tiles goes through the motions of one
          for (int hf = 0; ok && hf < 2; ++hf) {
            ok = pv_read(hf);
            tc::commit(s_full + 2 * st + hf);
          }
          ++cnt;
          for (int hf = 0; ok && hf < 2; ++hf) {
            ok = work_wait<false>(p_full + 2 * st + hf, (cnt - 1) & 1, abort);
            tc::commit(pv_done + 2 * st + hf);
          }
        }
        for (int j = first; ok && j < m.ntile; j += step) {
          const int iv = 2 * (tiles + j) + 1;
          const uint32_t v_addr = smem_u32(slot(iv));
          ++cnt;
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            ok = ok && work_wait<false>(p_full + 2 * st + hf, (cnt - 1) & 1, abort) &&
                 (hf > 0 || tc_wait(full + iv % NS, (iv / NS) & 1, abort));
            if (!ok) break;
            tc::fence_after_sync();
#pragma unroll
            for (int u = 0; u < 4; ++u)  // 16 keys each: 8 columns of P, two atoms of V
              tc::mma_f16_ta(ocol, scol + hf * 64 + u * 8,
                             tc::desc_sw128(v_addr + (hf * 4 + u) * 2 * Sh::ATOM, 1024, Sh::ATOM), IDESC_O,
                             j > first || hf > 0 || u > 0);
            tc::commit(pv_done + 2 * st + hf);
            if (hf) tc::commit(empty + iv % NS);
            if (j + step < m.ntile) ok = pv_read(hf) && issue_s(j + step, hf);
          }
        }
      }
      tiles += m.ntile;
      ++nq;
      ok = __all_sync(kFull, ok);
    }
    if (lane == 0) {
      tc::commit(fin + st);  // every MMA issued above has completed once this arrives
      mbar_wait(fin + st, 0);
    }
    __syncwarp();
  } else if (warp < 8) {
    // ---- rows
    const int w = warp >> 2;                  // stream
    const int row = 32 * (warp & 3) + lane;   // row of the stream: its tensor-memory lane
    const uint32_t scol = tc::taddr(tbase, 32 * (warp & 3), Sh::S_COL + w * NT);
    const uint32_t ocol = tc::taddr(tbase, 32 * (warp & 3), Sh::O_COL + w * 128);
    float* ml = reinterpret_cast<float*>(smem + Sh::OFF_ML);
    constexpr bool Q_AS_F16 = F8 && std::is_same<T, __nv_bfloat16>::value;
    // (an item is read where it lies, and its place freed at its end: the row loop has no registers to spare)
    int tiles = 0, cnt = 0;  // ring tiles of the items before, this stream's tiles
    float qscale = 1.f, qscale_next = 1.f;  // FP8 pool, bf16 query: the 2^-k the row was scaled by
    // this thread's row of an item, as an index into the output's rows; -1: none
    auto own_row = [&](const ScoredItem& i, int& ti, int& h) {
      const int rr = (shared_rows(i) ? 0 : w * ROWS) + row;
      if (rr >= i.nrows(G)) {
        ti = 0;
        h = i.kvh * G;
        return -1;
      }
      const long long r = i.row0() + rr;
      ti = (int)(r / G);
      h = i.kvh * G + (int)(r - (long long)ti * G);
      return (i.q0 + ti) * p.num_heads + h;
    };
    // bring an item's Q into place (the S of the item before have all read theirs), and say so
    auto start_q = [&](const ScoredItem& i) {
      int ti, h;
      const int own = own_row(i, ti, h);
      const bool shared = shared_rows(i);
      unsigned char* Qs = smem + (shared ? 0 : w * Sh::QT);
      if constexpr (Q_AS_F16)  // (both streams need the factors of shared rows)
        qscale_next = scored_fetch_q_bf16_as_f16<ROWS>(
            Qs, warp & 3, lane, reinterpret_cast<const __nv_bfloat16*>(p.query), own, !shared || w == 0);
      else if (!shared || w == 0)
        scored_fetch_q<T, D, ROWS>(Qs, warp & 3, lane, reinterpret_cast<const T*>(p.query), own);
    };
    auto finish_q = [&](const ScoredItem& i) {
      cp_async_wait_all();
      fence_proxy_async_smem();  // generic-proxy writes, read by the S MMAs
      mbar_arrive(q_full + w);
      if (w == 0 && shared_rows(i)) mbar_arrive(q_shared);
    };
    bool ok = rows_agree(wait_item(0));
    if (ok && info(0)->ntile > 0) {
      start_q(*info(0));
      finish_q(*info(0));
    }
    for (int k = 0; ok; ++k) {
      const ScoredItem& m = *info(k);
      if (m.ntile < 0) {
        free_item(k);
        break;
      }
      qscale = qscale_next;
      const bool shared = shared_rows(m);
      int ti, h;
      const int orow = own_row(m, ti, h);
      const bool active = orow >= 0;
      const int pos = m.ctx - m.q_len + ti;
      int lo = 0, hi = 0;
      if (active) scored_span(sc, m.q0 + ti, pos, m.ctx, lo, hi);
      const int base = scored_base(sc, m.ctx, m.q_len, BS);
      const int tok0 = base + m.part * P;
      const RowParts parts = row_parts(lo, hi, base, P);
      T* out_row = static_cast<T*>(p.out) + (size_t)(active ? orow : 0) * D;
      if (m.ntile == 0) {  // no key: the zeros of rows that see nothing
        if (active && parts.last < parts.first && (!shared || w == 0))
          for (int d = 0; d < D; d += 8) *reinterpret_cast<uint4*>(out_row + d) = make_uint4(0u, 0u, 0u, 0u);
        free_item(k);
        ok = rows_agree(wait_item(k + 1));
        if (ok && info(k + 1)->ntile > 0) {
          start_q(*info(k + 1));
          finish_q(*info(k + 1));
        }
        continue;
      }
      const int first = shared ? w : 0, step = shared ? 2 : 1;
      const float sl2 = p.scale_log2 * qscale;
      const float cap_in = sc.cap_in * qscale, cap_out = sc.cap_out;
      const float slope = BIAS ? sc.slopes[h] * 1.4426950408889634f : 0.f;
      // cap_out * tanh(x * cap_in) = x (c0 + c1 x^2 + c2 x^4 + c3 x^6) while |x * cap_in| <= 1/2: a minimax fit of
      // tanh(z) / z in z^2 on [0, 1/4], relative error 6e-7. The coefficients hold cap_in's powers, up to the seventh:
      // not for factors with which those come near the ends of fp32's range (caps far from the scale), whose tiles
      // take the long form. A bf16 query over an FP8 pool, whose cap_in has the row's 2^-k, would always be such a
      // one: there x is the product times cap_in, and the coefficients are cap_out's alone (a causal prompt of 8192
      // tokens, cap 50: 770 us; 750 with coefficients that vanished).
      const float unit = Q_AS_F16 ? 1.f : cap_in;  // of x, in tanh's argument
      f32x2 cc[4];
      float near1 = -1.f;  // the largest |x| that it is for
      if constexpr (CAP) {
        const float z2 = unit * unit, c3 = fabsf(cap_out * unit) * z2 * z2 * z2;
        float c = cap_out * unit;
        const float fit[4] = {0.999999456f, -0.333263179f, 0.131902965f, -0.0444022226f};
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          cc[u] = pair2(c * fit[u], c * fit[u]);
          c *= z2;
        }
        if (Q_AS_F16 || (c3 > 1e-36f && c3 < 1e30f)) near1 = 0.5f / fabsf(unit);
      }
      // (FP8 pool: read again where they are used, to keep the 128 registers a thread for the scores: held in
      // registers they took the causal prompt of 8192 tokens from 571 to 714 us)
      const int c0_ = m.c0, c1_ = m.c1, ntile_ = m.ntile;
      auto c0 = [&] { return F8 ? m.c0 : c0_; };
      auto c1 = [&] { return F8 ? m.c1 : c1_; };
      auto ntile = [&] { return F8 ? m.ntile : ntile_; };
      // which blocks of a tile were copied: lane b < NBT holds block b's test (the copying warps' own)
      auto load_ok = [&](int j) {
        const int b = c0() / BS + j * NBT + (lane & (NBT - 1));
        return b < (c1() + BS - 1) / BS &&
               (unsigned)p.block_tables[(size_t)m.s * p.max_blocks_per_seq + b] < (unsigned)p.num_blocks;
      };
      constexpr uint32_t all = (1u << NBT) - 1u;
      float m_ref = -INFINITY, l = 0.f;
      int n = 0;
      bool next = first < ntile() && load_ok(first);
      for (int j = first; j < ntile(); j += step, ++n, ++cnt) {
        const uint32_t blocks = __ballot_sync(kFull, next) & all;
        if (j + step < ntile()) next = load_ok(j + step);
        const int tb = c0() / BS * BS + j * NT;  // position of the tile's first token
        // V rows outside the item's keys, or not copied
        const bool edge = blocks != all || tb < c0() || tb + NT > c1();
#pragma unroll 1
        for (int hf = 0; hf < 2; ++hf) {
          const int th = tb + hf * 64;
          // (tensor-memory accesses are warp-wide: a warp leaves the loop as a whole)
          ok = __all_sync(kFull, tc_wait(s_full + 2 * w + hf, cnt & 1, abort));
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
          if constexpr (CAP && Q_AS_F16) {
#pragma unroll
            for (int u = 0; u < 32; ++u) x[u] = mul2(x[u], pair2(cap_in, cap_in));
          }
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
          float lsum;  // of the half's weights
          // bit t of see[i]: the row sees key 32 i + t of the half
          auto seen = [&](uint32_t (&see)[2]) {
#pragma unroll
            for (int i = 0; i < 2; ++i) see[i] = low_bits(hi - th - 32 * i) & ~low_bits(lo - th - 32 * i);
            if (blocks != all) {
#pragma unroll
              for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int b = 0; b < 32 / BS; ++b)
                  if (!((blocks >> (hf * (NBT / 2) + i * (32 / BS) + b)) & 1u))
                    see[i] &= ~((BS == 32 ? 0xffffffffu : (1u << (BS & 31)) - 1u) << (b * BS));
            }
          };
          const bool all_whole = __all_sync(kFull, whole);
          bool fast = false;  // the whole warp sees the whole half, and the scores take their short form
          float top = 0.f;
          if (!BIAS && all_whole) {
            if constexpr (CAP) {
              top = max64(x);
              const float bottom = -max64neg(x);
              fast = __all_sync(kFull, fmaxf(top, -bottom) <= near1);  // at most half the cap
              if (unit < 0.f) top = bottom;
            } else {
              fast = sl2 >= 0.f;
            }
          }
          if (fast) {
            if constexpr (CAP) {
              const f32x2 t = pair2(top, top), t2 = mul2(t, t);
              float mx, unused;
              unpair2(mul2(t, fma2(t2, fma2(t2, fma2(t2, cc[3], cc[2]), cc[1]), cc[0])), mx, unused);
              const float nm = reference(mx);
              const f32x2 sub = pair2(nm, nm);
              lsum = weights64<TP>(scol + hf * 64, [&](int u) {
                const f32x2 sq = mul2(x[u], x[u]);
                return fma2(x[u], fma2(sq, fma2(sq, fma2(sq, cc[3], cc[2]), cc[1]), cc[0]), sub);
              });
            } else {
              const float nm = reference(max64(x) * sl2);
              const f32x2 mul = pair2(sl2, sl2), sub = pair2(nm, nm);
              lsum = weights64<TP>(scol + hf * 64, [&](int u) { return fma2(x[u], mul, sub); });
            }
          } else {
            if constexpr (CAP) {
              bool near = (BIAS || !all_whole) && __all_sync(kFull, max3(max64(x), max64neg(x), 0.f) <= near1);
              if (!near && !all_whole) {  // (a key that is not seen may hold anything)
                uint32_t see[2];
                seen(see);
                near = __all_sync(kFull, max64_seen(x, see) <= near1);
              }
              if (near) {
#pragma unroll
                for (int u = 0; u < 32; ++u) {
                  const f32x2 sq = mul2(x[u], x[u]);
                  x[u] = mul2(x[u], fma2(sq, fma2(sq, fma2(sq, cc[3], cc[2]), cc[1]), cc[0]));
                }
              } else {
#pragma unroll
                for (int u = 0; u < 32; ++u) {
                  // Some score is of the cap's size: cap_out (1 - 2 / (e^(2 z) + 1)) for those, whose cancellation is
                  // small beside them, and the polynomial for the others, whatever stands beside them.
                  const f32x2 z = Q_AS_F16 ? x[u] : mul2(x[u], pair2(unit, unit)), sq = mul2(z, z);
                  f32x2 t = pair2(-0.0444022226f, -0.0444022226f);
                  t = fma2(sq, t, pair2(0.131902965f, 0.131902965f));
                  t = fma2(sq, t, pair2(-0.333263179f, -0.333263179f));
                  t = fma2(sq, t, pair2(0.999999456f, 0.999999456f));
                  float z0, z1, v0, v1, n0, n1;
                  unpair2(z, z0, z1);
                  unpair2(mul2(mul2(z, t), pair2(cap_out, cap_out)), n0, n1);
                  unpair2(mul2(z, pair2(2.8853900817779268f, 2.8853900817779268f)), v0, v1);  // e^(2z) = 2^v
                  unpair2(add2(pair2(fast_exp2(v0), fast_exp2(v1)), pair2(1.f, 1.f)), v0, v1);
                  unpair2(fma2(pair2(fast_rcp(v0), fast_rcp(v1)), pair2(-2.f * cap_out, -2.f * cap_out),
                               pair2(cap_out, cap_out)),
                          v0, v1);
                  x[u] = pair2(fabsf(z0) <= 0.5f ? n0 : v0, fabsf(z1) <= 0.5f ? n1 : v1);
                }
              }
              if constexpr (BIAS) add_bias(x, slope, pos - th);
            } else if (BIAS && (__all_sync(kFull, pos >= th + 63) || __all_sync(kFull, pos <= th))) {
              // keys all up to the tokens' own positions, or all from them on: -slope |p - j| is linear in j, four
              // chains of steps of 8
              const float d = (float)(th - pos), sl = pos <= th ? -slope : slope;
              const f32x2 mul = pair2(sl2, sl2), step8 = pair2(8.f * sl, 8.f * sl);
              f32x2 bias[4];
#pragma unroll
              for (int k4 = 0; k4 < 4; ++k4) bias[k4] = pair2(sl * (d + 2 * k4), sl * (d + 2 * k4 + 1));
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
              uint32_t see[2];
              seen(see);
              mask64(x, see);
            }
            const float nm = reference(max64(x));
            const f32x2 sub = pair2(nm, nm);
            lsum = weights64<TP>(scol + hf * 64, [&](int u) { return add2(x[u], sub); });
          }
          l = l * f + lsum;
          if (__any_sync(kFull, resc)) {  // the whole warp moves its rows' O (factor 1 for rows that keep theirs)
            // the half two before is done (its P's columns hold this S); the one before may still be multiplied
            // (a row that moves has seen keys, so there is one)
            ok = __all_sync(kFull, hf ? tc_wait(pv_done + 2 * w, cnt & 1, abort)
                                      : n == 0 || tc_wait(pv_done + 2 * w + 1, (cnt - 1) & 1, abort));
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
          tc::wait_st();
          // V rows that were not copied, or lie outside the CTA's keys, may hold anything (NaN): zero them once
          // V has landed, since P = 0 times NaN is NaN in the MMA
          if (edge && hf == 0) {
            const int iv = 2 * (tiles + j) + 1;
            ok = __all_sync(kFull, tc_wait(full + iv % NS, (iv / NS) & 1, abort));
            if (!ok) break;
            unsigned char* vs = slot(iv);
            for (int i = threadIdx.x & 127; i < NT * 8 * Sh::DH; i += 128) {
              const int t = i / (8 * Sh::DH), c = i % (8 * Sh::DH);
              if (!((blocks >> (t / BS)) & 1u) || tb + t >= c1() || tb + t < c0())
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
      if (first >= m.ntile) {  // a stream without tiles
        for (int hf = 0; ok && hf < 2; ++hf) {
          ok = __all_sync(kFull, tc_wait(s_full + 2 * w + hf, cnt & 1, abort));
          if (ok) mbar_arrive(p_full + 2 * w + hf);
        }
        ++cnt;
      }
      // ---- the next item's Q: this stream's S have all been read (of shared rows: both streams', below)
      bool going = false;
      auto next_q = [&] {
        going = wait_item(k + 1);
        if (going && info(k + 1)->ntile > 0) {
          start_q(*info(k + 1));
          if (Q_AS_F16) finish_q(*info(k + 1));
        }
      };
      if (ok && !shared) next_q();
      // ---- epilogue: O / l
      if (ok)
        ok = __all_sync(kFull, tc_wait(pv_done + 2 * w, (cnt - 1) & 1, abort) &&
                                   tc_wait(pv_done + 2 * w + 1, (cnt - 1) & 1, abort));
      tc::fence_after_sync();
      float f0 = 1.f, f1 = 0.f;  // factors of this stream's O and of the other's (shared rows)
      bool other = false;        // the other stream has an O
      if (shared) {  // stream 1 hands its (m, l) over; its O stays where it is until the item's end
        if (w == 1) {
          ml[row] = ok && n > 0 ? m_ref : -INFINITY;
          ml[ROWS + row] = ok && n > 0 ? l : 0.f;
        }
        tc::fence_before_sync();
        ok = rows_agree(ok);
        tc::fence_after_sync();
        if (w == 0) {
          other = m.ntile > 1;
          const float m1 = ml[row], l1 = ml[ROWS + row];
          const float M = fmaxf(m_ref, m1), Ms = M == -INFINITY ? 0.f : M;
          f0 = m_ref == -INFINITY ? (l == 0.f ? 0.f : 1.f) : fast_exp2(m_ref - Ms);
          f1 = m1 == -INFINITY ? (l1 == 0.f ? 0.f : 1.f) : fast_exp2(m1 - Ms);
          l = l * f0 + l1 * f1;
          m_ref = M;
        }
      }
      if (ok && shared) next_q();
      if (!Q_AS_F16 && going && info(k + 1)->ntile > 0) finish_q(*info(k + 1));
      if (!shared || w == 0) {
        const bool mine = active && parts.in(m.part), direct = parts.direct();
        // 1 / l (FP8 pool: times the value of one V code)
        const float inv = ok && l != 0.f ? (F8 ? p.v_scale : 1.f) / l : 0.f;
        bool fine = true;
        int quad_row[4];  // the rows of this lane's quad that go to the output; -1: not
#pragma unroll
        for (int i = 0; i < 4; ++i) quad_row[i] = __shfl_sync(kFull, mine && direct ? orow : -1, (lane & ~3) + i);
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          tc::ld32(ocol + c * 32, o);
          tc::wait_ld();
          float v[32];
#pragma unroll
          for (int u = 0; u < 32; ++u) v[u] = __uint_as_float(o[u]);
          if (other) {
            tc::ld32(ocol + 128 + c * 32, o);
            tc::wait_ld();
#pragma unroll
            for (int u = 0; u < 32; ++u) v[u] = f0 * v[u] + f1 * __uint_as_float(o[u]);
          }
#pragma unroll
          for (int u = 0; u < 32; ++u) {
            v[u] = ok ? v[u] * inv : 0.f;
            fine = fine && fabsf(v[u]) < INFINITY;
          }
          uint32_t o16[16];
#pragma unroll
          for (int u = 0; u < 16; ++u) o16[u] = Elem<T>::pack2(v[2 * u], v[2 * u + 1]);
          quad_transpose(o16, lane);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (quad_row[i] >= 0)
              *reinterpret_cast<uint4*>(static_cast<T*>(p.out) + (size_t)quad_row[i] * D + c * 32 + (lane & 3) * 8) =
                  make_uint4(o16[4 * i], o16[4 * i + 1], o16[4 * i + 2], o16[4 * i + 3]);
          if (mine && !direct) {
            float4* dst = reinterpret_cast<float4*>(p.part_o + ((size_t)orow * p.max_partitions + m.part) * D + c * 32);
#pragma unroll
            for (int u = 0; u < 8; ++u) dst[u] = make_float4(v[4 * u], v[4 * u + 1], v[4 * u + 2], v[4 * u + 3]);
          }
        }
        if (mine && !direct) {
          p.part_m[(size_t)orow * p.max_partitions + m.part] = ok ? m_ref : -INFINITY;
          p.part_l[(size_t)orow * p.max_partitions + m.part] = ok ? l : 0.f;
        }
        // Rows that came out non-finite by a masked key's value (not by NaN scores of their own): again, on the
        // whole warp. A value that a row sees is its own, so a NaN in the cache costs one look over the item's values.
        uint32_t redo = __ballot_sync(kFull, mine && !fine && ok && l == l && (lo > m.c0 || hi < m.c1));
        if (redo) {
          int bad0, bad1;
          bad_values<C, D>(p, m.s, m.kvh, m.c0, m.c1, BS, lane, bad0, bad1, abort + 1);
          redo &= __ballot_sync(kFull, bad0 > bad1 || lo > bad0 || hi <= bad1);
        }
        for (; redo; redo &= redo - 1) {
          const int src = __ffs(redo) - 1;
          const int rlo = __shfl_sync(kFull, lo, src), rhi = __shfl_sync(kFull, hi, src);
          const int rpos = __shfl_sync(kFull, pos, src), rh = __shfl_sync(kFull, h, src);
          const int at = __shfl_sync(kFull, orow, src);
          const bool rdirect = __shfl_sync(kFull, (int)direct, src);
          float rm, rl, o[D / 32];
          scored_row<T, C, D>(p, sc, at, m.s, rh, rpos, max(rlo, tok0), min(rhi, tok0 + P), BS, lane, rm, rl, o,
                              abort + 1);
          store_row<T, D>(p, at, m.part, rdirect, lane, rm, rl, o);
        }
      }
      // both streams go on together (stream 1's O has been read), or leave together
      tc::fence_before_sync();
      ok = rows_agree(ok && going);
      tc::fence_after_sync();
      tiles += m.ntile;
      free_item(k);
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
