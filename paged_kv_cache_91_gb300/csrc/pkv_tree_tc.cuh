// Tree attention with few rows per kv head, on the fifth-generation tensor cores (tcgen05).
//
// One CTA per SM takes up to 128 (query token, head) rows of a (partition, kv head, sequence) -- row r is query token
// r / G, head kvh * G + r % G -- and streams the keys that any of them sees in tiles of 64 tokens (64 / block_size pool
// blocks). Two streams of four row warps take the tiles in turn, each with the same rows and its own running softmax:
//   S = Q . K^T        M 128, N 64, K = head_dim       -> tensor memory (fp32), two buffers a stream
//   P = exp2(score(S) - m)   one thread per row, 16-bit, over S's columns
//   O += P . V         M 128, N = head_dim, K 64       A from tensor memory
// and at an item's end their (m, l, O) are merged, each stream's threads writing half of the head's dims.
//
// With at most 128 rows a (key, value) pair of a 16-bit pool is worth 128 flops a byte, below the machine's 290: the
// kernel is there to keep K and V coming. Their tiles go through rings of their own for each stream and for K and V
// (12 slots of 16 KB at head_dim 128), so that a stream frees a slot without waiting for the other. The next item is
// found while the one before is still being read, so the rings do not empty between items; a CTA stays and takes one
// item after the other from the hardware's queue, the longest sequences first where the batch is small enough for the
// order to be worked out in place (kTreeSortSeqs sequences).
//
// What bounds it: over a 16-bit pool HBM (19 sequences of 8192 tokens, 32/8 heads, trees of 32: 101 to 105 us, 6.1 to
// 6.4 TB/s, 91 to 94 % of the copy rate; a tile takes 0.75 us from HBM and 0.51 out of L2). An E4M3 tile, half the bytes,
// takes the same 0.5 us: a stream has some 2000 cycles for each of its tiles, in which the S MMAs, whose N of 64 keys is
// short beside what it takes to bring in 128 rows of Q, hold their issuing thread for 720 and the PV MMAs for 465, in turn
// with the other stream's (tensor pipe 41 %, HBM 47 %, issue slots 50 %). Q in tensor memory, in place of one of the four
// S buffers or of one O, would relieve them and is not built. With a cap it is the rows' arithmetic, some 1700 of a
// stream's 2650 cycles a tile (0.65 us); the four warps' chains wait for S, load it and store P for another 460, with two
// row warps a scheduler (issue slots 51 %). There the kernel's 128 registers do not hold everything: 20 to 28 bytes a
// thread are spilled and 40 to 44 loaded. An item's start and end cost 2.6 us over a 16-bit pool and 5 over an E4M3 one.
// Two threads to a row, each with half of a tile's keys, were slower (E4M3: 0.70 us a tile): what a tile costs a warp
// besides its keys doubles. With more than 128 rows per kv head K and V come once a row tile.
//
// Warps: 0-3 and 4-7 the streams' rows; 8 and 9 issue a stream's MMAs (one thread each); 10 copies K, 11 copies V and
// finds the items; FP8 pool: 12-15 widen the codes of one (stream, K or V) ring each to f16, from the slots where they
// land to the ring that the MMAs read. Every wait is bounded (work_wait): a copy or MMA that does not complete makes
// the CTA stop, set PKV_DEVERR_TIMEOUT and write zeros for the rows of the item at hand. The rows of one that it has
// already claimed for later stay as they were.
#pragma once

#include <type_traits>

#include "pkv_scored_tc.cuh"

namespace pkv {

template <typename T, int D, int BS, bool F8>
struct TreeTcShape {
  static constexpr int ROWS = 128;           // rows per item (M)
  static constexpr int NT = 64;              // tokens per tile
  static constexpr int NBT = NT / BS;        // pool blocks per tile
  static constexpr int DH = D / 64;          // 128-byte halves of a 16-bit row
  static constexpr int ATOM = DH * 1024;     // 8 tokens: their columns 0..63, then 64..127
  static constexpr int TILE = NT / 8 * ATOM; // bytes of a K or V tile slot
  static constexpr int QT = DH * ROWS * 128; // bytes of Q
  static constexpr int NR = F8 ? 2 : D == 128 ? 3 : 6;  // slots of a ring; rings: stream 0 K, V, stream 1 K, V
  static constexpr int NS = 4 * NR;
  static constexpr int CODES = NT * 128;     // FP8 pool: bytes of a tile's codes
  static constexpr int NC = F8 ? 2 : 0;      // and the slots of a ring where they land
  static constexpr int OFF_RING = QT;
  static constexpr int OFF_CODES = OFF_RING + NS * TILE;
  static constexpr int OFF_BARS = OFF_CODES + 4 * NC * CODES;
  // barriers: full[NS], done[NS], raw[4 NC], codes_free[4 NC]; per stream and buffer p_full; per stream fin; q_full;
  // items: info_full[2], info_empty[2], next
  static constexpr int NBARS = 2 * NS + 8 * NC + 4 + 2 + 1 + 5;
  static constexpr int OFF_NEXT = (OFF_BARS + NBARS * 8 + 15) / 16 * 16;  // the hardware's answer: the next CTA
  static constexpr int OFF_MISC = OFF_NEXT + 16;                         // tensor-memory base, abort flag, sign of work
  static constexpr int OFF_INFO = OFF_MISC + 16;                         // two items
  static constexpr int OFF_ML = OFF_INFO + 2 * 64;                       // the streams' (m, l) at an item's end
  static constexpr int OFF_ORDER = OFF_ML + 4 * ROWS * 4;
  static constexpr int OFF_EXPS = OFF_ORDER + kTreeSortSeqs;             // FP8 pool, bf16 query: the rows' powers of two
  static constexpr int SMEM = OFF_EXPS + (F8 ? ROWS : 0);
  static constexpr int S_COL = 0, O_COL = 256;  // tensor memory: stream w's S at 128 w, its O at 256 + 128 w
  static constexpr int TMEM_COLS = 512;
  static constexpr int MMA_WARP = 8, COPY_WARP = 10, WIDEN_WARP = 12;
  static constexpr int THREADS = (F8 ? 16 : 12) * 32;
  static constexpr int AHEAD = 6;  // tiles left to copy of an item when the next is asked for
  static_assert(SMEM <= 232448, "one CTA's shared memory");
  static_assert(NBT >= 2 && NBT <= 8, "blocks per tile");
  static_assert(!F8 || D == 128, "an FP8 pool: head_dim 128");
};

// Whether the phase with the given parity has completed, without waiting.
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// One CTA's work of the grid: the rows of a row tile and their keys [c0, c1).
struct TreeItem {
  int ntile;  // tiles; 0: no key (rows that see nothing may need their zeros); -1: no more items
  int part, rt, kvh, s;
  int ctx, q0, q_len;
  int c0, c1;
  __device__ __forceinline__ int tiles(int stream) const { return (ntile + 1 - stream) >> 1; }
  __device__ __forceinline__ long long row0() const { return (long long)rt * 128; }
  __device__ __forceinline__ int nrows(int G) const { return (int)min(128ll, (long long)q_len * G - row0()); }
};

// The item of CTA (x, y) of the grid for sequence s, on one warp. ntile = -2: nothing to do.
template <int BS, int NT>
__device__ __forceinline__ TreeItem tree_item(const DecodeParams& p, const ScoreParams& sc, int x, int y, int s,
                                              int lane) {
  TreeItem m;
  m.ntile = -2;
  m.part = x / sc.row_tiles;
  m.rt = x % sc.row_tiles;
  m.kvh = y;
  m.s = s;
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
  if (m.part > 0 && m.part * p.partition_size >= m.ctx) return m;
  // its rows' first visible key; the last is the context's
  int a = 0, b = m.ctx;
  if (sc.key_begin) {
    const int ta = (int)(m.row0() / G), tb = (int)((m.row0() + m.nrows(G) - 1) / G);
    a = INT32_MAX;
    for (int t = ta + lane; t <= tb; t += 32) a = min(a, max(0, sc.key_begin[m.q0 + t]));
    a = __reduce_min_sync(kFull, a);
  }
  const int tok0 = m.part * p.partition_size;  // (no overflow: the host bounds contexts by 2^30)
  m.c0 = max(a, tok0);
  m.c1 = min(b, tok0 + p.partition_size);
  if (m.c1 <= m.c0)
    m.ntile = m.part == 0 ? 0 : -2;
  else
    m.ntile = (m.c1 - m.c0 / BS * BS + NT - 1) / NT;
  return m;
}

// FP8 pool: one warp widens a tile's 64 rows of 128 codes at src to f16 in the operand layout at slot. Lane (t = lane
// / 8, c = lane % 8) takes codes 16 c .. 16 c + 15 of token 4 a + t as two groups of 8, which become two 16-byte
// chunks of its row. Lanes take their second group first where c / 4 + t is odd, so that 16 lanes read all banks once
// and 8 lanes store to all banks once: the f16 row's halves lie 1024 bytes apart. (Two rounds of one loop: its code shares
// the instruction caches with the rows', whose warps waited for instructions less. With a cap 121 us against 125.)
__device__ __forceinline__ void tree_widen(unsigned char* slot, const unsigned char* src, int lane) {
  const int t = lane >> 3, c = lane & 7;
  const int g0 = ((c >> 2) + t) & 1;
  const unsigned char* from = src + t * 128 + 16 * c;
#pragma unroll 1
  for (int batch = 0; batch < 2; ++batch) {
    uint2 x[8][2];
#pragma unroll
    for (int a = 0; a < 8; ++a) {
      x[a][0] = *reinterpret_cast<const uint2*>(from + (8 * batch + a) * 512 + 8 * g0);
      x[a][1] = *reinterpret_cast<const uint2*>(from + (8 * batch + a) * 512 + 8 * (g0 ^ 1));
    }
#pragma unroll
    for (int a = 0; a < 8; ++a) {
      const int row = 4 * (a & 1) + t;  // of its atom
      unsigned char* to = slot + (4 * batch + a / 2) * 2048 + (c >> 2) * 1024 + row * 128;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        uint32_t h[4];
        e4m3x4_to_f16x2(x[a][k].x, h[0], h[1]);
        e4m3x4_to_f16x2(x[a][k].y, h[2], h[3]);
        *reinterpret_cast<uint4*>(to + (((2 * (c & 3) + (g0 ^ k)) ^ row) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
      }
    }
  }
}

// A warp brings rows 32 wq + 16 half .. + 15 of an item into Q's A-operand layout (128-byte swizzled rows, columns
// 64.. in the next 128 x 128 bytes), asynchronously. own: lane l's row is row 32 wq + l: its index in query, or -1
// for zeros.
template <typename T, int D>
__device__ __forceinline__ void tree_fetch_q(unsigned char* Qs, int wq, int half, int lane, const T* query, int own) {
  constexpr int CH = D / 8, RPI = 32 / CH;  // 16-byte chunks of a row, rows per instruction
  const int c = lane % CH;
#pragma unroll
  for (int i = 0; i < 16 / RPI; ++i) {
    const int rl = 16 * half + i * RPI + lane / CH;
    const int idx = __shfl_sync(kFull, own, rl);
    const int r = 32 * wq + rl;
    cp_async16(smem_u32(Qs) + r * 128 + (c / 8) * (128 * 128) + (((c % 8) ^ (r & 7)) << 4),
               query + (idx < 0 ? 0 : (size_t)idx * D) + c * 8, idx < 0 ? 0u : 16u);
  }
}

// FP8 pool with a bf16 query: the same 16 rows in f16, each multiplied by 2^k so that its largest magnitude lies in
// [1, 2): every bf16 value keeps its 8 significant bits unless it lies below 2^-16 of that, where it is off by at most
// 2^-25 of it. (So the row's 2^-k leaves a cap's factors near where the scale put them.) exps[r] = k for the rows.
__device__ __forceinline__ void tree_fetch_q_bf16_as_f16(unsigned char* Qs, int wq, int half, int lane,
                                                         const __nv_bfloat16* query, int own, signed char* exps) {
  constexpr int D = 128;
  const int c = lane & 15;
  uint4 rows[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int idx = __shfl_sync(kFull, own, 16 * half + 2 * i + (lane >> 4));
    rows[i] = make_uint4(0, 0, 0, 0);
    if (idx >= 0) rows[i] = *reinterpret_cast<const uint4*>(query + (size_t)idx * D + c * 8);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    uint32_t w[4] = {rows[i].x, rows[i].y, rows[i].z, rows[i].w};
    // the largest exponent, by the magnitudes' bits (NaN and infinity count as the largest)
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) top = max(top, max(w[e] & 0x7fffu, (w[e] >> 16) & 0x7fffu));
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) top = max(top, __shfl_xor_sync(kFull, top, o));
    int k = top ? 127 - (int)(top >> 7) : 0;
    k = max(-126, min(126, k));
    const float pw = __uint_as_float((uint32_t)(127 + k) << 23);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 f = Elem<__nv_bfloat16>::to_float2(w[e]);
      w[e] = Elem<__half>::pack2(f.x * pw, f.y * pw);
    }
    const int r = 32 * wq + 16 * half + 2 * i + (lane >> 4);
    *reinterpret_cast<uint4*>(Qs + r * 128 + (c / 8) * (128 * 128) + (((c % 8) ^ (r & 7)) << 4)) =
        make_uint4(w[0], w[1], w[2], w[3]);
    if (c == 0) exps[r] = (signed char)k;
  }
}

// The largest magnitude of 64 values held as pairs.
__device__ __forceinline__ float max64abs(const f32x2 (&x)[32]) {
  float m[4], a, b;
#pragma unroll
  for (int u = 0; u < 32; ++u) {
    unpair2(x[u], a, b);
    m[u & 3] = u < 4 ? fmaxf(fabsf(a), fabsf(b)) : max3(m[u & 3], fabsf(a), fabsf(b));
  }
  return max3(fmaxf(m[0], m[1]), m[2], m[3]);
}

template <typename T, int D, int BS, bool F8, bool CAP>
__global__ void __launch_bounds__(F8 ? 512 : 384, 1)
    pkv_tree_tc_kernel(const __grid_constant__ DecodeParams p, const __grid_constant__ ScoreParams sc,
                       const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
  pdl_begin();
  using Sh = TreeTcShape<T, D, BS, F8>;
  using TP = typename std::conditional<F8, __half, T>::type;        // the MMAs' type
  using C = typename std::conditional<F8, __nv_fp8_e4m3, T>::type;  // the cache's
  constexpr int NT = Sh::NT, NBT = Sh::NBT, NR = Sh::NR, NS = Sh::NS, NC = Sh::NC, ROWS = Sh::ROWS;
  extern __shared__ __align__(1024) unsigned char smem[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Sh::OFF_BARS);
  // full: the tile is in its slot. done: its MMAs have read it, so that S (a K slot) is there or O holds its PV (a V
  // slot): one barrier for all who wait for that, since a commit costs the issuing thread some 90 cycles.
  uint64_t *full = bars, *done = bars + NS, *raw = bars + 2 * NS, *codes_free = raw + 4 * NC;
  uint64_t* p_full = codes_free + 4 * NC;  // [stream][buffer]
  uint64_t* fin = p_full + 4;              // [stream]: everything issued
  uint64_t* q_full = fin + 2;
  uint64_t* info_full = q_full + 1;   // [2]
  uint64_t* info_empty = info_full + 2;
  uint64_t* next_bar = info_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Sh::OFF_MISC);
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);
  static_assert(sizeof(TreeItem) <= 64, "an item's place");
  auto info = [&](int k) { return reinterpret_cast<TreeItem*>(smem + Sh::OFF_INFO + (k & 1) * 64); };
  // The c-th tile of ring (stream, kv): its slot, and the phase of that slot's barriers.
  auto slot_of = [](int stream, int kv, int c) { return (2 * stream + kv) * NR + c % NR; };
  auto phase_of = [](int c) { return (uint32_t)(c / NR) & 1u; };
  auto slot = [&](int i) { return smem + Sh::OFF_RING + i * Sh::TILE; };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = p.group, P = p.partition_size;
  if (smem_u32(smem) & 1023u) {  // not expected on any supported GPU; nothing is written
    if (threadIdx.x == 0) atomicOr(p.err, PKV_DEVERR_LAYOUT);
    return;
  }
  unsigned char* order = smem + Sh::OFF_ORDER;
  int* lens = reinterpret_cast<int*>(smem + Sh::OFF_ML);
  if ((int)threadIdx.x < sc.sort_seqs) lens[threadIdx.x] = p.context_lens[threadIdx.x];
  if (threadIdx.x == 0) {
    prefetch_tensormap(&kmap);
    prefetch_tensormap(&vmap);
    for (int k = 0; k < NS; ++k) {
      mbar_init(full + k, 1);
      mbar_init(done + k, 1);
    }
    for (int k = 0; k < 4 * NC; ++k) {
      mbar_init(raw + k, 1);
      mbar_init(codes_free + k, 1);
    }
    for (int k = 0; k < 4; ++k) mbar_init(p_full + k, ROWS);
    for (int k = 0; k < 2; ++k) {
      mbar_init(fin + k, 1);
      mbar_init(info_full + k, 1);
      mbar_init(info_empty + k, Sh::THREADS / 32 - 1);  // every warp but the one that finds the items
    }
    mbar_init(q_full, 2 * ROWS + 2);  // and the threads that issue MMAs, once they have seen the Q before
    mbar_init(next_bar, 1);
    fence_mbar_init();
    abort[0] = 0;
    abort[1] = (int)work_clock();
  }
  if (warp == Sh::MMA_WARP) tc::alloc(tmem_slot, Sh::TMEM_COLS);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tbase = *tmem_slot;
  if (sc.sort_seqs) {  // sequences by context length, longest first (equal ones in their order)
    if ((int)threadIdx.x < sc.sort_seqs) {
      const int mine = lens[threadIdx.x];
      int rank = 0;
      for (int j = 0; j < sc.sort_seqs; ++j) {
        const int other = lens[j];
        rank += other > mine || (other == mine && j < (int)threadIdx.x);
      }
      order[rank] = (unsigned char)threadIdx.x;
    }
    __syncthreads();
  }

  // Item k, read by a whole warp; its place is then free again. False: none came in time.
  auto wait_item = [&](int k) {
    return __all_sync(kFull, work_wait<F8>(info_full + (k & 1), (k >> 1) & 1, abort)) != 0;
  };
  auto free_item = [&](int k) {
    __syncwarp();
    if (lane == 0) mbar_arrive(info_empty + (k & 1));
  };
  auto read_item = [&](int k, TreeItem& m) {
    if (!wait_item(k)) return false;
    m = *info(k);
    free_item(k);
    return true;
  };

  if (warp == Sh::COPY_WARP || warp == Sh::COPY_WARP + 1) {
    // ---- copies: the blocks of this warp's K or V tiles, a lane a block (a copy takes about 100 cycles to issue). V's
    // warp also finds the items: this CTA's own, then whatever the hardware's queue still holds. It asks for the next
    // one AHEAD tiles before an item's end, looks for the answer between copies, and reads what that item is while the
    // tiles on their way keep the others busy.
    const int kv = warp - Sh::COPY_WARP;
    const bool finder = kv == 1;
    TreeItem m, then;  // the item at hand; the finder's next one
    bool ok = true;
    int issued[2] = {0, 0};  // tiles of the streams' rings
    uint64_t* landed = F8 ? raw : full;
    constexpr int NL = F8 ? NC : NR;  // slots of a ring where tiles land
    int asked = 0;
    bool pending = false;  // an answer is on its way
    auto ask = [&] {
      if (lane == 0) {
        fence_proxy_async_smem();  // the answer before has been read
        ask_next_cta(smem + Sh::OFF_NEXT, next_bar);
      }
      __syncwarp();
      ++asked;
      pending = true;
    };
    // the item of the answer at hand, or of this CTA: as item k, once two before is free; false if it is empty
    auto publish = [&](int k, bool have, int x, int y, int z) {
      then.ntile = -1;
      if (have) then = tree_item<BS, NT>(p, sc, x, y, sc.sort_seqs ? order[z] : z, lane);
      if (then.ntile == -2) {
        if (lane == 0) abort[1] = (int)work_clock();
        return false;
      }
      if (k >= 2) ok = __all_sync(kFull, work_wait<F8>(info_empty + (k & 1), ((k >> 1) - 1) & 1, abort));
      if (ok && lane == 0) {
        *info(k) = then;
        mbar_arrive(info_full + (k & 1));
      }
      __syncwarp();
      return true;
    };
    // take the answer that has come (or wait for it) and go on asking while the answers are empty
    bool found = true;
    auto look = [&](int k, bool block) {
      while (ok && !found) {
        if (block)
          ok = __all_sync(kFull, tc_wait(next_bar, (asked - 1) & 1, abort));
        else if (!__all_sync(kFull, mbar_test(next_bar, (asked - 1) & 1)))
          return;
        if (!ok) return;
        pending = false;
        int x, y, z;
        const bool have = next_cta(smem + Sh::OFF_NEXT, x, y, z);
        __syncwarp();
        found = publish(k, have, x, y, z);
        if (!found) ask();
      }
    };
    if (finder) {
      found = publish(0, true, blockIdx.x, blockIdx.y, blockIdx.z);
      if (!found) {
        ask();
        look(0, true);
      }
    }
    for (int k = 0; ok; ++k) {
      if (finder)
        m = then;
      else
        ok = read_item(k, m);
      if (!ok || m.ntile < 0) break;
      const int ask_at = max(0, m.ntile - 1 - Sh::AHEAD);
      const int blk0 = m.c0 / BS, nblk = m.ntile > 0 ? (m.c1 + BS - 1) / BS - blk0 : 0;
      const int32_t* table = p.block_tables + (size_t)m.s * p.max_blocks_per_seq + blk0;
      auto load_ids = [&](int b0) { return b0 + lane < nblk ? table[b0 + lane] : -1; };
      auto checked = [&](int b0, int id) {
        if (b0 + lane < nblk && (unsigned)id >= (unsigned)p.num_blocks) {
          const int last = (int)((m.row0() + m.nrows(G) - 1) / G);
          if (!finder && block_seen<true, BS>(sc, m.q0, m.q_len, m.ctx, (int)(m.row0() / G), last,
                                              (blk0 + b0 + lane) * BS))
            atomicOr(p.err, PKV_DEVERR_BLOCK_ID);
          return -1;
        }
        return id;
      };
      int next = load_ids(0), cur = -1;  // the ids of 32 blocks at a time, the next 32 ahead
      if (finder) {
        found = false;
        if (m.ntile == 0) ask();
      }
#pragma unroll 1
      for (int t = 0; ok && t < m.ntile; ++t) {
        const int b0 = t * NBT, stream = t & 1;
        if (b0 % 32 == 0) {
          cur = checked(b0, next);
          next = load_ids(b0 + 32);
        }
        const int at = lane % NBT;  // lane < NBT: block of the tile
        const int id = __shfl_sync(kFull, cur, (b0 + at) % 32);
        const bool mine = lane < NBT && id >= 0;
        const int n = __popc(__ballot_sync(kFull, mine));
        const int row = (id * p.num_kv_heads + m.kvh) * BS;  // first pool row of the block
        const int c = stream ? issued[1] : issued[0], i = (2 * stream + kv) * NL + c % NL;
        if (c >= NL) ok = __all_sync(kFull, work_wait<F8>((F8 ? codes_free : done) + i, (c / NL - 1) & 1, abort));
        if (!ok) break;
        if (lane == 0) {
          if (!F8) fence_proxy_async_smem();  // generic stores into the slot (zeroed rows): before the copies
          mbar_arrive_expect_tx(landed + i, n * BS * (F8 ? 128 : D * 2));
        }
        __syncwarp();
        if (mine) {
          const CUtensorMap* map = kv ? &vmap : &kmap;
          if constexpr (F8)
            tma_load_2d(smem + Sh::OFF_CODES + i * Sh::CODES + at * BS * 128, map, 0, row, landed + i);
          else if constexpr (Sh::DH == 2)
            tma_load_4d(slot(i) + at * (BS / 8) * Sh::ATOM, map, 0, 0, 0, row / 8, landed + i);
          else
            tma_load_2d(slot(i) + at * (BS / 8) * Sh::ATOM, map, 0, row, landed + i);
        }
        if (stream)
          ++issued[1];
        else
          ++issued[0];
        if (finder && t == ask_at) ask();
        if (finder && t > ask_at) look(k + 1, false);
      }
      if (finder) look(k + 1, true);
    }
    // no answer and no copy may still be landing when the CTA leaves
    if (pending) mbar_wait(next_bar, (asked - 1) & 1);
    if (lane == 0)
      for (int st = 0; st < 2; ++st)
        for (int c = max(0, issued[st] - NL); c < issued[st]; ++c)
          mbar_wait(landed + (2 * st + kv) * NL + c % NL, (c / NL) & 1);
  } else if (F8 && warp >= Sh::WIDEN_WARP) {
    // ---- FP8 pool: this warp's ring: the codes that have landed, to f16
    if constexpr (F8) {
      const int r = warp - Sh::WIDEN_WARP;
      TreeItem m;
      int c = 0;
      bool ok = true;
      for (int k = 0; ok; ++k) {
        ok = read_item(k, m);
        if (!ok || m.ntile < 0) break;
        const int end = c + m.tiles(r >> 1);
        for (; ok && c < end; ++c) {
          const int from = r * NC + c % NC, to = slot_of(r >> 1, r & 1, c);
          ok = __all_sync(kFull, work_wait<F8>(raw + from, (c / NC) & 1, abort) &&
                                     (c < NR || work_wait<F8>(done + to, (c / NR - 1) & 1, abort)));
          if (!ok) break;
          tree_widen(slot(to), smem + Sh::OFF_CODES + from * Sh::CODES, lane);
          fence_proxy_async_smem();  // generic stores, read by the MMAs
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(full + to);
            mbar_arrive(codes_free + from);
          }
        }
      }
    }
  } else if (warp == Sh::MMA_WARP || warp == Sh::MMA_WARP + 1) {
    // ---- MMA issue: one thread per stream, in the order S S | PV S | PV S | ...
    const int st = warp - Sh::MMA_WARP;
    constexpr bool BF = std::is_same<TP, __nv_bfloat16>::value;
    constexpr uint32_t IDESC_S = tc::idesc_f16(BF, ROWS, NT, false, false);
    constexpr uint32_t IDESC_O = tc::idesc_f16(BF, ROWS, D, false, true);
    const uint32_t scol = tbase + Sh::S_COL + st * 128, ocol = tbase + Sh::O_COL + st * 128;
    // (descriptors are built once and stepped by constants: one built anew for every MMA kept the issuing thread, which
    // is what bounds a tile out of L2, for 80 cycles an MMA)
    const uint64_t q_desc = tc::desc_sw128(smem_u32(smem), 16, 1024);
    const uint64_t k_desc = tc::desc_sw128(smem_u32(slot(slot_of(st, 0, 0))), 16, Sh::ATOM);
    const uint64_t v_desc = tc::desc_sw128(smem_u32(slot(slot_of(st, 1, 0))), 1024, Sh::ATOM);
    TreeItem m;
    int cnt = 0, nq = 0;  // this stream's tiles and the items with keys before
    bool ok = true;
    if (lane == 0) mbar_arrive(q_full);
    for (int k = 0; ok; ++k) {
      ok = read_item(k, m);
      if (!ok || m.ntile < 0) break;
      if (m.ntile == 0) continue;
      const int end = cnt + m.tiles(st);
      if (lane == 0) {
        // (the waits for tiles to land stand where MMAs run meanwhile: a wait costs some 90 cycles also when it is over)
        auto landed = [&](int kv, int c) { return c >= end || tc_wait(full + slot_of(st, kv, c), phase_of(c), abort); };
        // S of the stream's tile c, whose K has landed, once the PV two before has read its P from these columns
        auto issue_s = [&](int c) {
          const int i = slot_of(st, 0, c);
          if (c >= 2 && !tc_wait(done + slot_of(st, 1, c - 2), phase_of(c - 2), abort)) return false;
          tc::fence_after_sync();
          const uint64_t b_desc = k_desc + (uint64_t)((c % NR) * (Sh::TILE / 16));
          const uint32_t to = scol + (c & 1) * 64;
#pragma unroll
          for (int u = 0; u < D / 16; ++u)
            tc::mma_f16(to, q_desc + ((u / 4) * (ROWS * 128) + (u % 4) * 32) / 16,
                        b_desc + ((u / 4) * 1024 + (u % 4) * 32) / 16, IDESC_S, u > 0);
          tc::commit(done + i);
          return true;
        };
        // (a stream without tiles in an item holds nobody up there: by its arrival the next Q's phase cannot complete
        // before it has seen this one's, whose parity would be that of the one after next)
        ok = landed(0, cnt) && work_wait<F8>(q_full, nq & 1, abort);
        if (ok) mbar_arrive(q_full);
        for (int c = cnt; ok && c < min(end, cnt + 2); ++c) ok = landed(0, c) && issue_s(c);
        ok = ok && landed(1, cnt);
        for (int c = cnt; ok && c < end; ++c) {
          const int i = slot_of(st, 1, c);
          ok = work_wait<F8>(p_full + 2 * st + (c & 1), (c >> 1) & 1, abort);
          if (!ok) break;
          tc::fence_after_sync();
          const uint64_t b_desc = v_desc + (uint64_t)((c % NR) * (Sh::TILE / 16));
          const uint32_t from = scol + (c & 1) * 64;
#pragma unroll
          for (int u = 0; u < NT / 16; ++u)  // 16 keys each: 8 columns of P, two atoms of V
            tc::mma_f16_ta(ocol, from + u * 8, b_desc + u * 2 * Sh::ATOM / 16, IDESC_O, u > 0 || c > cnt);
          tc::commit(done + i);
          ok = landed(0, c + 2) && landed(1, c + 1);
          if (ok && c + 2 < end) ok = issue_s(c + 2);
        }
      }
      cnt = end;
      ++nq;
      ok = __all_sync(kFull, ok);
    }
    if (lane == 0) {
      tc::commit(fin + st);  // every MMA issued above has completed once this arrives
      mbar_wait(fin + st, 0);
    }
    __syncwarp();
  } else {
    // ---- rows
    const int w = warp >> 2;                 // stream
    const int row = 32 * (warp & 3) + lane;  // its tensor-memory lane
    const uint32_t scol = tc::taddr(tbase, 32 * (warp & 3), Sh::S_COL + w * 128);
    const uint32_t ocol = tc::taddr(tbase, 32 * (warp & 3), Sh::O_COL);
    float* ml = reinterpret_cast<float*>(smem + Sh::OFF_ML);
    constexpr bool Q_AS_F16 = F8 && std::is_same<T, __nv_bfloat16>::value;
    // (an item is read where it lies, and its place freed at its end: the row loop has no registers to spare)
    int cnt = 0;                             // this stream's tiles of the items before
    float qscale = 1.f;                      // FP8 pool, bf16 query: the 2^-k the row was scaled by
    signed char* exps = reinterpret_cast<signed char*>(smem + Sh::OFF_EXPS);
    // this thread's row of an item, as an index into the output's rows; -1: none
    auto own_row = [&](const TreeItem& i, int& ti, int& h) {
      if (row >= i.nrows(G)) {
        ti = 0;
        h = i.kvh * G;
        return -1;
      }
      const long long r = i.row0() + row;
      ti = (int)(r / G);
      h = i.kvh * G + (int)(r - (long long)ti * G);
      return (i.q0 + ti) * p.num_heads + h;
    };
    // bring an item's Q into place (the S of the item before have all read theirs), and say so
    auto start_q = [&](const TreeItem& i) {
      int ti, h;
      const int own = own_row(i, ti, h);
      if constexpr (Q_AS_F16)
        tree_fetch_q_bf16_as_f16(smem, warp & 3, w, lane, reinterpret_cast<const __nv_bfloat16*>(p.query), own, exps);
      else
        tree_fetch_q<T, D>(smem, warp & 3, w, lane, reinterpret_cast<const T*>(p.query), own);
    };
    auto finish_q = [&] {
      cp_async_wait_all();
      fence_proxy_async_smem();  // generic-proxy writes, read by the S MMAs
      mbar_arrive(q_full);
    };
    bool ok = wait_item(0);
    if (ok && info(0)->ntile > 0) {
      start_q(*info(0));
      finish_q();
    }
    ok = rows_agree(ok);
    for (int k = 0; ok; ++k) {
      const TreeItem& m = *info(k);
      if (m.ntile < 0) {
        free_item(k);
        break;
      }
      if (Q_AS_F16 && m.ntile > 0) qscale = __uint_as_float((uint32_t)(127 - exps[row]) << 23);
      int ti, h;
      const int orow = own_row(m, ti, h);
      const bool active = orow >= 0;
      const int node0 = m.ctx - m.q_len;  // position of the tree's node 0
      int lo = 0, hi = 0;
      if (active) scored_span<true>(sc, m.q0 + ti, 0, m.ctx, lo, hi);
      const RowParts parts = row_parts(lo, hi, 0, P);
      T* out_row = static_cast<T*>(p.out) + (size_t)(active ? orow : 0) * D;
      if (m.ntile == 0) {  // no key: the zeros of rows that see nothing
        if (active && parts.last < parts.first && w == 0)
          for (int d = 0; d < D; d += 8) *reinterpret_cast<uint4*>(out_row + d) = make_uint4(0u, 0u, 0u, 0u);
        ok = wait_item(k + 1);
        if (ok && info(k + 1)->ntile > 0) {
          start_q(*info(k + 1));
          finish_q();
        }
        ok = rows_agree(ok);
        free_item(k);
        continue;
      }
      const float sl2 = p.scale_log2 * qscale;
      const float cap_in = sc.cap_in * qscale, cap_out = sc.cap_out;
      // cap_out * tanh(x * cap_in) as in the scored tile: x (c0 + c1 x^2 + c2 x^4 + c3 x^6) while |x * cap_in| <= 1/2,
      // the coefficients holding cap_in's powers where fp32 holds them; elsewhere the tiles take the long form
      f32x2 cc[4];
      float near1 = -1.f;  // the largest |x| that it is for
      if constexpr (CAP) {
        const float z2 = cap_in * cap_in, c3 = fabsf(cap_out * cap_in) * z2 * z2 * z2;
        float c = cap_out * cap_in;
        const float fit[4] = {0.999999456f, -0.333263179f, 0.131902965f, -0.0444022226f};
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          cc[u] = pair2(c * fit[u], c * fit[u]);
          c *= z2;
        }
        if (c3 > 1e-36f && c3 < 1e30f) near1 = 0.5f / fabsf(cap_in);
      }
      // (FP8 pool: read again where they are used, to keep the 128 registers a thread for the scores)
      const int c0_ = m.c0, c1_ = m.c1, ntile_ = m.ntile;
      auto c0 = [&] { return F8 ? m.c0 : c0_; };
      auto c1 = [&] { return F8 ? m.c1 : c1_; };
      auto ntile = [&] { return F8 ? m.ntile : ntile_; };
      // Which blocks of a tile were copied: lane b < NBT holds block b's id, -1 past the last, to put to the copying
      // warp's own test. (Loaded a tile ahead and tested when it is used: tested at once, the load held the warp up for
      // 500 of a tile's 2000 cycles.)
      auto load_id = [&](int t) {
        const int b = c0() / BS + t * NBT + (lane & (NBT - 1));
        return b < (c1() + BS - 1) / BS ? p.block_tables[(size_t)m.s * p.max_blocks_per_seq + b] : -1;
      };
      constexpr uint32_t all = (1u << NBT) - 1u;
      float m_ref = -INFINITY, l = 0.f;
      int n = 0;
      int next = w < ntile() ? load_id(w) : -1;
#pragma unroll 1
      for (int t = w; t < ntile(); t += 2, ++n) {
        const int c = cnt + n, b = c & 1;
        const uint32_t blocks = __ballot_sync(kFull, (unsigned)next < (unsigned)p.num_blocks) & all;
        if (t + 2 < ntile()) next = load_id(t + 2);
        const int th = c0() / BS * BS + t * NT;  // position of the tile's first token
        // V rows outside the item's keys, or not copied
        const bool edge = blocks != all || th < c0() || th + NT > c1();
        uint32_t nodes[2] = {0u, 0u};  // the tile's keys in the mask of the row's tree (read before the wait)
        const bool drafted = th + NT > node0;
        if (drafted) {
          nodes[0] = tree_bits(sc, m.q0 + ti, th - node0);
          nodes[1] = tree_bits(sc, m.q0 + ti, th + 32 - node0);
        }
        // (tensor-memory accesses are warp-wide: a warp leaves the loop as a whole)
        ok = __all_sync(kFull, tc_wait(done + slot_of(w, 0, c), phase_of(c), abort));
        if (!ok) break;
        tc::fence_after_sync();
        uint32_t sr[2][32];
        tc::ld32(scol + b * 64, sr[0]);
        tc::ld32(scol + b * 64 + 32, sr[1]);
        tc::wait_ld();
        f32x2 x[32];  // keys 2 u and 2 u + 1 of the tile
#pragma unroll
        for (int u = 0; u < 32; ++u)
          x[u] = pair2(__uint_as_float(sr[u >> 4][(2 * u) & 31]), __uint_as_float(sr[u >> 4][(2 * u + 1) & 31]));
        // (a row past the last one, which is not stored, needs no mask: its warp may leave them out)
        const bool whole = !edge && (!active || (th >= lo && th + NT <= hi && !drafted));
        float f = 1.f;      // factor of what the row holds
        bool resc = false;  // O's row holds terms to rescale
        // The reference m moves, and the row is rescaled, only when a score exceeds it by more than 8, so weights are
        // at most 2^8. A row that has seen nothing yet exponentiates against 0 (its scores are -inf, or NaN, which
        // must stay).
        auto reference = [&](float mx) {
          const bool move = mx > m_ref + 8.f;
          resc = move && m_ref != -INFINITY;
          f = resc ? fast_exp2(m_ref - mx) : 1.f;
          if (move) m_ref = mx;
          return m_ref == -INFINITY ? 0.f : -m_ref;
        };
        float lsum;  // of the tile's weights
        // bit t of see[i]: the row sees key 32 i + t of the tile
        auto seen = [&](uint32_t (&see)[2]) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            see[i] = low_bits(hi - th - 32 * i) & ~low_bits(lo - th - 32 * i);
            if (drafted) see[i] &= nodes[i];
          }
          if (blocks != all) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
              for (int u = 0; u < 32 / BS; ++u)
                if (!((blocks >> (i * (32 / BS) + u)) & 1u))
                  see[i] &= ~((BS == 32 ? 0xffffffffu : (1u << (BS & 31)) - 1u) << (u * BS));
          }
        };
        const bool all_whole = __all_sync(kFull, whole);
        bool fast = false;  // the whole warp sees the whole tile, and the scores take their short form
        float big = 0.f;
        if (all_whole) {
          if constexpr (CAP) {
            big = max64abs(x);
            fast = __all_sync(kFull, big <= near1);  // at most half the cap
          } else {
            fast = sl2 >= 0.f;
          }
        }
        if (fast) {
          if constexpr (CAP) {
            auto capped = [&](float v) {
              const f32x2 t1 = pair2(v, v), t2 = mul2(t1, t1);
              float mx, unused;
              unpair2(mul2(t1, fma2(t2, fma2(t2, fma2(t2, cc[3], cc[2]), cc[1]), cc[0])), mx, unused);
              return mx;
            };
            // (the largest magnitude bounds the scores: while no row's reference can move, their maximum is not needed.
            // 117 us against 121)
            float nm = -m_ref;
            if (!__all_sync(kFull, fabsf(capped(big)) <= m_ref + 8.f))
              nm = reference(capped(cap_in < 0.f ? -max64neg(x) : max64(x)));
            const f32x2 sub = pair2(nm, nm);
            lsum = weights64<TP>(scol + b * 64, [&](int u) {
              const f32x2 sq = mul2(x[u], x[u]);
              return fma2(x[u], fma2(sq, fma2(sq, fma2(sq, cc[3], cc[2]), cc[1]), cc[0]), sub);
            });
          } else {
            const float nm = reference(max64(x) * sl2);
            const f32x2 mul = pair2(sl2, sl2), sub = pair2(nm, nm);
            lsum = weights64<TP>(scol + b * 64, [&](int u) { return fma2(x[u], mul, sub); });
          }
        } else {
          if constexpr (CAP) {
            bool near = !all_whole && __all_sync(kFull, max64abs(x) <= near1);
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
                const f32x2 z = mul2(x[u], pair2(cap_in, cap_in)), sq = mul2(z, z);
                f32x2 q = pair2(-0.0444022226f, -0.0444022226f);
                q = fma2(sq, q, pair2(0.131902965f, 0.131902965f));
                q = fma2(sq, q, pair2(-0.333263179f, -0.333263179f));
                q = fma2(sq, q, pair2(0.999999456f, 0.999999456f));
                float z0, z1, v0, v1, n0, n1;
                unpair2(z, z0, z1);
                unpair2(mul2(mul2(z, q), pair2(cap_out, cap_out)), n0, n1);
                unpair2(mul2(z, pair2(2.8853900817779268f, 2.8853900817779268f)), v0, v1);  // e^(2z) = 2^v
                unpair2(add2(pair2(fast_exp2(v0), fast_exp2(v1)), pair2(1.f, 1.f)), v0, v1);
                unpair2(fma2(pair2(fast_rcp(v0), fast_rcp(v1)), pair2(-2.f * cap_out, -2.f * cap_out),
                             pair2(cap_out, cap_out)),
                        v0, v1);
                x[u] = pair2(fabsf(z0) <= 0.5f ? n0 : v0, fabsf(z1) <= 0.5f ? n1 : v1);
              }
            }
          } else {
            const f32x2 mul = pair2(sl2, sl2);
#pragma unroll
            for (int u = 0; u < 32; ++u) x[u] = mul2(x[u], mul);
          }
          if (!whole) {
            uint32_t see[2];
            seen(see);
            mask64(x, see);
          }
          const float nm = reference(max64(x));
          const f32x2 sub = pair2(nm, nm);
          lsum = weights64<TP>(scol + b * 64, [&](int u) { return add2(x[u], sub); });
        }
        l = l * f + lsum;
        if (__any_sync(kFull, resc)) {  // the whole warp moves its rows' O (factor 1 for rows that keep theirs)
          // the PV two before is done (its P's columns hold this S); the one before may still be multiplied
          // (a row that moves has seen keys, so there is one)
          ok = __all_sync(kFull, n == 0 || tc_wait(done + slot_of(w, 1, c - 1), phase_of(c - 1), abort));
          if (!ok) break;
          tc::fence_after_sync();
#pragma unroll
          for (int u = 0; u < D / 32; ++u) {
            uint32_t o[32];
            tc::ld32(ocol + w * 128 + u * 32, o);
            tc::wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
            tc::st32(ocol + w * 128 + u * 32, o);
          }
        }
        tc::wait_st();
        // V rows that were not copied, or lie outside the CTA's keys, may hold anything (NaN): zero them once V has
        // landed, since P = 0 times NaN is NaN in the MMA
        if (edge) {
          const int i = slot_of(w, 1, c);
          ok = __all_sync(kFull, tc_wait(full + i, phase_of(c), abort));
          if (!ok) break;
          unsigned char* vs = slot(i);
          for (int e = threadIdx.x & 127; e < NT * 8 * Sh::DH; e += 128) {
            const int r = e / (8 * Sh::DH), ch = e % (8 * Sh::DH);
            if (!((blocks >> (r / BS)) & 1u) || th + r >= c1() || th + r < c0())
              *reinterpret_cast<uint4*>(vs + (r / 8) * Sh::ATOM + (ch / 8) * 1024 + tc::sw128(r % 8, ch % 8)) =
                  make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();  // the zeros precede the PV's reads
        }
        tc::fence_before_sync();
        mbar_arrive(p_full + 2 * w + b);
      }
      cnt += n;
      // ---- the streams meet: their PVs are done, their (m, l) at hand, and Q's place is free
      if (ok && n > 0)
        ok = __all_sync(kFull, tc_wait(done + slot_of(w, 1, cnt - 1), phase_of(cnt - 1), abort));
      ml[2 * ROWS * w + row] = n > 0 ? m_ref : -INFINITY;
      ml[2 * ROWS * w + ROWS + row] = n > 0 ? l : 0.f;
      tc::fence_before_sync();
      ok = rows_agree(ok);
      tc::fence_after_sync();
      // the next item's Q, if it is known by now
      const bool early = ok && __all_sync(kFull, mbar_test(info_full + ((k + 1) & 1), ((k + 1) >> 1) & 1));
      if (early && info(k + 1)->ntile > 0) {
        start_q(*info(k + 1));
        if (Q_AS_F16) finish_q();
      }
      // ---- O / l, half of the dims a stream
      {
        const float m0 = ml[row], l0 = ml[ROWS + row], m1 = ml[2 * ROWS + row], l1 = ml[3 * ROWS + row];
        const float M = fmaxf(m0, m1), Ms = M == -INFINITY ? 0.f : M;
        const float f0 = m0 == -INFINITY ? (l0 == 0.f ? 0.f : 1.f) : fast_exp2(m0 - Ms);
        const float f1 = m1 == -INFINITY ? (l1 == 0.f ? 0.f : 1.f) : fast_exp2(m1 - Ms);
        const bool both = m.ntile > 1;  // stream 1 has an O
        l = l0 * f0 + l1 * f1;
        const bool mine = active && parts.in(m.part), direct = parts.direct();
        // 1 / l (FP8 pool: times the value of one V code)
        const float inv = ok && l != 0.f ? (F8 ? p.v_scale : 1.f) / l : 0.f;
        const int part_at = m.part;
        bool fine = true;
        int quad_row[4];  // the rows of this lane's quad that are stored; -1: not
#pragma unroll
        for (int i = 0; i < 4; ++i) quad_row[i] = __shfl_sync(kFull, mine ? orow : -1, (lane & ~3) + i);
        const uint32_t warp_direct = __ballot_sync(kFull, direct), quad_direct = warp_direct >> (lane & ~3);
#pragma unroll 1
        for (int u = 0; u < D / 64; ++u) {
          const int d0 = w * (D / 2) + u * 32;
          uint32_t o[32];
          tc::ld32(ocol + d0, o);
          tc::wait_ld();
          float v[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = __uint_as_float(o[e]);
          if (both) {
            tc::ld32(ocol + 128 + d0, o);
            tc::wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = f0 * v[e] + f1 * __uint_as_float(o[e]);
          }
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            v[e] = ok ? v[e] * inv : 0.f;
            fine = fine && fabsf(v[e]) < INFINITY;
          }
          if (warp_direct) {
            uint32_t o16[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) o16[e] = Elem<T>::pack2(v[2 * e], v[2 * e + 1]);
            quad_transpose(o16, lane);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (quad_row[i] >= 0 && ((quad_direct >> i) & 1u))
                *reinterpret_cast<uint4*>(static_cast<T*>(p.out) + (size_t)quad_row[i] * D + d0 + (lane & 3) * 8) =
                    make_uint4(o16[4 * i], o16[4 * i + 1], o16[4 * i + 2], o16[4 * i + 3]);
          }
          if (~warp_direct) {
#pragma unroll
            for (int g = 0; g < 2; ++g) {
              uint32_t o32[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) o32[e] = __float_as_uint(v[16 * g + e]);
              quad_transpose(o32, lane);
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (quad_row[i] >= 0 && !((quad_direct >> i) & 1u))
                  *reinterpret_cast<uint4*>(p.part_o + ((size_t)quad_row[i] * p.max_partitions + part_at) * D + d0 +
                                            16 * g + (lane & 3) * 4) =
                      make_uint4(o32[4 * i], o32[4 * i + 1], o32[4 * i + 2], o32[4 * i + 3]);
            }
          }
        }
        if (mine && !direct && w == 0) {
          p.part_m[(size_t)orow * p.max_partitions + part_at] = ok ? M : -INFINITY;
          p.part_l[(size_t)orow * p.max_partitions + part_at] = ok ? l : 0.f;
        }
        // Rows that came out non-finite by a masked key's value (not by NaN scores of their own): this half again, on
        // the whole warp. A value that a row sees is its own, so a NaN in the cache costs one look over the item's
        // values.
        __syncwarp();  // (a redone row is stored over)
        uint32_t redo = __ballot_sync(
            kFull, mine && !fine && ok && l == l && (lo > m.c0 || hi < m.c1 || m.c1 > node0));
        if (redo) {
          int bad0, bad1;
          bad_values<C, D>(p, m.s, m.kvh, m.c0, m.c1, BS, lane, bad0, bad1, abort + 1);
          redo &= __ballot_sync(kFull, bad0 > bad1 || lo > bad0 || hi <= bad1 || bad1 >= node0);
        }
        for (; redo; redo &= redo - 1) {
          const int src = __ffs(redo) - 1, tok0 = part_at * P;
          const int rlo = __shfl_sync(kFull, lo, src), rhi = __shfl_sync(kFull, hi, src);
          const int rh = __shfl_sync(kFull, h, src), at = __shfl_sync(kFull, orow, src);
          const bool rdirect = __shfl_sync(kFull, (int)direct, src);
          float rm, rl, o[D / 32];
          scored_row<T, C, D, true>(p, sc, at, m.s, rh, node0, max(rlo, tok0), min(rhi, tok0 + P), BS, lane, rm, rl, o,
                                    abort + 1);
          if ((lane >> 4) == w) {  // (D / 32 dims a lane)
            constexpr int DPL = D / 32;
            if (rdirect) {
              uint32_t* dst =
                  reinterpret_cast<uint32_t*>(static_cast<T*>(p.out) + (size_t)at * D + lane * DPL);
#pragma unroll
              for (int e = 0; e < DPL / 2; ++e) dst[e] = Elem<T>::pack2(o[2 * e], o[2 * e + 1]);
            } else {
              float* dst = p.part_o + ((size_t)at * p.max_partitions + part_at) * D + lane * DPL;
#pragma unroll
              for (int e = 0; e < DPL; ++e) dst[e] = o[e];
            }
          }
          __syncwarp();
        }
      }
      bool going = ok;
      if (ok && !early) {
        going = wait_item(k + 1);
        if (going && info(k + 1)->ntile > 0) {
          start_q(*info(k + 1));
          if (Q_AS_F16) finish_q();
        }
      }
      if (!Q_AS_F16 && going && info(k + 1)->ntile > 0) finish_q();
      // both streams go on together (both O have been read), or leave together
      tc::fence_before_sync();
      ok = rows_agree(ok && going);
      tc::fence_after_sync();
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

template <typename T, int D, int BS, bool F8, bool CAP>
cudaError_t launch_tree_mode(const DecodeParams& p, const ScoreParams& sc, const CUtensorMap& kmap,
                             const CUtensorMap& vmap, int num_seqs, cudaStream_t stream) {
  using Sh = TreeTcShape<T, D, BS, F8>;
  auto kern = pkv_tree_tc_kernel<T, D, BS, F8, CAP>;
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

template <typename T, int D, bool F8>
cudaError_t dispatch_tree_block(const DecodeParams& p, const ScoreParams& sc, const CUtensorMap& kmap,
                                const CUtensorMap& vmap, int block_size, int num_seqs, cudaStream_t stream) {
  auto of = [&](auto bs) {
    constexpr int BS = decltype(bs)::value;
    return sc.cap_out != 0.f ? launch_tree_mode<T, D, BS, F8, true>(p, sc, kmap, vmap, num_seqs, stream)
                             : launch_tree_mode<T, D, BS, F8, false>(p, sc, kmap, vmap, num_seqs, stream);
  };
  if (block_size == 16) return of(std::integral_constant<int, 16>{});
  if (block_size == 8) return of(std::integral_constant<int, 8>{});
  if (block_size == 32) return of(std::integral_constant<int, 32>{});
  return cudaErrorInvalidValue;
}

template <typename T>
cudaError_t dispatch_tree_tc(const DecodeParams& p, const ScoreParams& sc, const CUtensorMap& kmap,
                             const CUtensorMap& vmap, bool fp8, int head_dim, int block_size, int num_seqs,
                             cudaStream_t stream) {
  if (fp8) return dispatch_tree_block<T, 128, true>(p, sc, kmap, vmap, block_size, num_seqs, stream);
  if (head_dim == 128) return dispatch_tree_block<T, 128, false>(p, sc, kmap, vmap, block_size, num_seqs, stream);
  if (head_dim == 64) return dispatch_tree_block<T, 64, false>(p, sc, kmap, vmap, block_size, num_seqs, stream);
  return cudaErrorInvalidValue;
}

}  // namespace pkv
