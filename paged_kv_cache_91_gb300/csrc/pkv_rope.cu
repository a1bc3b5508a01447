// paged_kv_write_rope: the queries' and keys' norm per head and rotation, fused with the cache write. One pass: every
// row is read once, held in registers as fp32, and written once in its final type.
//
// Per row x of D values (a token's head), with w and the token's angles c, s:
//   y = x * rsqrt(mean(x^2) + eps) * w,  (y_a, y_b) <- (y_a c - y_b s, y_b c + y_a s) for the pairs of the rotary dims
// D / 8 lanes hold a row, two groups of 4 consecutive dims (8 bytes) each. Where halves are paired, (i, i + R / 2), a
// lane of the first R / 8 takes the dims 4 c .. and R / 2 + 4 c .., so that both of a pair are its own: no exchange, and
// four cosines and sines for its eight dims. The other lanes, and all of them where neighbours are paired, take eight
// dims in a row.
//
// Bound by HBM once the batch is large, with the issue slots close behind (16384 tokens, 32/8 heads, bf16: 72 us, 5.7 TB/s,
// 84 % of the copy rate; issue 73 %; into an E4M3 pool, whose rows are divided and converted too, 80 us of 56); a step's
// 256 tokens into an E4M3 pool take 4.7 us replayed from a graph, latency. At 64 registers a thread all but one of the
// forms spill: 52 bytes stored and 76 loaded in the bf16 one above, up to 84 and 168 for f16 rows into an E4M3 pool.
// On the way there (16384 tokens, with the launch, us): eight dims in a row a lane with the partner's values by shuffle 122,
// pairs within a lane 107, 64 registers a thread for 8 CTAs an SM 98, packed arithmetic and loops of their own for
// queries, keys and values 88.
#include <math.h>
#include <stdint.h>

#include "paged_kv.h"
#include "pkv_common.cuh"
#include "pkv_f32x2.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

struct RopeParams {
  unsigned char* query_out;
  const unsigned char *query, *key, *value;
  unsigned char *key_cache, *value_cache;
  const int64_t* slot_mapping;
  const int32_t* positions;
  const float* cos_sin;
  const float *q_weight, *k_weight;
  unsigned* err;
  long long query_stride, key_stride, value_stride;  // elements between tokens
  long long num_slots;
  int num_heads, num_kv_heads, block_size;
  int max_position, rotary_dim;
  int parts;  // CTAs that share a token's rows
  float eps, k_scale, v_scale;
};

constexpr int kRopeThreads = 128;
constexpr int kRopeUnroll = 4;   // query rows that a thread has in flight
constexpr int kRopeCtas = 8;     // CTAs an SM holds (64 registers a thread)
constexpr int kRopeFill = 608;   // CTAs that fill the GPU: four an SM

// A lane's part of a 16-bit row: its two groups of four dims.
struct Part {
  uint2 a, b;
};

__device__ __forceinline__ Part load_part(const unsigned char* row, int da, int db) {
  return {__ldg(reinterpret_cast<const uint2*>(row + da * 2)), __ldg(reinterpret_cast<const uint2*>(row + db * 2))};
}
// The same of a query row, which the call may write in place: not through the read-only path, which holds only what a
// kernel does not write.
__device__ __forceinline__ Part load_query(const unsigned char* row, int da, int db) {
  return {*reinterpret_cast<const uint2*>(row + da * 2), *reinterpret_cast<const uint2*>(row + db * 2)};
}
__device__ __forceinline__ void store_part(unsigned char* row, int da, int db, const Part& y) {
  *reinterpret_cast<uint2*>(row + da * 2) = y.a;
  *reinterpret_cast<uint2*>(row + db * 2) = y.b;
}

template <typename T>
__device__ __forceinline__ f32x2 widen2(uint32_t w) {
  const float2 f = Elem<T>::to_float2(w);
  return pair2(f.x, f.y);
}
template <typename T>
__device__ __forceinline__ uint32_t pack2(f32x2 v) {
  float a, b;
  unpair2(v, a, b);
  return Elem<T>::pack2(a, b);
}

// E4M3(x / scale) of four values, as paged_kv_write_fp8 rounds it.
__device__ __forceinline__ uint32_t codes4(f32x2 p, f32x2 q, float scale) {
  float a, b, c, d;
  unpair2(p, a, b);
  unpair2(q, c, d);
  const uint32_t lo =
      __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(a, scale), __fdiv_rn(b, scale)), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi =
      __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(c, scale), __fdiv_rn(d, scale)), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

// What a lane holds for its dims of every row of a token: the norm's weights, and the cosines and sines of its four
// pairs (halves: as two pairs of pairs; neighbours: one by one).
struct Turn {
  f32x2 w[4];
  bool normed, turned;
  float4 cs, sn;
};

__device__ __forceinline__ void load_weights(Turn& t, const float* w, int da, int db) {
  t.normed = w != nullptr;
  if (!w) return;
  const float4 a = __ldg(reinterpret_cast<const float4*>(w + da)), b = __ldg(reinterpret_cast<const float4*>(w + db));
  t.w[0] = pair2(a.x, a.y);
  t.w[1] = pair2(a.z, a.w);
  t.w[2] = pair2(b.x, b.y);
  t.w[3] = pair2(b.z, b.w);
}

// The row of which this lane holds y: normed and turned, in fp32. All lanes of the warp take part.
template <typename T, int D, bool INTERLEAVED>
__device__ __forceinline__ void norm_and_turn(const Part& y, const Turn& t, float eps, f32x2 (&x)[4]) {
  x[0] = widen2<T>(y.a.x);
  x[1] = widen2<T>(y.a.y);
  x[2] = widen2<T>(y.b.x);
  x[3] = widen2<T>(y.b.y);
  if (t.normed) {
    float s0, s1;
    unpair2(fma2(x[3], x[3], fma2(x[2], x[2], fma2(x[1], x[1], mul2(x[0], x[0])))), s0, s1);
    float sum = s0 + s1;
#pragma unroll
    for (int o = 1; o < D / 8; o <<= 1) sum += __shfl_xor_sync(kFull, sum, o);
    const float inv = rsqrtf(sum * (1.f / D) + eps);
    const f32x2 inv2 = pair2(inv, inv);
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = mul2(mul2(x[e], inv2), t.w[e]);
  }
  if (t.turned) {
    if constexpr (INTERLEAVED) {
      const float co[4] = {t.cs.x, t.cs.y, t.cs.z, t.cs.w}, si[4] = {t.sn.x, t.sn.y, t.sn.z, t.sn.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float a, b;
        unpair2(x[e], a, b);
        x[e] = pair2(a * co[e] - b * si[e], b * co[e] + a * si[e]);
      }
    } else {
      const f32x2 co[2] = {pair2(t.cs.x, t.cs.y), pair2(t.cs.z, t.cs.w)};
      const f32x2 si[2] = {pair2(t.sn.x, t.sn.y), pair2(t.sn.z, t.sn.w)};
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const f32x2 a = x[e], b = x[2 + e];
        x[e] = sub2(mul2(a, co[e]), mul2(b, si[e]));
        x[2 + e] = fma2(b, co[e], mul2(a, si[e]));
      }
    }
  }
}

// A CTA takes 1 / parts of one token's rows, a group of D / 8 lanes a row: of the queries, the keys and the values, in
// loops of their own.
template <typename T, int D, bool F8, bool INTERLEAVED>
__global__ void __launch_bounds__(kRopeThreads, kRopeCtas) pkv_write_rope_kernel(const RopeParams p) {
  pdl_begin();
  constexpr int LPR = D / 8, RG = kRopeThreads / LPR;  // lanes a row, rows at a time
  const int t = blockIdx.x / p.parts, part = blockIdx.x % p.parts;
  const int c = threadIdx.x % LPR;
  const int H = p.num_heads, Hkv = p.num_kv_heads, R = p.rotary_dim;
  Turn turn;
  turn.turned = c * 8 < R;
  const int da = INTERLEAVED || !turn.turned ? 8 * c : 4 * c;  // the lane's first dims
  const int db = da + (INTERLEAVED || !turn.turned ? 4 : R / 2);
  const int first = part * RG, g = threadIdx.x / LPR, step = RG * p.parts;
  const unsigned char* q = p.query + ((size_t)t * p.query_stride + (size_t)(first + g) * D) * 2;
  const unsigned char* k = p.key + ((size_t)t * p.key_stride + (size_t)(first + g) * D) * 2;
  const unsigned char* v = p.value + ((size_t)t * p.value_stride + (size_t)(first + g) * D) * 2;
  // the first rows load beside the slot and the position, which they do not depend on
  Part q_in[kRopeUnroll], k_in, v_in;
#pragma unroll
  for (int u = 0; u < kRopeUnroll; ++u)
    if (first + g + u * step < H) q_in[u] = load_query(q + (size_t)u * step * D * 2, da, db);
  if (first + g < Hkv) {
    k_in = load_part(k, da, db);
    v_in = load_part(v, da, db);
  }
  const long long slot = __ldg(p.slot_mapping + t);
  const int pos = R ? __ldg(p.positions + t) : 0;
  const bool lost = R && (unsigned)pos >= (unsigned)p.max_position;  // no angles
  const bool stored = slot >= 0 && slot < p.num_slots && !lost;
  if (part == 0 && threadIdx.x == 0) {
    if (slot >= p.num_slots) atomicOr(p.err, PKV_DEVERR_SLOT);
    if (lost && slot >= 0) atomicOr(p.err, PKV_DEVERR_CONTEXT);
  }
  turn.cs = turn.sn = make_float4(0.f, 0.f, 0.f, 0.f);
  if (turn.turned && !lost) {  // of pairs 4 c ..
    const float4* row = reinterpret_cast<const float4*>(p.cos_sin + (size_t)pos * R);
    turn.cs = __ldg(row + c);
    turn.sn = __ldg(row + R / 8 + c);
  }
  if (stored) {
    constexpr int EB = F8 ? 1 : 2;
    const long long blk = slot / p.block_size, off = slot - blk * p.block_size;
    const size_t head = (size_t)p.block_size * D * EB;  // bytes between heads of a block
    const size_t at = ((size_t)blk * Hkv + first + g) * head + (size_t)off * D * EB;
    unsigned char *kc = p.key_cache + at, *vc = p.value_cache + at;
    load_weights(turn, p.k_weight, da, db);
    for (int base = first; base < Hkv; base += step) {
      const bool mine = base + g < Hkv;
      f32x2 x[4];
      norm_and_turn<T, D, INTERLEAVED>(k_in, turn, p.eps, x);
      if (mine) {
        if constexpr (F8) {
          *reinterpret_cast<uint32_t*>(kc + da) = codes4(x[0], x[1], p.k_scale);
          *reinterpret_cast<uint32_t*>(kc + db) = codes4(x[2], x[3], p.k_scale);
          *reinterpret_cast<uint32_t*>(vc + da) = codes4(widen2<T>(v_in.a.x), widen2<T>(v_in.a.y), p.v_scale);
          *reinterpret_cast<uint32_t*>(vc + db) = codes4(widen2<T>(v_in.b.x), widen2<T>(v_in.b.y), p.v_scale);
        } else {
          store_part(kc, da, db,
                     {make_uint2(pack2<T>(x[0]), pack2<T>(x[1])), make_uint2(pack2<T>(x[2]), pack2<T>(x[3]))});
          store_part(vc, da, db, v_in);
        }
      }
      k += (size_t)step * D * 2;
      v += (size_t)step * D * 2;
      kc += step * head;
      vc += step * head;
      if (base + step + g < Hkv) {
        k_in = load_part(k, da, db);
        v_in = load_part(v, da, db);
      }
    }
  }
  load_weights(turn, p.q_weight, da, db);
  unsigned char* out = p.query_out + ((size_t)t * H + first + g) * D * 2;
  // (all threads of a warp go through the same number of rounds, for the shuffles)
  for (int base = first; base < H; base += kRopeUnroll * step) {
#pragma unroll
    for (int u = 0; u < kRopeUnroll; ++u) {
      if (base + u * step >= H) break;
      const int r = base + u * step + g;
      const Part y = q_in[u];
      if (r + kRopeUnroll * step < H) q_in[u] = load_query(q + (size_t)(kRopeUnroll + u) * step * D * 2, da, db);
      f32x2 x[4];
      norm_and_turn<T, D, INTERLEAVED>(y, turn, p.eps, x);
      Part z = {make_uint2(pack2<T>(x[0]), pack2<T>(x[1])), make_uint2(pack2<T>(x[2]), pack2<T>(x[3]))};
      if (lost) z = {make_uint2(0u, 0u), make_uint2(0u, 0u)};
      if (r < H) store_part(out + (size_t)u * step * D * 2, da, db, z);
    }
    q += (size_t)kRopeUnroll * step * D * 2;
    out += (size_t)kRopeUnroll * step * D * 2;
  }
}

bool aligned(const void* ptr, uintptr_t n) { return (reinterpret_cast<uintptr_t>(ptr) & (n - 1)) == 0; }

template <typename T, int D, bool F8>
cudaError_t launch_rope(const RopeParams& p, bool interleaved, unsigned grid, cudaStream_t stream) {
  return interleaved
             ? launch_kernel(pkv_write_rope_kernel<T, D, F8, true>, dim3(grid), dim3(kRopeThreads), 0, stream, p)
             : launch_kernel(pkv_write_rope_kernel<T, D, F8, false>, dim3(grid), dim3(kRopeThreads), 0, stream, p);
}

// Everything a call passes, under the header's names.
struct RopeCall {
  void* query_out;
  const void *query, *key, *value;
  void *key_cache, *value_cache;
  const int64_t* slot_mapping;
  const int32_t* positions;
  const float* cos_sin;
  int32_t max_position, rotary_dim, interleaved;
  const float *q_weight, *k_weight;
  float eps;
  int32_t num_tokens;
  int64_t query_stride, key_stride, value_stride;
  int32_t num_heads, num_kv_heads, head_dim, block_size, num_blocks;
  pkv_dtype_t dtype;
  bool fp8;
  float k_scale, v_scale;
  cudaStream_t stream;
};

pkv_status_t rope_impl(const RopeCall& c) {
  set_last_error_message("");
  if (c.num_tokens < 0) return fail(PKV_ERR_INVALID_ARG, "num_tokens < 0");
  if (c.dtype != PKV_F16 && c.dtype != PKV_BF16) return fail(PKV_ERR_INVALID_ARG, "unknown dtype %d", (int)c.dtype);
  if (c.num_heads <= 0 || c.num_kv_heads <= 0 || c.num_blocks <= 0)
    return fail(PKV_ERR_INVALID_ARG, "num_heads, num_kv_heads and num_blocks must be > 0");
  if (c.num_heads > 65535 || c.num_kv_heads > 65535)
    return fail(PKV_ERR_UNSUPPORTED, "num_heads and num_kv_heads must be <= 65535");
  if (c.head_dim != 64 && c.head_dim != 128)
    return fail(PKV_ERR_UNSUPPORTED, "head_dim %d (supported: 64, 128)", c.head_dim);
  if (c.block_size != 8 && c.block_size != 16 && c.block_size != 32)
    return fail(PKV_ERR_UNSUPPORTED, "block_size %d (supported: 8, 16, 32)", c.block_size);
  if (c.rotary_dim < 0 || c.rotary_dim > c.head_dim)
    return fail(PKV_ERR_INVALID_ARG, "rotary_dim %d outside [0, head_dim %d]", c.rotary_dim, c.head_dim);
  if (c.rotary_dim % 16) return fail(PKV_ERR_UNSUPPORTED, "rotary_dim %d must be a multiple of 16", c.rotary_dim);
  if (c.max_position < 0) return fail(PKV_ERR_INVALID_ARG, "max_position < 0");
  if (!(isfinite(c.eps) && c.eps >= 0.f)) return fail(PKV_ERR_INVALID_ARG, "eps must be finite and >= 0");
  if (c.fp8 && !(isfinite(c.k_scale) && isfinite(c.v_scale) && c.k_scale > 0.f && c.v_scale > 0.f))
    return fail(PKV_ERR_INVALID_ARG, "k_scale and v_scale must be finite and > 0");
  const int64_t q_row = (int64_t)c.num_heads * c.head_dim, kv_row = (int64_t)c.num_kv_heads * c.head_dim;
  if (c.query_stride < q_row || c.key_stride < kv_row || c.value_stride < kv_row)
    return fail(PKV_ERR_INVALID_ARG, "a stride is shorter than a token's rows");
  if (c.query_stride % 8 || c.key_stride % 8 || c.value_stride % 8)
    return fail(PKV_ERR_INVALID_ARG, "strides must be multiples of 8 elements");
  if (c.query_stride > (1LL << 31) || c.key_stride > (1LL << 31) || c.value_stride > (1LL << 31))
    return fail(PKV_ERR_UNSUPPORTED, "strides must be <= 2^31");
  if (c.num_tokens == 0) return PKV_OK;
  if (!c.query_out || !c.query || !c.key || !c.value || !c.key_cache || !c.value_cache || !c.slot_mapping ||
      (c.rotary_dim > 0 && (!c.positions || !c.cos_sin)))
    return fail(PKV_ERR_INVALID_ARG, "null pointer argument");
  if (!aligned(c.query_out, 16) || !aligned(c.query, 16) || !aligned(c.key, 16) || !aligned(c.value, 16) ||
      !aligned(c.key_cache, 16) || !aligned(c.value_cache, 16) || !aligned(c.cos_sin, 16) ||
      !aligned(c.q_weight, 16) || !aligned(c.k_weight, 16))
    return fail(PKV_ERR_INVALID_ARG, "query_out, query, key, value, caches, cos_sin and weights must be 16-byte aligned");
  // query_out's rows are written while other CTAs read: it may be query itself, but not lie across it
  {
    const uintptr_t out = reinterpret_cast<uintptr_t>(c.query_out);
    const size_t out_bytes = (size_t)c.num_tokens * q_row * 2;
    auto apart = [&](const void* at, int64_t stride, int64_t row) {
      const uintptr_t a = reinterpret_cast<uintptr_t>(at);
      const size_t bytes = ((size_t)(c.num_tokens - 1) * stride + row) * 2;
      return out + out_bytes <= a || a + bytes <= out;
    };
    if (!apart(c.query, c.query_stride, q_row) && !(c.query_out == c.query && c.query_stride == q_row))
      return fail(PKV_ERR_INVALID_ARG, "query_out must be query itself (contiguous) or not overlap it");
    if (!apart(c.key, c.key_stride, kv_row) || !apart(c.value, c.value_stride, kv_row))
      return fail(PKV_ERR_INVALID_ARG, "query_out must not overlap key or value");
  }
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  RopeParams p{};
  p.query_out = static_cast<unsigned char*>(c.query_out);
  p.query = static_cast<const unsigned char*>(c.query);
  p.key = static_cast<const unsigned char*>(c.key);
  p.value = static_cast<const unsigned char*>(c.value);
  p.key_cache = static_cast<unsigned char*>(c.key_cache);
  p.value_cache = static_cast<unsigned char*>(c.value_cache);
  p.slot_mapping = c.slot_mapping;
  p.positions = c.positions;
  p.cos_sin = c.cos_sin;
  p.q_weight = c.q_weight;
  p.k_weight = c.k_weight;
  p.err = device_error_word(dev);
  if (!p.err) return fail(PKV_ERR_CUDA, "device error word unavailable on device %d", dev);
  p.query_stride = c.query_stride;
  p.key_stride = c.key_stride;
  p.value_stride = c.value_stride;
  p.num_slots = (long long)c.num_blocks * c.block_size;
  p.num_heads = c.num_heads;
  p.num_kv_heads = c.num_kv_heads;
  p.block_size = c.block_size;
  p.max_position = c.max_position;
  p.rotary_dim = c.rotary_dim;
  p.eps = c.eps;
  p.k_scale = c.k_scale;
  p.v_scale = c.v_scale;
  // a token's rows are shared by several CTAs while those would not fill the GPU
  const int at_once = kRopeThreads / (c.head_dim / 8);
  const long long rounds = ((long long)(c.num_heads > c.num_kv_heads ? c.num_heads : c.num_kv_heads) + at_once - 1) / at_once;
  long long parts = (kRopeFill + c.num_tokens - 1) / c.num_tokens;
  if (parts > rounds) parts = rounds;
  p.parts = (int)parts;
  const unsigned grid = (unsigned)(parts * c.num_tokens);  // (one part a token from kRopeFill tokens on)
  const bool il = c.interleaved != 0;
  auto of = [&](auto type) {
    using T = decltype(type);
    if (c.head_dim == 128)
      return c.fp8 ? launch_rope<T, 128, true>(p, il, grid, c.stream) : launch_rope<T, 128, false>(p, il, grid, c.stream);
    return c.fp8 ? launch_rope<T, 64, true>(p, il, grid, c.stream) : launch_rope<T, 64, false>(p, il, grid, c.stream);
  };
  e = c.dtype == PKV_F16 ? of(__half{}) : of(__nv_bfloat16{});
  if (e != cudaSuccess) return cuda_fail(e, "paged_kv_write_rope launch");
  return PKV_OK;
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" {

pkv_status_t paged_kv_write_rope(void* query_out, const void* query, const void* key, const void* value,
                                 void* key_cache, void* value_cache, const int64_t* slot_mapping,
                                 const int32_t* positions, const float* cos_sin, int32_t max_position,
                                 int32_t rotary_dim, int32_t interleaved, const float* q_weight,
                                 const float* k_weight, float eps, int32_t num_tokens, int64_t query_stride,
                                 int64_t key_stride, int64_t value_stride, int32_t num_heads, int32_t num_kv_heads,
                                 int32_t head_dim, int32_t block_size, int32_t num_blocks, pkv_dtype_t dtype,
                                 cudaStream_t stream) {
  return rope_impl({query_out, query, key, value, key_cache, value_cache, slot_mapping, positions, cos_sin,
                    max_position, rotary_dim, interleaved, q_weight, k_weight, eps, num_tokens, query_stride,
                    key_stride, value_stride, num_heads, num_kv_heads, head_dim, block_size, num_blocks, dtype, false,
                    1.f, 1.f, stream});
}

pkv_status_t paged_kv_write_rope_fp8(void* query_out, const void* query, const void* key, const void* value,
                                     void* key_cache, void* value_cache, const int64_t* slot_mapping,
                                     const int32_t* positions, const float* cos_sin, int32_t max_position,
                                     int32_t rotary_dim, int32_t interleaved, const float* q_weight,
                                     const float* k_weight, float eps, int32_t num_tokens, int64_t query_stride,
                                     int64_t key_stride, int64_t value_stride, int32_t num_heads,
                                     int32_t num_kv_heads, int32_t head_dim, int32_t block_size, int32_t num_blocks,
                                     pkv_dtype_t dtype, float k_scale, float v_scale, cudaStream_t stream) {
  return rope_impl({query_out, query, key, value, key_cache, value_cache, slot_mapping, positions, cos_sin,
                    max_position, rotary_dim, interleaved, q_weight, k_weight, eps, num_tokens, query_stride,
                    key_stride, value_stride, num_heads, num_kv_heads, head_dim, block_size, num_blocks, dtype, true,
                    k_scale, v_scale, stream});
}

}  // extern "C"
