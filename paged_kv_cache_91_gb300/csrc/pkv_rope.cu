// paged_kv_write_rope: the queries' and keys' norm per head and rotation, fused with the cache write. One pass: every
// row is read once, held in registers as fp32, and written once in its final type.
//
// Per row x of D values (a token's head), with w and the token's angles c, s:
//   y = x * rsqrt(mean(x^2) + eps) * w,  (y_a, y_b) <- (y_a c - y_b s, y_b c + y_a s) for the pairs of the rotary dims
// D / 8 lanes hold a row, 8 consecutive dims (16 bytes) each, so a warp moves whole 128- or 256-byte rows. With halves
// paired (i, i + R / 2) a lane's partners are all in one other lane (R / 2 is a multiple of 8): one shuffle a value.
#include <math.h>
#include <stdint.h>

#include "paged_kv.h"
#include "pkv_common.cuh"
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
constexpr int kRopeUnroll = 4;   // rows that a thread has in flight
constexpr int kRopeFill = 608;   // CTAs that fill the GPU: four an SM

template <typename T>
__device__ __forceinline__ void widen8(const uint4& r, float (&x)[8]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 f = Elem<T>::to_float2(w[e]);
    x[2 * e] = f.x;
    x[2 * e + 1] = f.y;
  }
}

template <typename T>
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(Elem<T>::pack2(x[0], x[1]), Elem<T>::pack2(x[2], x[3]), Elem<T>::pack2(x[4], x[5]),
                    Elem<T>::pack2(x[6], x[7]));
}

// E4M3(x / scale), as paged_kv_write_fp8 rounds it.
__device__ __forceinline__ uint2 codes8(const float (&x)[8], float scale) {
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e)
    w[e] = __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(x[2 * e], scale), __fdiv_rn(x[2 * e + 1], scale)),
                                    __NV_SATFINITE, __NV_E4M3);
  return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}

// A CTA takes 1 / parts of one token's rows: queries, then keys, then values, a group of D / 8 lanes a row.
template <typename T, int D, bool F8, bool INTERLEAVED>
__global__ void __launch_bounds__(kRopeThreads) pkv_write_rope_kernel(const RopeParams p) {
  pdl_begin();
  constexpr int LPR = D / 8, RG = kRopeThreads / LPR;  // lanes a row, rows at a time
  const int t = blockIdx.x / p.parts, part = blockIdx.x % p.parts;
  const int c = threadIdx.x % LPR, d0 = c * 8;
  const int H = p.num_heads, Hkv = p.num_kv_heads, R = p.rotary_dim;
  const int rows = H + 2 * Hkv, step = RG * p.parts;
  const unsigned char* q = p.query + (size_t)t * p.query_stride * 2;
  const unsigned char* k = p.key + (size_t)t * p.key_stride * 2;
  const unsigned char* v = p.value + (size_t)t * p.value_stride * 2;
  auto load = [&](int r) {
    const unsigned char* src = r < H ? q + (size_t)r * D * 2
                               : r < H + Hkv ? k + (size_t)(r - H) * D * 2 : v + (size_t)(r - H - Hkv) * D * 2;
    return __ldg(reinterpret_cast<const uint4*>(src) + c);
  };
  // the first rows load beside the slot and the position, which they do not depend on
  const int r0 = part * RG + threadIdx.x / LPR;
  uint4 raw[kRopeUnroll];
#pragma unroll
  for (int u = 0; u < kRopeUnroll; ++u)
    if (r0 + u * step < rows) raw[u] = load(r0 + u * step);
  const long long slot = __ldg(p.slot_mapping + t);
  const int pos = R ? __ldg(p.positions + t) : 0;
  const bool lost = R && (unsigned)pos >= (unsigned)p.max_position;  // no angles
  const bool stored = slot >= 0 && slot < p.num_slots && !lost;
  if (part == 0 && threadIdx.x == 0) {
    if (slot >= p.num_slots) atomicOr(p.err, PKV_DEVERR_SLOT);
    if (lost && slot >= 0) atomicOr(p.err, PKV_DEVERR_CONTEXT);
  }
  // this lane's angles: of pairs i0 .. (halves: 8 of them, the lane holds one side; interleaved: 4, both sides)
  const bool turned = d0 < R;
  const bool second = !INTERLEAVED && d0 >= R / 2;
  float cs[8], sn[8];
  if (turned && !lost) {
    const float* row = p.cos_sin + (size_t)pos * R;
    if constexpr (INTERLEAVED) {
      const float4 a = __ldg(reinterpret_cast<const float4*>(row + d0 / 2));
      const float4 b = __ldg(reinterpret_cast<const float4*>(row + R / 2 + d0 / 2));
      cs[0] = a.x; cs[1] = a.y; cs[2] = a.z; cs[3] = a.w;
      sn[0] = b.x; sn[1] = b.y; sn[2] = b.z; sn[3] = b.w;
    } else {
      const int i0 = second ? d0 - R / 2 : d0;
      load8(row + i0, cs);
      load8(row + R / 2 + i0, sn);
      if (!second)
#pragma unroll
        for (int e = 0; e < 8; ++e) sn[e] = -sn[e];  // y_a c - y_b s; the other side is y_b c + y_a s
    }
  }
  const int lane = threadIdx.x & 31;
  const int partner = (lane & ~(LPR - 1)) | (turned ? (second ? c - R / 16 : c + R / 16) : c);
  const long long blk = stored ? slot / p.block_size : 0, off = stored ? slot - blk * p.block_size : 0;
  // (all threads of a warp go through the same number of rounds, for the shuffles)
  for (int base = part * RG; base < rows; base += kRopeUnroll * step) {
#pragma unroll
    for (int u = 0; u < kRopeUnroll; ++u) {
      if (base + u * step >= rows) break;
      const int r = base + u * step + threadIdx.x / LPR;
      const bool row = r < rows, is_q = r < H, is_v = r >= H + Hkv;
      const uint4 x16 = raw[u];
      if (r + kRopeUnroll * step < rows) raw[u] = load(r + kRopeUnroll * step);
      float x[8];
      widen8<T>(x16, x);
      const float* w = is_q ? p.q_weight : p.k_weight;
      float sum = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) sum = fmaf(x[e], x[e], sum);
#pragma unroll
      for (int o = 1; o < LPR; o <<= 1) sum += __shfl_xor_sync(kFull, sum, o);
      if (w && !is_v) {
        const float inv = rsqrtf(sum * (1.f / D) + p.eps);
        float wt[8];
        load8(w + d0, wt);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = x[e] * inv * wt[e];
      }
      if constexpr (INTERLEAVED) {
        if (turned && !is_v) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float a = x[2 * e], b = x[2 * e + 1];
            x[2 * e] = a * cs[e] - b * sn[e];
            x[2 * e + 1] = b * cs[e] + a * sn[e];
          }
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float other = __shfl_sync(kFull, x[e], partner);
          if (turned && !is_v) x[e] = x[e] * cs[e] + other * sn[e];
        }
      }
      if (!row) continue;
      if (is_q) {
        const uint4 y = lost ? make_uint4(0u, 0u, 0u, 0u) : pack8<T>(x);
        reinterpret_cast<uint4*>(p.query_out + ((size_t)t * H + r) * D * 2)[c] = y;
      } else if (stored) {
        const int h = is_v ? r - H - Hkv : r - H;
        unsigned char* pool = is_v ? p.value_cache : p.key_cache;
        const size_t at = (((size_t)blk * Hkv + h) * p.block_size + off) * D;
        if constexpr (F8)
          reinterpret_cast<uint2*>(pool + at)[c] = codes8(x, is_v ? p.v_scale : p.k_scale);
        else
          reinterpret_cast<uint4*>(pool + at * 2)[c] = is_v ? x16 : pack8<T>(x);
      }
    }
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
  const long long rounds = ((long long)c.num_heads + 2 * c.num_kv_heads + at_once - 1) / at_once;
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
