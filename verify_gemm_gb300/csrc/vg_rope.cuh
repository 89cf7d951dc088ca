// vg_rope.cuh -- what the kernels that turn q and k and append k and v to the
// cache share: the angles, a token's addresses, 16 elements at a time, and
// the calls' checks.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "vg_cache.h"

namespace vg {
namespace {

struct RopeParams {
  const void *q, *k, *v;
  void *q_out, *ck, *cv;
  int64_t qs[3], ks[3], vs[3];     // batch, node, head
  int64_t cks[3], cvs[3];          // page, token, head
  const double *inv_freq;
  const int32_t *lens, *depth, *counts;
  CacheView cache;
  int64_t tokens;                  // batch * n
  int n, hq, hkv, d, rot;
  float factor, k_inv, v_inv;       // E4M3: 1 / scale
};

__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
__device__ __forceinline__ void from_f(__nv_bfloat16 &o, float x) { o = __float2bfloat16_rn(x); }
__device__ __forceinline__ void from_f(__half &o, float x) { o = __float2half_rn(x); }
__device__ __forceinline__ void from_f(__nv_fp8_e4m3 &o, float x) {
  o.__x = __nv_cvt_float_to_fp8(x, __NV_SATFINITE, __NV_E4M3);
}

// Frequency j, m 2^e with an m of 53 bits, as a fraction of a turn in units of
// 2^-64: m (2^66 / 2 pi) 2^(e - 2), of which whole turns fall off at the top.
// (Integers: this GPU does two FP64 operations a clock and SM, and a block of
// few heads waited for them.)
__device__ __forceinline__ uint64_t turn_step(const RopeParams &p, int j) {
  const uint64_t bits = uint64_t(__double_as_longlong(p.inv_freq[j]));
  const int field = int(bits >> 52 & 0x7FF);
  if (field == 0) return 0;                                  // below 2^-1022
  const uint64_t m = (bits & ((uint64_t(1) << 52) - 1)) | uint64_t(1) << 52;
  constexpr uint64_t kTurn = 0xA2F9836E4E441529ull;           // 2^66 / 2 pi
  const uint64_t lo = m * kTurn, hi = __umul64hi(m, kTurn);
  const int right = 1077 - field;                            // 2 - e
  const uint64_t r = right <= 0    ? (right > -64 ? lo << -right : 0)
                     : right < 64  ? hi << (64 - right) | lo >> right
                     : right < 128 ? hi >> (right - 64)
                                   : 0;
  return bits >> 63 ? -r : r;
}
// Cosine and sine, times the factor, of the angle position * step: of its
// upper 32 bits, 2^-32 turns.
__device__ __forceinline__ float2 turn(const RopeParams &p, int64_t position, uint64_t step) {
  const int32_t at = int32_t(uint64_t(position) * step >> 32);
  float s, c;
  sincospif(__int2float_rn(at) * 4.6566128730773926e-10f, &s, &c);   // * 2^-31: half turns
  return make_float2(c * p.factor, s * p.factor);
}

// What a token's append needs, worked out once by its block.
struct Token {
  int64_t q, k, v, out, ck, cv;    // element offsets of its first head; ck < 0: nowhere to append
  int used, pad;
};
// Token `at` of the batch and its position.
__device__ __forceinline__ Token rope_token(const RopeParams &p, int64_t at, int64_t &position) {
  const int b = int(uint32_t(at) / uint32_t(p.n)), i = int(at - int64_t(b) * p.n);   // tokens are below 2^31
  const int64_t len = p.lens[b];
  const int count = p.counts ? min(max(p.counts[b], 0), p.n) : p.n;
  Token t;
  t.used = i < count;
  position = len + (p.depth ? p.depth[at] : i);
  const int64_t slot = len + i;
  const int64_t page = t.used && slot >= 0 ? cache_page(p.cache, b, slot) : -1;
  const int64_t off = uint32_t(slot) % uint32_t(p.cache.page_size);
  t.q = b * p.qs[0] + i * p.qs[1];
  t.k = b * p.ks[0] + i * p.ks[1];
  t.v = b * p.vs[0] + i * p.vs[1];
  t.out = at * p.hq * p.d;
  t.ck = page < 0 ? -1 : page * p.cks[0] + off * p.cks[1];
  t.cv = page * p.cvs[0] + off * p.cvs[1];
  return t;
}

template <typename T>
__device__ __forceinline__ void unpack8(float (&f)[8], const uint4 &v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    T lo, hi;
    memcpy(&lo, &w[i], 2);
    const uint32_t h = w[i] >> 16;
    memcpy(&hi, &h, 2);
    f[2 * i] = to_f(lo);
    f[2 * i + 1] = to_f(hi);
  }
}
template <typename T>
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  T t[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) from_f(t[i], f[i]);
  uint4 v;
  memcpy(&v, t, 16);
  return v;
}
__device__ __forceinline__ uint2 pack8_e4m3(const float (&f)[8], float inv) {
  __nv_fp8_e4m3 t[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) from_f(t[i], f[i] * inv);
  uint2 v;
  memcpy(&v, t, 8);
  return v;
}

// Turns 16 elements by the angles `a`.
template <bool kInterleaved>
__device__ __forceinline__ void rotate16(float (&x1)[8], float (&x2)[8], const float2 *a) {
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float2 cs = a[k];
    if (kInterleaved) {
      // pair k of the 16 elements: 2k, 2k + 1
      float &u = k < 4 ? x1[2 * (k & 3)] : x2[2 * (k & 3)];
      float &v = k < 4 ? x1[2 * (k & 3) + 1] : x2[2 * (k & 3) + 1];
      const float y = u * cs.x - v * cs.y;
      v = u * cs.y + v * cs.x;
      u = y;
    } else {
      const float y = x1[k] * cs.x - x2[k] * cs.y;
      x2[k] = x1[k] * cs.y + x2[k] * cs.x;
      x1[k] = y;
    }
  }
}

// Stores elements e1 .. e1 + 7 and e2 .. e2 + 7 of head h of a token: q to q_out, the others to the cache.
template <typename T, typename C>
__device__ __forceinline__ void store16(const RopeParams &p, const Token &t, int h, int e1, int e2, float (&x1)[8],
                                        float (&x2)[8]) {
  const bool is_q = h < p.hq, is_v = h >= p.hq + p.hkv;
  if (is_q) {
    T *dst = static_cast<T *>(p.q_out) + t.out + h * p.d;
    if (!t.used) {
#pragma unroll
      for (int k = 0; k < 8; ++k) x1[k] = x2[k] = 0.f;
    }
    *reinterpret_cast<uint4 *>(dst + e1) = pack8<T>(x1);
    *reinterpret_cast<uint4 *>(dst + e2) = pack8<T>(x2);
  } else {
    C *dst = is_v ? static_cast<C *>(p.cv) + t.cv + (h - p.hq - p.hkv) * p.cvs[2]
                  : static_cast<C *>(p.ck) + t.ck + (h - p.hq) * p.cks[2];
    if constexpr (sizeof(C) == 1) {
      const float inv = is_v ? p.v_inv : p.k_inv;
      *reinterpret_cast<uint2 *>(dst + e1) = pack8_e4m3(x1, inv);
      *reinterpret_cast<uint2 *>(dst + e2) = pack8_e4m3(x2, inv);
    } else {
      *reinterpret_cast<uint4 *>(dst + e1) = pack8<T>(x1);
      *reinterpret_cast<uint4 *>(dst + e2) = pack8<T>(x2);
    }
  }
}

// The checks of a call, its parameters, and whether it can go 16 elements at a time.
inline vg_status rope_params(const vg_rope_desc *d, const vg_kv_cache *cache, RopeParams &p, bool &vector) {
  if (!d) return VG_ERR_INVALID_ARG;
  if (vg_status s = cache_ready(cache)) return s;
  if (!d->q || !d->k || !d->v || !d->q_out || !d->lens || d->n < 1 || d->q_heads < 1 ||
      d->rot < 0 || d->rot % 2 || d->rot > cache->head_dim || (d->rot && !d->inv_freq))
    return VG_ERR_INVALID_ARG;
  if (d->type != VG_TYPE_BF16 && d->type != VG_TYPE_FP16) return VG_ERR_INVALID_ARG;
  if (cache->type != VG_TYPE_E4M3 && cache->type != d->type) return VG_ERR_INVALID_ARG;
  if (d->layout != VG_ROPE_HALF && d->layout != VG_ROPE_INTERLEAVED) return VG_ERR_INVALID_ARG;
  for (const void *at : {d->q, d->k, d->v, static_cast<const void *>(d->q_out)})
    if (reinterpret_cast<uintptr_t>(at) & 1) return VG_ERR_ALIGNMENT;
  const int64_t tokens = int64_t(cache->batch) * d->n;
  if (tokens >= (int64_t(1) << 31) || d->q_heads > 65535) return VG_ERR_UNSUPPORTED;
  p.q = d->q;
  p.k = d->k;
  p.v = d->v;
  p.q_out = d->q_out;
  p.ck = cache->k;
  p.cv = cache->v;
  for (int i = 0; i < 3; ++i) {
    p.qs[i] = d->q_stride[i];
    p.ks[i] = d->k_stride[i];
    p.vs[i] = d->v_stride[i];
    p.cks[i] = cache->k_stride[i];
    p.cvs[i] = cache->v_stride[i];
  }
  p.inv_freq = d->inv_freq;
  p.lens = d->lens;
  p.depth = d->depth;
  p.counts = d->counts;
  p.cache = cache_view(*cache);
  p.tokens = tokens;
  p.n = d->n;
  p.hq = d->q_heads;
  p.hkv = cache->heads;
  p.d = cache->head_dim;
  p.rot = d->rot;
  p.factor = d->factor;
  p.k_inv = 1.f / cache->k_scale;
  p.v_inv = 1.f / cache->v_scale;
  vector = d->rot % 16 == 0 && aligned16(d->q) && aligned16(d->k) && aligned16(d->v) &&
           aligned16(d->q_out);
  for (int i = 0; i < 3; ++i)
    vector = vector && d->q_stride[i] % 8 == 0 && d->k_stride[i] % 8 == 0 && d->v_stride[i] % 8 == 0;
  return VG_OK;
}

// Calls f with a value of q's type and one of the cache's.
template <typename F>
void rope_types(const vg_rope_desc *d, const vg_kv_cache *cache, F &&f) {
  const bool f8 = cache->type == VG_TYPE_E4M3;
  if (d->type == VG_TYPE_BF16) {
    if (f8) f(__nv_bfloat16{}, __nv_fp8_e4m3{});
    else f(__nv_bfloat16{}, __nv_bfloat16{});
  } else {
    if (f8) f(__half{}, __nv_fp8_e4m3{});
    else f(__half{}, __half{});
  }
}

}  // namespace
}  // namespace vg
