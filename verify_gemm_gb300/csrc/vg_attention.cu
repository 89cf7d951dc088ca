// vg_attention.cu -- vg_tree_attention: the nodes of each sequence's tree
// over its paged cache.
//
// A block computes one row (a node's head): its warps share out the keys,
// each with a running maximum m, sum l and output o of its own
//     m' = max(m, s),  l' = l e^(m - m') + e^(s - m'),  o' = o e^(m - m') + v e^(s - m'),
// and the warps' results are joined at the end in warp order.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cmath>

#include "vg_cache.h"

namespace vg {
namespace {

constexpr int kHead = 256;                    // workspace header bytes
constexpr int kWarps = 8;
constexpr int kMaxD = 256;

struct AttnParams {
  const void *q, *k, *v;
  void *out;
  float *lse;
  const int32_t *lens, *counts;
  const uint64_t *tree;
  int64_t qs[3], ks[3], vs[3];
  CacheView cache;
  int n, hq, hkv, d;
  float scale, v_scale;             // scale includes k_scale
};

__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f(__nv_fp8_e4m3 x) { return float(x); }

template <typename T, typename C>
__global__ void __launch_bounds__(kWarps * 32) attention_kernel(const AttnParams p) {
  __shared__ float sm[kWarps], sl[kWarps], so[kWarps][kMaxD];
  const int h = blockIdx.x % p.hq, i = blockIdx.x / p.hq, b = blockIdx.y;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int64_t len = max(p.lens[b], 0);
  const int count = p.counts ? min(max(p.counts[b], 0), p.n) : p.n;
  const int64_t total = i < count ? len + count : 0;
  const uint64_t word = p.tree ? p.tree[int64_t(b) * p.n + i] : (~0ull >> (63 - i));
  const int hk = h / (p.hq / p.hkv);
  const T *q = static_cast<const T *>(p.q) + b * p.qs[0] + i * p.qs[1] + h * p.qs[2];
  float qr[kMaxD / 32], o[kMaxD / 32];
#pragma unroll
  for (int k = 0; k < kMaxD / 32; ++k) {
    qr[k] = lane + 32 * k < p.d ? to_f(q[lane + 32 * k]) * p.scale : 0.f;
    o[k] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int64_t s = warp; s < total; s += kWarps) {
    if (s >= len && !((word >> (s - len)) & 1)) continue;
    const int64_t page = cache_page(p.cache, b, s), off = s % p.cache.page_size;
    if (page < 0) continue;
    const C *k = static_cast<const C *>(p.k) + page * p.ks[0] + off * p.ks[1] + hk * p.ks[2];
    const C *v = static_cast<const C *>(p.v) + page * p.vs[0] + off * p.vs[1] + hk * p.vs[2];
    float x = 0.f;
#pragma unroll
    for (int c = 0; c < kMaxD / 32; ++c)
      if (lane + 32 * c < p.d) x += qr[c] * to_f(k[lane + 32 * c]);
#pragma unroll
    for (int w = 16; w; w /= 2) x += __shfl_xor_sync(~0u, x, w);
    const float m2 = fmaxf(m, x), keep = m == -INFINITY ? 0.f : expf(m - m2);
    const float e = x == -INFINITY ? 0.f : expf(x - m2);
    l = l * keep + e;
    m = m2;
#pragma unroll
    for (int c = 0; c < kMaxD / 32; ++c)
      if (lane + 32 * c < p.d) o[c] = o[c] * keep + e * to_f(v[lane + 32 * c]);
  }
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
#pragma unroll
  for (int c = 0; c < kMaxD / 32; ++c)
    if (lane + 32 * c < p.d) so[warp][lane + 32 * c] = o[c];
  __syncthreads();
  float top = -INFINITY, sum = 0.f;
  for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sm[w]);
  for (int w = 0; w < kWarps; ++w) sum += sm[w] == -INFINITY ? 0.f : sl[w] * expf(sm[w] - top);
  const int64_t row = (int64_t(b) * p.n + i) * p.hq + h;
  T *out = static_cast<T *>(p.out) + row * p.d;
  for (int e = threadIdx.x; e < p.d; e += kWarps * 32) {
    float y = 0.f;
    for (int w = 0; w < kWarps; ++w) y += sm[w] == -INFINITY ? 0.f : so[w][e] * expf(sm[w] - top);
    out[e] = T(sum == 0.f ? 0.f : y / sum * p.v_scale);
  }
  if (p.lse && threadIdx.x == 0) p.lse[row] = sum == 0.f ? -INFINITY : top + logf(sum);
}

}  // namespace
}  // namespace vg

using namespace vg;

extern "C" vg_status vg_tree_attention_workspace_size(int n, int q_heads, const vg_kv_cache *cache,
                                                      size_t *bytes) {
  if (!bytes || n < 1 || n > 64 || q_heads < 1) return VG_ERR_INVALID_ARG;
  if (vg_status s = cache_ready(cache)) return s;
  if (q_heads % cache->heads) return VG_ERR_INVALID_ARG;
  *bytes = kHead;
  return VG_OK;
}

extern "C" vg_status vg_tree_attention(const vg_attention_desc *d, const vg_kv_cache *cache,
                                       void *workspace, size_t workspace_bytes,
                                       vg_stream_t stream) {
  if (!d) return VG_ERR_INVALID_ARG;
  size_t need = 0;
  if (vg_status s = vg_tree_attention_workspace_size(d->n, d->q_heads, cache, &need)) return s;
  if (!d->q || !d->out || !d->lens || !std::isfinite(d->scale)) return VG_ERR_INVALID_ARG;
  if (d->type != VG_TYPE_BF16 && d->type != VG_TYPE_FP16) return VG_ERR_INVALID_ARG;
  if (cache->type != VG_TYPE_E4M3 && cache->type != d->type) return VG_ERR_INVALID_ARG;
  for (int i = 0; i < 3; ++i)
    if (d->q_stride[i] % 8) return VG_ERR_ALIGNMENT;
  if (!aligned16(d->q) || !aligned16(d->out)) return VG_ERR_ALIGNMENT;
  if (!workspace || workspace_bytes < need) return VG_ERR_WORKSPACE;
  if (!aligned16(workspace)) return VG_ERR_ALIGNMENT;
  int sms = 0;
  if (vg_status s = device_sms(&sms)) return s;
  AttnParams p;
  p.q = d->q;
  p.k = cache->k;
  p.v = cache->v;
  p.out = d->out;
  p.lse = d->lse;
  p.lens = d->lens;
  p.counts = d->counts;
  p.tree = d->tree;
  for (int i = 0; i < 3; ++i) {
    p.qs[i] = d->q_stride[i];
    p.ks[i] = cache->k_stride[i];
    p.vs[i] = cache->v_stride[i];
  }
  p.cache = cache_view(*cache);
  p.n = d->n;
  p.hq = d->q_heads;
  p.hkv = cache->heads;
  p.d = cache->head_dim;
  p.scale = d->scale * cache->k_scale;
  p.v_scale = cache->v_scale;
  const dim3 grid(unsigned(d->n) * unsigned(d->q_heads), unsigned(cache->batch));
  cudaStream_t st = as_cuda(stream);
  const bool f8 = cache->type == VG_TYPE_E4M3;
  if (d->type == VG_TYPE_BF16) {
    if (f8) attention_kernel<__nv_bfloat16, __nv_fp8_e4m3><<<grid, kWarps * 32, 0, st>>>(p);
    else attention_kernel<__nv_bfloat16, __nv_bfloat16><<<grid, kWarps * 32, 0, st>>>(p);
  } else {
    if (f8) attention_kernel<__half, __nv_fp8_e4m3><<<grid, kWarps * 32, 0, st>>>(p);
    else attention_kernel<__half, __half><<<grid, kWarps * 32, 0, st>>>(p);
  }
  VG_LAUNCH_CHECK();
  return VG_OK;
}
