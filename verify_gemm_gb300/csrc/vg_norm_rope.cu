// vg_norm_rope.cu -- vg_qk_norm_rope_append: RMS norms of the heads of q and k,
// their rotary positions and the append of k and v to the paged cache, in one
// launch.
//
// With r = 1 / sqrt(sum x^2 / d + eps) over a head, the elements x r w turn as
// vg_rope.cu turns x.  A head is read once: its d / 16 threads hold it, their
// sums of squares meet by shuffles, and what is normed goes on to the rotation
// in FP32 (norms by themselves would round to 16 bits between and move q and k
// twice more).  Bytes bound it for prompts and latency for single tokens.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "vg_rope.cuh"

namespace vg {
namespace {

struct NormParams {
  const void *q_weight, *k_weight;   // NULL: ones
  int f32;                           // the weights are FP32, else of q's type
  float eps;
};

constexpr int kNormThreads = 256;
constexpr int kNormBlocks = 4;       // of an SM at once
constexpr int kNormTokens = 16;
// A BF16 head's squares can pass FP32's range: such a head is taken times this,
// which leaves the largest sum of 256 squares below 2^124 (and eps nothing).
constexpr float kNormDown = 0x1p-70f;

template <typename T>
__device__ __forceinline__ float weight_at(const NormParams &n, bool k, int e) {
  const void *w = k ? n.k_weight : n.q_weight;
  return !w ? 1.f : n.f32 ? static_cast<const float *>(w)[e] : to_f(static_cast<const T *>(w)[e]);
}

// A warp a head, one pair of elements a lane at a time: for heads of which a part
// turns that is no multiple of 16 elements and for inputs that are not 16-byte
// aligned.
template <typename T, typename C, bool kInterleaved>
__global__ void __launch_bounds__(kNormThreads) norm_rope_kernel(const RopeParams p, const NormParams n) {
  extern __shared__ float2 angles[];                          // [rot / 2]
  int64_t position;
  const Token t = rope_token(p, blockIdx.x, position);
  const int half = p.rot / 2, lane = threadIdx.x % 32;
  for (int j = threadIdx.x; j < half; j += kNormThreads) angles[j] = turn(p, position, turn_step(p, j));
  __syncthreads();
  const int pairs = half + (p.d - p.rot);                     // turned pairs, then single elements
  for (int h = threadIdx.x / 32; h < p.hq + 2 * p.hkv; h += kNormThreads / 32) {
    const bool is_q = h < p.hq, is_v = h >= p.hq + p.hkv;
    const T *src = is_q ? static_cast<const T *>(p.q) + t.q + h * p.qs[2]
                 : is_v ? static_cast<const T *>(p.v) + t.v + (h - p.hq - p.hkv) * p.vs[2]
                        : static_cast<const T *>(p.k) + t.k + (h - p.hq) * p.ks[2];
    if (!is_q && t.ck < 0) continue;
    float down = 1.f, r = 1.f;
    if (!is_v) {
      auto squares = [&] {
        float s = 0.f;
        for (int e = lane; e < p.d; e += 32) {
          const float x = to_f(src[e]) * down;
          s += x * x;
        }
#pragma unroll
        for (int m = 16; m; m /= 2) s += __shfl_xor_sync(~0u, s, m);
        return s;
      };
      float s = squares();
      if (s == INFINITY) {
        down = kNormDown;
        s = squares();
      }
      r = rsqrtf(s / float(p.d) + n.eps * (down * down));
    }
    for (int w = lane; w < pairs; w += 32) {
      const bool single = w >= half;
      const int e1 = single ? p.rot + w - half : kInterleaved ? 2 * w : w;
      const int e2 = single ? e1 : kInterleaved ? 2 * w + 1 : w + half;
      float x1 = to_f(src[e1]), x2 = to_f(src[e2]);
      if (!is_v) {
        x1 = x1 * down * r * weight_at<T>(n, !is_q, e1);
        x2 = x2 * down * r * weight_at<T>(n, !is_q, e2);
        if (!single) {
          const float2 cs = angles[w];
          const float y1 = x1 * cs.x - x2 * cs.y;
          x2 = x1 * cs.y + x2 * cs.x;
          x1 = y1;
        }
      }
      if (is_q) {
        T *dst = static_cast<T *>(p.q_out) + t.out + h * p.d;
        from_f(dst[e1], t.used ? x1 : 0.f);
        if (!single) from_f(dst[e2], t.used ? x2 : 0.f);
      } else {
        C *dst = is_v ? static_cast<C *>(p.cv) + t.cv + (h - p.hq - p.hkv) * p.cvs[2]
                      : static_cast<C *>(p.ck) + t.ck + (h - p.hq) * p.cks[2];
        if (sizeof(C) == 1) {
          const float inv = is_v ? p.v_inv : p.k_inv;
          x1 *= inv;
          x2 *= inv;
        }
        from_f(dst[e1], x1);
        if (!single) from_f(dst[e2], x2);
      }
    }
  }
}

// 16 elements a thread, 2^kLog threads a head (those past d / 16 idle).
// blockIdx.x: tokens, blockIdx.y: heads.
template <typename T, typename C, bool kInterleaved, int kLog>
__global__ void __launch_bounds__(kNormThreads, kNormBlocks)
    norm_rope_vector_kernel(const RopeParams p, const NormParams n, int tokens_per_block, int heads_per_block) {
  extern __shared__ __align__(16) uint8_t norm_smem[];        // angles [tokens][rot / 2], the steps, the weights
  __shared__ Token tok[kNormTokens];
  __shared__ int64_t position[kNormTokens];
  const int half = p.rot / 2, tid = threadIdx.x;
  float2 *angles = reinterpret_cast<float2 *>(norm_smem);
  uint64_t *steps = reinterpret_cast<uint64_t *>(angles + tokens_per_block * half);
  float *weights = reinterpret_cast<float *>(steps + half);   // [q, k][d]
  const int64_t first = int64_t(blockIdx.x) * tokens_per_block;
  const int tokens = int(min(int64_t(tokens_per_block), p.tokens - first));
  const int h0 = blockIdx.y * heads_per_block;
  const int heads = min(heads_per_block, p.hq + 2 * p.hkv - h0);
  for (int j = tid; j < half; j += kNormThreads) steps[j] = turn_step(p, j);
  for (int j = tid; j < 2 * p.d; j += kNormThreads) weights[j] = weight_at<T>(n, j >= p.d, j >= p.d ? j - p.d : j);
  if (tid < tokens) {
    int64_t at;
    const Token t = rope_token(p, first + tid, at);
    position[tid] = at;
    tok[tid] = t;
  }
  __syncthreads();
  for (int w = tid; w < tokens * half; w += kNormThreads)
    angles[w] = turn(p, position[w / half], steps[w % half]);
  __syncthreads();
  const int c = tid & ((1 << kLog) - 1), items = (tokens * heads) << kLog;
  const bool here = c < p.d / 16, turns = c < p.rot / 16;
  // "half" pairs lie rot / 2 apart; everything else is 16 elements in a row
  const bool apart = turns && !kInterleaved;
  const int e1 = apart ? 8 * c : 16 * c, e2 = apart ? 8 * c + half : 16 * c + 8;
  const float inv_d = 1.f / float(p.d);
#pragma unroll 2
  for (int w0 = tid & ~31; w0 < items; w0 += kNormThreads) {
    const int th = (w0 + (tid & 31)) >> kLog, ti = th / heads, h = h0 + th - ti * heads;
    const bool is_q = h < p.hq, is_v = h >= p.hq + p.hkv;
    const bool any = here && ti < tokens;
    const Token &t = tok[any ? ti : 0];
    const T *src = is_q ? static_cast<const T *>(p.q) + t.q + h * p.qs[2]
                 : is_v ? static_cast<const T *>(p.v) + t.v + (h - p.hq - p.hkv) * p.vs[2]
                        : static_cast<const T *>(p.k) + t.k + (h - p.hq) * p.ks[2];
    uint4 r1 = make_uint4(0, 0, 0, 0), r2 = r1;
    if (any) {
      r1 = *reinterpret_cast<const uint4 *>(src + e1);
      r2 = *reinterpret_cast<const uint4 *>(src + e2);
    }
    float x1[8], x2[8];
    unpack8<T>(x1, r1);
    unpack8<T>(x2, r2);
    auto squares = [&] {
      float s1 = 0.f, s2 = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        s1 = fmaf(x1[k], x1[k], s1);
        s2 = fmaf(x2[k], x2[k], s2);
      }
      float s = s1 + s2;
#pragma unroll
      for (int m = 1; m < 1 << kLog; m *= 2) s += __shfl_xor_sync(~0u, s, m);
      return s;
    };
    float s = squares(), eps = n.eps;
    if constexpr (std::is_same_v<T, __nv_bfloat16>) {
      const bool over = !is_v && s == INFINITY;
      if (__any_sync(~0u, over)) {
        if (over) {
          eps = 0.f;
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            x1[k] *= kNormDown;
            x2[k] *= kNormDown;
          }
        }
        s = squares();
      }
    }
    if (!any || (!is_q && t.ck < 0)) continue;
    if (!is_v) {
      const float r = rsqrtf(s * inv_d + eps);
      const float *wt = weights + (is_q ? 0 : p.d);
#pragma unroll
      for (int k = 0; k < 8; k += 4) {
        const float4 a = *reinterpret_cast<const float4 *>(wt + e1 + k), b = *reinterpret_cast<const float4 *>(wt + e2 + k);
        x1[k] = x1[k] * r * a.x;
        x1[k + 1] = x1[k + 1] * r * a.y;
        x1[k + 2] = x1[k + 2] * r * a.z;
        x1[k + 3] = x1[k + 3] * r * a.w;
        x2[k] = x2[k] * r * b.x;
        x2[k + 1] = x2[k + 1] * r * b.y;
        x2[k + 2] = x2[k + 2] * r * b.z;
        x2[k + 3] = x2[k + 3] * r * b.w;
      }
      if (turns) rotate16<kInterleaved>(x1, x2, angles + ti * half + 8 * c);
    }
    store16<T, C>(p, t, h, e1, e2, x1, x2);
  }
}

template <typename T, typename C, bool kInterleaved>
void launch_norm_rope(const RopeParams &p, const NormParams &n, bool vector, int sms, cudaStream_t st) {
  const int half = p.rot / 2;
  if (!vector) {
    norm_rope_kernel<T, C, kInterleaved><<<unsigned(p.tokens), kNormThreads, size_t(half) * sizeof(float2), st>>>(p, n);
    return;
  }
  // tokens a block and heads a block as rope_append's
  int log = 0;
  while (p.d / 16 > 1 << log) ++log;
  const int heads = p.hq + 2 * p.hkv;
  const int64_t resident = int64_t(kNormBlocks) * sms;
  const int tb = int(std::max<int64_t>(
      1, std::min({int64_t(kNormTokens), int64_t(2048 / (heads << log)), (p.tokens + resident - 1) / resident})));
  const int hb = p.tokens < 2 * sms ? std::max(1, kNormThreads >> log) : heads;
  const dim3 grid(unsigned((p.tokens + tb - 1) / tb), unsigned((heads + hb - 1) / hb));
  const size_t smem = size_t(tb) * half * sizeof(float2) + size_t(half) * sizeof(uint64_t) + size_t(2 * p.d) * sizeof(float);
  auto go = [&](auto kernel) { kernel<<<grid, kNormThreads, smem, st>>>(p, n, tb, hb); };
  switch (log) {
    case 0: go(norm_rope_vector_kernel<T, C, kInterleaved, 0>); break;
    case 1: go(norm_rope_vector_kernel<T, C, kInterleaved, 1>); break;
    case 2: go(norm_rope_vector_kernel<T, C, kInterleaved, 2>); break;
    case 3: go(norm_rope_vector_kernel<T, C, kInterleaved, 3>); break;
    default: go(norm_rope_vector_kernel<T, C, kInterleaved, 4>); break;
  }
}

}  // namespace
}  // namespace vg

using namespace vg;

extern "C" vg_status vg_qk_norm_rope_append(const vg_qk_norm_rope_desc *d, const vg_kv_cache *cache,
                                            vg_stream_t stream) {
  if (!d) return VG_ERR_INVALID_ARG;
  RopeParams p;
  bool vector;
  if (vg_status s = rope_params(&d->rope, cache, p, vector)) return s;
  // (eps may not be so small that a square which FP32 does not hold counts beside it)
  if (!(d->eps >= 0x1p-126f) || !std::isfinite(d->eps)) return VG_ERR_INVALID_ARG;
  if (d->weight_type != VG_TYPE_FP32 && d->weight_type != d->rope.type) return VG_ERR_INVALID_ARG;
  const uintptr_t low = d->weight_type == VG_TYPE_FP32 ? 3 : 1;
  if ((reinterpret_cast<uintptr_t>(d->q_weight) | reinterpret_cast<uintptr_t>(d->k_weight)) & low)
    return VG_ERR_ALIGNMENT;
  int sms = 0;
  if (vg_status s = device_sms(&sms)) return s;
  const NormParams n{d->q_weight, d->k_weight, d->weight_type == VG_TYPE_FP32, d->eps};
  rope_types(&d->rope, cache, [&](auto t, auto c) {
    using T = decltype(t);
    using C = decltype(c);
    if (d->rope.layout == VG_ROPE_INTERLEAVED) launch_norm_rope<T, C, true>(p, n, vector, sms, as_cuda(stream));
    else launch_norm_rope<T, C, false>(p, n, vector, sms, as_cuda(stream));
  });
  VG_LAUNCH_CHECK();
  return VG_OK;
}
