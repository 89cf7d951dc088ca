// vg_norm_rope.cu -- vg_qk_norm_rope_append: RMS norms of the heads of q and k,
// their rotary positions and the append of k and v to the paged cache, in one
// launch.
//
// With r = 1 / sqrt(sum x^2 / d + eps) over a head, the elements x r w turn as
// vg_rope.cu turns x.  A head is read once: its d / 16 threads hold it, their
// sums of squares meet by shuffles, and what is normed goes on to the rotation
// in FP32 (norms by themselves would round to 16 bits between and move q and k
// twice more).
//
// Bytes bound it for prompts and latency for single tokens.  The shuffles and the shared memory
// of weights and angles make an item's chain long, so the loads of two items
// go ahead of it, and a block takes as many tokens (up to 32) as let all
// blocks run at once.  16381 tokens of 40 + 2 x 8 heads of 128 in FP16 (470 MB) 88 us, 5.3
// TB/s, 0.78 of a copy's rate (rows of weights and angles in the elements' order met in four
// banks each: 107 us; loads one item ahead 92; three ahead do not fit the
// registers: 130); one token of 40 + 2 x 8 heads 5.4 us a call, the host's time.  A head has a power of two of
// threads, so that heads of 80, 96 and 112 leave 3/8 to 1/8 of them idle: 16381 tokens take 86 to 88 us whichever it is
// (floors 43 to 61).
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "vg_pairs.cuh"
#include "vg_rope.cuh"

namespace vg {
namespace {

struct NormParams {
  const void *q_weight, *k_weight;   // NULL: ones
  int f32;                           // the weights are FP32, else of q's type
  float eps;
};

constexpr int kNormThreads = 256;
constexpr int kNormBlocks = 4;       // of an SM at once: 64 registers a thread (5 blocks spill: 139 us for 88)
constexpr int kNormTokens = 32;
// A BF16 head's squares, or their mean and eps, can pass FP32's range: such a head is taken times this (and eps
// times its square), which leaves the largest sum of 256 squares below 2^124.
constexpr float kNormDown = 0x1p-70f;

template <typename T>
__device__ __forceinline__ float weight_at(const NormParams &n, bool k, int e) {
  const void *w = k ? n.k_weight : n.q_weight;
  return !w ? 1.f : n.f32 ? static_cast<const float *>(w)[e] : to_f(static_cast<const T *>(w)[e]);
}

// A warp a head, one pair of elements a lane at a time: for heads of which a part
// turns that is no multiple of 16 elements and for inputs that are not 16-byte
// aligned.  Loads of 2 bytes, and each head read twice, set its pace: 16381 tokens of 40 + 2 x 8 heads of
// 80 of which 40 elements turn 345 us (floor 43), of 128 that are not aligned 292 (69).
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
      float mean = squares() / float(p.d) + n.eps;
      if (mean == INFINITY) {
        down = kNormDown;
        mean = squares() / float(p.d) + n.eps * down * down;
      }
      r = rsqrtf(mean);
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

template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if constexpr (std::is_same_v<T, __half>) {
    __half2 h;
    memcpy(&h, &w, 4);
    return __half22float2(h);
  } else {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  }
}
template <typename T>
__device__ __forceinline__ uint32_t round2(float a, float b) {
  uint32_t w;
  if constexpr (std::is_same_v<T, __half>) {
    const __half2 h = __floats2half2_rn(a, b);
    memcpy(&w, &h, 4);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    memcpy(&w, &h, 4);
  }
  return w;
}

// 16 elements a thread, 2^kLog threads a head (those past d / 16 idle), as two rows of 8: the first and
// the second of the pairs that turn.  blockIdx.x: tokens, blockIdx.y: heads.
template <typename T, typename C, bool kInterleaved, int kLog>
__global__ void __launch_bounds__(kNormThreads, kNormBlocks)
    norm_rope_vector_kernel(const RopeParams p, const NormParams n, int tokens_per_block, int heads_per_block) {
  extern __shared__ __align__(16) uint8_t norm_smem[];        // cosines, sines [tokens][rot / 2], the steps, the weights
  __shared__ Token tok[kNormTokens];
  __shared__ int64_t position[kNormTokens];
  const int half = p.rot / 2, tid = threadIdx.x;
  float *cosines = reinterpret_cast<float *>(norm_smem), *sines = cosines + tokens_per_block * half;
  uint64_t *steps = reinterpret_cast<uint64_t *>(sines + tokens_per_block * half);
  float *weights = reinterpret_cast<float *>(steps + half);   // [q, k][4][thread of the head][4]
  const int64_t first = int64_t(blockIdx.x) * tokens_per_block;
  const int tokens = int(min(int64_t(tokens_per_block), p.tokens - first));
  const int h0 = blockIdx.y * heads_per_block;
  const int heads = min(heads_per_block, p.hq + 2 * p.hkv - h0);
  const int c = tid & ((1 << kLog) - 1), items = (tokens * heads) << kLog;
  const int turned = p.rot / 16;
  const bool here = c < p.d / 16, turns = c < turned;
  // "half" pairs lie rot / 2 apart; everything else is 16 elements in a row
  const bool apart = turns && !kInterleaved;
  const int e1 = apart ? 8 * c : 16 * c, e2 = apart ? 8 * c + half : 16 * c + 8;
  const float inv_d = 1.f / float(p.d);
  // An item's loads go ahead of the item before, and the first one's of the angles.
  struct Item {
    int ti, h;
    uint4 r1, r2;
  };
  auto fetch = [&](Item &x, int w, auto &&begins) {
    const int th = w >> kLog;
    x.ti = th / heads;
    x.h = h0 + th - x.ti * heads;
    if (!here || x.ti >= tokens) return;
    int64_t q, k, v;
    begins(x.ti, q, k, v);
    const T *src = x.h < p.hq           ? static_cast<const T *>(p.q) + q + x.h * p.qs[2]
                   : x.h < p.hq + p.hkv ? static_cast<const T *>(p.k) + k + (x.h - p.hq) * p.ks[2]
                                        : static_cast<const T *>(p.v) + v + (x.h - p.hq - p.hkv) * p.vs[2];
    x.r1 = *reinterpret_cast<const uint4 *>(src + e1);
    x.r2 = *reinterpret_cast<const uint4 *>(src + e2);
  };
  constexpr int kAhead = 2;
  Item next[kAhead];
  auto first_at = [&](int ti, int64_t &q, int64_t &k, int64_t &v) {
    const int64_t at = first + ti;
    const int b = int(uint32_t(at) / uint32_t(p.n)), i = int(at - int64_t(b) * p.n);
    q = b * p.qs[0] + i * p.qs[1];
    k = b * p.ks[0] + i * p.ks[1];
    v = b * p.vs[0] + i * p.vs[1];
  };
#pragma unroll
  for (int k = 0; k < kAhead; ++k)
    if ((tid & ~31) + k * kNormThreads < items) fetch(next[k], tid + k * kNormThreads, first_at);
  for (int j = tid; j < half; j += kNormThreads) steps[j] = turn_step(p, j);
  for (int j = tid; j < 2 * p.d; j += kNormThreads) {
    const int at = j >= p.d ? j - p.d : j, chunk = at / 16, k = at % 16;
    const int e = kInterleaved     ? 16 * chunk + 2 * (k % 8) + k / 8
                  : chunk < turned ? 8 * chunk + k % 8 + k / 8 * half
                                   : at;
    // fours of a head's threads lie side by side: a quarter of a warp reads 128 bytes in a row
    weights[(((j >= p.d) * 4 + k / 4 << kLog) + chunk) * 4 + k % 4] = weight_at<T>(n, j >= p.d, e);
  }
  if (tid < tokens) {
    int64_t at;
    const Token t = rope_token(p, first + tid, at);
    position[tid] = at;
    tok[tid] = t;
  }
  __syncthreads();
  for (int w = tid; w < tokens * half; w += kNormThreads) {
    const int ti = w / half, j = w - ti * half, to = ti * half + (j / 4 % 2 * turned + j / 8) * 4 + j % 4;
    const float2 a = turn(p, position[ti], steps[j]);
    cosines[to] = a.x;
    sines[to] = a.y;
  }
  __syncthreads();
  for (int w0 = tid & ~31; w0 < items; w0 += kNormThreads) {
    const Item now = next[0];
#pragma unroll
    for (int k = 1; k < kAhead; ++k) next[k - 1] = next[k];
    if (w0 + kAhead * kNormThreads < items)
      fetch(next[kAhead - 1], w0 + kAhead * kNormThreads + (tid & 31), [&](int ti, int64_t &q, int64_t &k, int64_t &v) {
        q = tok[ti].q;
        k = tok[ti].k;
        v = tok[ti].v;
      });
    const int ti = now.ti, h = now.h;
    const bool is_q = h < p.hq, is_v = h >= p.hq + p.hkv;
    const bool any = here && ti < tokens;
    const Token &t = tok[any ? ti : 0];
    const uint32_t r[8] = {now.r1.x, now.r1.y, now.r1.z, now.r1.w, now.r2.x, now.r2.y, now.r2.z, now.r2.w};
    float2 x1[4], x2[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (kInterleaved) {
        const float2 a = unpack2<T>(r[2 * j]), b = unpack2<T>(r[2 * j + 1]);
        x1[j] = make_float2(a.x, b.x);
        x2[j] = make_float2(a.y, b.y);
      } else {
        x1[j] = unpack2<T>(r[j]);
        x2[j] = unpack2<T>(r[4 + j]);
      }
    }
    auto squares = [&] {
      float2 a = mul2(x1[0], x1[0]), b = mul2(x2[0], x2[0]);
#pragma unroll
      for (int j = 1; j < 4; ++j) {
        a = fma2(x1[j], x1[j], a);
        b = fma2(x2[j], x2[j], b);
      }
      float s = any ? (a.x + a.y) + (b.x + b.y) : 0.f;
#pragma unroll
      for (int m = 1; m < 1 << kLog; m *= 2) s += __shfl_xor_sync(~0u, s, m);
      return s;
    };
    float mean = fmaf(squares(), inv_d, n.eps);
    if constexpr (std::is_same_v<T, __nv_bfloat16>) {
      const bool over = !is_v && mean == INFINITY;
      if (__any_sync(~0u, over)) {
        if (over) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            x1[j] = mul2(x1[j], both(kNormDown));
            x2[j] = mul2(x2[j], both(kNormDown));
          }
        }
        const float s = squares();
        if (over) mean = fmaf(s, inv_d, n.eps * kNormDown * kNormDown);
      }
    }
    if (!any || (!is_q && t.ck < 0)) continue;
    if (!is_v) {
      const float inv = rsqrtf(mean);
      const float4 *wt = reinterpret_cast<const float4 *>(weights) + (is_q ? 0 : 4 << kLog) + c;
#pragma unroll
      for (int j = 0; j < 4; j += 2) {
        const float4 a = wt[j / 2 << kLog], b = wt[2 + j / 2 << kLog];
        x1[j] = mul2(mul2(x1[j], both(inv)), make_float2(a.x, a.y));
        x1[j + 1] = mul2(mul2(x1[j + 1], both(inv)), make_float2(a.z, a.w));
        x2[j] = mul2(mul2(x2[j], both(inv)), make_float2(b.x, b.y));
        x2[j + 1] = mul2(mul2(x2[j + 1], both(inv)), make_float2(b.z, b.w));
      }
      if (turns) {
        const float4 *cs = reinterpret_cast<const float4 *>(cosines + ti * half) + c;
        const float4 *sn = reinterpret_cast<const float4 *>(sines + ti * half) + c;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float4 c4 = cs[j / 2 * turned], s4 = sn[j / 2 * turned];
          const float2 co = j % 2 ? make_float2(c4.z, c4.w) : make_float2(c4.x, c4.y);
          const float2 si = j % 2 ? make_float2(s4.z, s4.w) : make_float2(s4.x, s4.y);
          const float2 u = x1[j], v = x2[j], y = mul2(v, si);
          x1[j] = fma2(u, co, make_float2(-y.x, -y.y));
          x2[j] = fma2(u, si, mul2(v, co));
        }
      }
    }
    // the 8 words of e1 .. e1 + 7 and e2 .. e2 + 7
    float2 y[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      y[kInterleaved ? 2 * j : j] = kInterleaved ? make_float2(x1[j].x, x2[j].x) : x1[j];
      y[kInterleaved ? 2 * j + 1 : 4 + j] = kInterleaved ? make_float2(x1[j].y, x2[j].y) : x2[j];
    }
    if (is_q || sizeof(C) == 2) {
      uint32_t w[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = is_q && !t.used ? 0 : round2<T>(y[j].x, y[j].y);
      T *dst = is_q   ? static_cast<T *>(p.q_out) + t.out + h * p.d
               : is_v ? static_cast<T *>(p.cv) + t.cv + (h - p.hq - p.hkv) * p.cvs[2]
                      : static_cast<T *>(p.ck) + t.ck + (h - p.hq) * p.cks[2];
      *reinterpret_cast<uint4 *>(dst + e1) = make_uint4(w[0], w[1], w[2], w[3]);
      *reinterpret_cast<uint4 *>(dst + e2) = make_uint4(w[4], w[5], w[6], w[7]);
    } else {
      const float2 inv = both(is_v ? p.v_inv : p.k_inv);
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 a = mul2(y[2 * j], inv), b = mul2(y[2 * j + 1], inv);
        w[j] = uint32_t(__nv_cvt_float2_to_fp8x2(a, __NV_SATFINITE, __NV_E4M3)) |
               uint32_t(__nv_cvt_float2_to_fp8x2(b, __NV_SATFINITE, __NV_E4M3)) << 16;
      }
      uint8_t *dst = is_v ? static_cast<uint8_t *>(p.cv) + t.cv + (h - p.hq - p.hkv) * p.cvs[2]
                          : static_cast<uint8_t *>(p.ck) + t.ck + (h - p.hq) * p.cks[2];
      *reinterpret_cast<uint2 *>(dst + e1) = make_uint2(w[0], w[1]);
      *reinterpret_cast<uint2 *>(dst + e2) = make_uint2(w[2], w[3]);
    }
  }
}

template <typename T, typename C, bool kInterleaved>
void launch_norm_rope(const RopeParams &p, const NormParams &n, bool vector, int sms, cudaStream_t st) {
  const int half = p.rot / 2;
  if (!vector) {
    norm_rope_kernel<T, C, kInterleaved><<<unsigned(p.tokens), kNormThreads, size_t(half) * sizeof(float2), st>>>(p, n);
    return;
  }
  // all blocks at once, up to 32 tokens each (16381 tokens, 27 a block: 88 us; 8 a block 90, 4 93); with
  // fewer than two an SM the heads are spread over blocks, 256 items each
  int log = 0;
  while (p.d / 16 > 1 << log) ++log;
  const int heads = p.hq + 2 * p.hkv;
  const int64_t resident = int64_t(kNormBlocks) * sms;
  const int tb = int(std::min(int64_t(kNormTokens), (p.tokens + resident - 1) / resident));
  const int hb = p.tokens < 2 * sms ? std::max(1, kNormThreads >> log) : heads;
  const dim3 grid(unsigned((p.tokens + tb - 1) / tb), unsigned((heads + hb - 1) / hb));
  const size_t smem = size_t(tb) * half * 2 * sizeof(float) + size_t(half) * sizeof(uint64_t) + (size_t(32) << log) * sizeof(float);
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
