// vg_rope.cu -- vg_kv_cache_init, and vg_rope_append: rotary positions of q
// and k with the append of k and v to the paged cache, in one launch.
//
// The angle of pair j at position s is s * inv_freq[j].  As a fraction of a
// turn it is s * f mod 1 with f = inv_freq[j] / 2 pi, so f is taken as a
// 64-bit integer in units of 2^-64 turns and the product with the integer
// position wraps by itself: no range reduction and no loss at far positions
// (an FP32 product is 0.06 radians off at position 10^6).  What remains, a
// signed fraction of a turn, goes through sincospif in FP32.
//
// Bytes bound it for prompts and latency for single tokens: a block takes
// the heads of up to 16 tokens, so that their angles are worked out once,
// and 16 elements of a head (two 16-byte loads) are a thread's item; with few
// tokens the heads are spread over more blocks instead.  Measured: 16381 tokens
// of 40 + 2 x 8 heads of 128 in FP16 (470 MB) 78 us, 6.0 TB/s, 0.89 of a copy's
// rate; one token of 40 + 2 x 40 heads 3.0 us, a launch.
#include <algorithm>
#include <cmath>

#include "vg_rope.cuh"

namespace vg {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeBlocks = 6;     // of an SM at once: 42 registers a thread (5 blocks: 82 us for 78)

// One pair of elements at a time: for parts of a head that are no multiple of
// 16 elements and for inputs that are not 16-byte aligned.  Its 2-byte loads and
// the divisions of an item set its pace: 16381 tokens of 40 + 2 x 8 heads of 80 with
// 40 elements turned take 186 us, 1.6 TB/s (59 us for all 80 in the kernel below).
template <typename T, typename C, bool kInterleaved>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeParams p) {
  extern __shared__ float2 angles[];                          // [rot / 2]
  const int64_t tok = blockIdx.x;
  const int b = int(tok / p.n), i = int(tok % p.n);
  const int64_t len = p.lens[b];
  const int count = p.counts ? min(max(p.counts[b], 0), p.n) : p.n;
  const bool used = i < count;
  const int half = p.rot / 2;
  const int64_t position = len + (p.depth ? p.depth[tok] : i);
  for (int j = threadIdx.x; j < half; j += kRopeThreads) angles[j] = turn(p, position, turn_step(p, j));
  __syncthreads();
  const int64_t slot = len + i;
  const int64_t page = used && slot >= 0 ? cache_page(p.cache, b, slot) : -1;
  const int64_t off = slot % p.cache.page_size;
  const int pairs = half + (p.d - p.rot);                     // turned pairs, then single elements
  const int heads = p.hq + 2 * p.hkv;
  for (int w = threadIdx.x; w < heads * pairs; w += kRopeThreads) {
    const int h = w / pairs, e = w % pairs;
    const bool single = e >= half;
    const int e1 = single ? p.rot + e - half : kInterleaved ? 2 * e : e;
    const int e2 = single ? e1 : kInterleaved ? 2 * e + 1 : e + half;
    const bool is_q = h < p.hq, is_v = h >= p.hq + p.hkv;
    const T *src = is_q ? static_cast<const T *>(p.q) + b * p.qs[0] + i * p.qs[1] + h * p.qs[2]
                 : is_v ? static_cast<const T *>(p.v) + b * p.vs[0] + i * p.vs[1] +
                              (h - p.hq - p.hkv) * p.vs[2]
                        : static_cast<const T *>(p.k) + b * p.ks[0] + i * p.ks[1] +
                              (h - p.hq) * p.ks[2];
    float x1 = to_f(src[e1]), x2 = to_f(src[e2]);
    if (!single && !is_v) {
      const float2 cs = angles[e];
      const float y1 = x1 * cs.x - x2 * cs.y;
      x2 = x1 * cs.y + x2 * cs.x;
      x1 = y1;
    }
    if (is_q) {
      T *dst = static_cast<T *>(p.q_out) + (tok * p.hq + h) * p.d;
      from_f(dst[e1], used ? x1 : 0.f);
      if (!single) from_f(dst[e2], used ? x2 : 0.f);
    } else if (page >= 0) {
      const int hc = is_v ? h - p.hq - p.hkv : h - p.hq;
      const int64_t *cs = is_v ? p.cvs : p.cks;
      C *dst = static_cast<C *>(is_v ? p.cv : p.ck) + page * cs[0] + off * cs[1] + hc * cs[2];
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

constexpr int kRopeTokens = 16;

// 16 elements at a time.  blockIdx.x: tokens, blockIdx.y: heads.
template <typename T, typename C, bool kInterleaved>
__global__ void __launch_bounds__(kRopeThreads, kRopeBlocks)
    rope_vector_kernel(const RopeParams p, int tokens_per_block, int heads_per_block) {
  extern __shared__ float2 angles[];                          // [tokens][rot / 2], then the steps
  __shared__ Token tok[kRopeTokens];
  const int half = p.rot / 2, tid = threadIdx.x;
  uint64_t *steps = reinterpret_cast<uint64_t *>(angles + tokens_per_block * half);
  const int64_t first = int64_t(blockIdx.x) * tokens_per_block;
  const int tokens = int(min(int64_t(tokens_per_block), p.tokens - first));
  const int h0 = blockIdx.y * heads_per_block;
  const int heads = min(heads_per_block, p.hq + 2 * p.hkv - h0);
  for (int j = tid; j < half; j += kRopeThreads) steps[j] = turn_step(p, j);
  __shared__ int64_t position[kRopeTokens];
  if (tid < tokens) {
    int64_t at;
    const Token t = rope_token(p, first + tid, at);
    position[tid] = at;
    tok[tid] = t;
  }
  __syncthreads();
  for (int w = tid; w < tokens * half; w += kRopeThreads)
    angles[w] = turn(p, position[w / half], steps[w % half]);
  __syncthreads();
  const int chunks = p.d / 16, turned = p.rot / 16;
  const int items = tokens * heads * chunks;
#pragma unroll 2
  for (int w = tid; w < items; w += kRopeThreads) {
    const int c = w % chunks, th = w / chunks, h = h0 + th % heads, ti = th / heads;
    const Token &t = tok[ti];
    const bool is_q = h < p.hq, is_v = h >= p.hq + p.hkv;
    const bool turns = c < turned;
    // "half" pairs lie rot / 2 apart; everything else is 16 elements in a row
    const bool apart = turns && !kInterleaved;
    const int e1 = apart ? 8 * c : 16 * c, e2 = apart ? 8 * c + half : 16 * c + 8;
    const T *src = is_q ? static_cast<const T *>(p.q) + t.q + h * p.qs[2]
                 : is_v ? static_cast<const T *>(p.v) + t.v + (h - p.hq - p.hkv) * p.vs[2]
                        : static_cast<const T *>(p.k) + t.k + (h - p.hq) * p.ks[2];
    const uint4 r1 = *reinterpret_cast<const uint4 *>(src + e1);
    const uint4 r2 = *reinterpret_cast<const uint4 *>(src + e2);
    if (!is_q && t.ck < 0) continue;
    float x1[8], x2[8];
    unpack8<T>(x1, r1);
    unpack8<T>(x2, r2);
    if (turns && !is_v) rotate16<kInterleaved>(x1, x2, angles + ti * half + 8 * c);
    store16<T, C>(p, t, h, e1, e2, x1, x2);
  }
}

template <typename T, typename C, bool kInterleaved>
void launch_rope(const RopeParams &p, bool vector, int sms, cudaStream_t st) {
  const int half = p.rot / 2;
  if (!vector) {
    rope_kernel<T, C, kInterleaved><<<unsigned(p.tokens), kRopeThreads, size_t(half) * sizeof(float2), st>>>(p);
    return;
  }
  // as many tokens a block as fit the device at once, up to 2048 items, eight
  // a thread: what a block waits for before its first item (lengths, pages,
  // angles) is as long for one token as for sixteen.  Under one block an SM,
  // 256 items a block.  19005 tokens of 10 heads of 128 take 32 us with 4 tokens
  // a block and 25 with 16; 1001 tokens of 12 heads of 64 5.3 with 1 and 3.5 with 2.
  const int heads = p.hq + 2 * p.hkv;
  const int64_t resident = int64_t(kRopeBlocks) * sms;
  const int tb = int(std::max<int64_t>(
      1, std::min({int64_t(kRopeTokens), int64_t(2048 / (heads * (p.d / 16))), (p.tokens + resident - 1) / resident})));
  const int hb = p.tokens < 2 * sms ? std::max(1, kRopeThreads / (p.d / 16)) : heads;
  const dim3 grid(unsigned((p.tokens + tb - 1) / tb), unsigned((heads + hb - 1) / hb));
  const size_t smem = size_t(tb) * half * sizeof(float2) + size_t(half) * sizeof(uint64_t);
  rope_vector_kernel<T, C, kInterleaved><<<grid, kRopeThreads, smem, st>>>(p, tb, hb);
}

bool map_cache(CUtensorMap *map, const vg_kv_cache &c, void *base, const int64_t *stride) {
  PFN_cuTensorMapEncodeTiled_v12000 fn = encode_tiled();
  if (!fn) return false;
  const bool f8 = c.type == VG_TYPE_E4M3;
  const cuuint64_t size = f8 ? 1 : 2;
  const cuuint64_t dims[4] = {cuuint64_t(c.head_dim), cuuint64_t(c.page_size), cuuint64_t(c.heads),
                              cuuint64_t(c.pages)};
  const cuuint64_t strides[3] = {cuuint64_t(stride[1]) * size, cuuint64_t(stride[2]) * size,
                                 cuuint64_t(stride[0]) * size};
  const cuuint32_t box[4] = {cuuint32_t(cache_box_bytes(c)) / cuuint32_t(size), cuuint32_t(cache_box_tokens(c.page_size)),
                             1u, 1u};
  const cuuint32_t one[4] = {1u, 1u, 1u, 1u};
  return fn(map, f8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 4, base, dims,
            strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
            cache_box_bytes(c) == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace
}  // namespace vg

using namespace vg;

extern "C" vg_status vg_kv_cache_init(vg_kv_cache *c) {
  if (!c) return VG_ERR_INVALID_ARG;
  c->opaque[kCacheMark] = 0;
  if (!c->k || !c->v || !c->page_table || c->heads < 1 || c->batch < 1 || c->max_pages < 1 ||
      c->pages < 1 || c->head_dim < 16 || c->head_dim % 16 || c->page_size < 16 ||
      c->page_size % 16 || c->table_stride < c->max_pages)
    return VG_ERR_INVALID_ARG;
  if (c->type != VG_TYPE_BF16 && c->type != VG_TYPE_FP16 && c->type != VG_TYPE_E4M3)
    return VG_ERR_INVALID_ARG;
  if (c->head_dim > 256 || c->pages >= (int64_t(1) << 31) || c->heads > 65535 ||
      c->batch > 65535 || int64_t(c->max_pages) * c->page_size > kCacheMaxSlots)
    return VG_ERR_UNSUPPORTED;
  const int64_t size = c->type == VG_TYPE_E4M3 ? 1 : 2;
  if (c->type == VG_TYPE_E4M3) {
    if (!(c->k_scale > 0 && c->v_scale > 0) || !std::isfinite(c->k_scale) ||
        !std::isfinite(c->v_scale))
      return VG_ERR_INVALID_ARG;
  } else if (c->k_scale != 1.f || c->v_scale != 1.f) {
    return VG_ERR_INVALID_ARG;
  }
  for (int i = 0; i < 3; ++i)
    for (const int64_t st : {c->k_stride[i], c->v_stride[i]}) {
      if (st < c->head_dim || st * size % 16) return VG_ERR_INVALID_ARG;
      if (st * size >= (int64_t(1) << 40)) return VG_ERR_UNSUPPORTED;
    }
  if (!aligned16(c->k) || !aligned16(c->v)) return VG_ERR_ALIGNMENT;
  alignas(64) CUtensorMap map;
  if (!map_cache(&map, *c, c->k, c->k_stride)) return VG_ERR_UNSUPPORTED;
  std::memcpy(c->opaque, &map, sizeof map);
  if (!map_cache(&map, *c, c->v, c->v_stride)) return VG_ERR_UNSUPPORTED;
  std::memcpy(c->opaque + kCacheMapWords, &map, sizeof map);
  c->opaque[kCacheMark] = cache_mark(*c);
  return VG_OK;
}

extern "C" vg_status vg_rope_append(const vg_rope_desc *d, const vg_kv_cache *cache,
                                    vg_stream_t stream) {
  RopeParams p;
  bool vector;
  if (vg_status s = rope_params(d, cache, p, vector)) return s;
  int sms = 0;
  if (vg_status s = device_sms(&sms)) return s;
  rope_types(d, cache, [&](auto t, auto c) {
    using T = decltype(t);
    using C = decltype(c);
    if (d->layout == VG_ROPE_INTERLEAVED) launch_rope<T, C, true>(p, vector, sms, as_cuda(stream));
    else launch_rope<T, C, false>(p, vector, sms, as_cuda(stream));
  });
  VG_LAUNCH_CHECK();
  return VG_OK;
}
