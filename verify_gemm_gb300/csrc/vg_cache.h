// vg_cache.h -- the paged key/value cache as the verify-round kernels see it.
#pragma once

#include "vg_internal.h"

namespace vg {

// What vg_kv_cache_init leaves in vg_kv_cache.opaque: the tensor maps of k
// and v (4-D: element, token of a page, head, page) in the first 32 words,
// then a mark over the fields that were checked.
constexpr int kCacheMapWords = 16;            // 128 bytes each
constexpr int kCacheMark = 32;                // opaque[32]
// Slots of a sequence: a length, its tree's nodes and the pages that are fetched
// ahead of them are counted in 32 bits.
constexpr int64_t kCacheMaxSlots = (int64_t(1) << 31) - 8192;
// Boxes of the maps: 128 bytes of a head (64 bytes of E4M3 heads up to 64
// elements) of the largest power of two of tokens, at most 64, that divides
// the page.
inline int cache_box_bytes(const vg_kv_cache &c) {
  return c.type == VG_TYPE_E4M3 && c.head_dim <= 64 ? 64 : 128;
}
inline int cache_box_tokens(int page_size) {
  int t = 16;
  while (t < 64 && page_size % (2 * t) == 0) t *= 2;
  return t;
}

// Fields that the kernels use, checked by vg_kv_cache_init: a cache whose
// fields were changed after it is refused.
inline uint64_t cache_mark(const vg_kv_cache &c) {
  uint64_t h = 0xcbf29ce484222325ull;
  auto add = [&h](uint64_t v) { h = (h ^ v) * 0x100000001b3ull; h ^= h >> 29; };
  add(reinterpret_cast<uintptr_t>(c.k));
  add(reinterpret_cast<uintptr_t>(c.v));
  add(reinterpret_cast<uintptr_t>(c.page_table));
  add(uint64_t(uint32_t(c.type)) | uint64_t(uint32_t(c.heads)) << 32);
  add(uint64_t(uint32_t(c.head_dim)) | uint64_t(uint32_t(c.page_size)) << 32);
  add(uint64_t(c.pages));
  for (int i = 0; i < 3; ++i) {
    add(uint64_t(c.k_stride[i]));
    add(uint64_t(c.v_stride[i]));
  }
  add(uint64_t(c.table_stride));
  add(uint64_t(uint32_t(c.batch)) | uint64_t(uint32_t(c.max_pages)) << 32);
  uint32_t scales[2];
  std::memcpy(&scales[0], &c.k_scale, 4);
  std::memcpy(&scales[1], &c.v_scale, 4);
  add(uint64_t(scales[0]) | uint64_t(scales[1]) << 32);
  return h | 1;
}

inline vg_status cache_ready(const vg_kv_cache *c) {
  if (!c || c->opaque[kCacheMark] != cache_mark(*c)) return VG_ERR_INVALID_ARG;
  return VG_OK;
}

// Addressing of the cache in a kernel.
struct CacheView {
  const int32_t *table;
  int64_t table_stride, pages;
  int32_t page_size, max_pages;
};

inline CacheView cache_view(const vg_kv_cache &c) {
  return {c.page_table, c.table_stride, c.pages, c.page_size, c.max_pages};
}

#ifdef __CUDACC__
// Page of slot `s` (below 2^32) of sequence b, or -1.
__device__ __forceinline__ int64_t cache_page(const CacheView &c, int b, int64_t s) {
  const uint32_t i = uint32_t(s) / uint32_t(c.page_size);
  if (i >= uint32_t(c.max_pages)) return -1;
  const int32_t p = c.table[b * c.table_stride + i];
  return p >= 0 && p < c.pages ? p : -1;
}
#endif

}  // namespace vg
