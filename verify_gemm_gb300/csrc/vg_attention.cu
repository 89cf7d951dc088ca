// vg_attention.cu -- vg_tree_attention's entry points: argument checks, the
// choice of a kernel variant and its launch.
#include <algorithm>
#include <cmath>

#include "vg_attention.cuh"

namespace vg {
namespace {

using namespace attn;

// tcgen05 where mma.sync would set the pace.
bool is_wide(int d, int rows) { return d <= 128 && rows > 32; }

// Row groups: the fewest that hold the rows of a head, so that as many warps
// as can share out the keys; above 128 rows, blocks of 128.
int row_index(int rows) { return rows <= 16 ? 0 : rows <= 32 ? 1 : rows <= 64 ? 2 : 3; }

const Variant &pick(int type, int d, int rows) {
  if (is_wide(d, rows)) return kWide[type][d <= 64 ? 0 : 1][rows <= 128 ? 0 : 1];
  const Variants &of = type == kBf16 ? kVariantsBf16 : type == kF16 ? kVariantsF16 : kVariantsE4M3;
  const int r = row_index(rows);
  return of[d <= 64 ? 0 : d <= 128 ? 1 : d <= 192 && r >= 2 ? 2 : 3][r];
}

int cache_type(const vg_kv_cache &c) {
  return c.type == VG_TYPE_E4M3 ? kE4M3 : c.type == VG_TYPE_FP16 ? kF16 : kBf16;
}

// Lets the kernel have its shared memory, once for each device.
vg_status allow_smem(const Variant &v) {
  int dev = 0;
  VG_CUDA(cudaGetDevice(&dev));
  const uint64_t bit = uint64_t(1) << (dev & 63);       // device_sms refuses higher numbers
  if (v.allowed->load(std::memory_order_relaxed) & bit) return VG_OK;
  VG_CUDA(cudaFuncSetAttribute(reinterpret_cast<const void *>(v.fn),
                               cudaFuncAttributeMaxDynamicSharedMemorySize, v.smem));
  v.allowed->fetch_or(bit, std::memory_order_relaxed);
  return VG_OK;
}

size_t workspace_bytes_of(const Variant &v, int sms) {
  return kHeader + 3 * kMaxGrid * sizeof(uint32_t) + size_t(sms) * 2 * size_t(v.partial) * sizeof(float);
}

}  // namespace
}  // namespace vg

using namespace vg;

extern "C" vg_status vg_tree_attention_workspace_size(int n, int q_heads, const vg_kv_cache *cache,
                                                      size_t *bytes) {
  if (!bytes || n < 1 || n > 64 || q_heads < 1) return VG_ERR_INVALID_ARG;
  if (vg_status s = cache_ready(cache)) return s;
  if (q_heads % cache->heads) return VG_ERR_INVALID_ARG;
  if (q_heads / cache->heads > 4096) return VG_ERR_UNSUPPORTED;
  int sms = 0;
  if (vg_status s = device_sms(&sms)) return s;
  *bytes = workspace_bytes_of(pick(cache_type(*cache), cache->head_dim, n * (q_heads / cache->heads)), sms);
  return VG_OK;
}

extern "C" vg_status vg_tree_attention(const vg_attention_desc *d, const vg_kv_cache *cache,
                                       void *workspace, size_t workspace_bytes,
                                       vg_stream_t stream) {
  if (!d || d->n < 1 || d->n > 64 || d->q_heads < 1) return VG_ERR_INVALID_ARG;
  if (vg_status s = cache_ready(cache)) return s;
  if (d->q_heads % cache->heads) return VG_ERR_INVALID_ARG;
  if (!d->q || !d->out || !d->lens || !std::isfinite(d->scale)) return VG_ERR_INVALID_ARG;
  if (d->type != VG_TYPE_BF16 && d->type != VG_TYPE_FP16) return VG_ERR_INVALID_ARG;
  if (cache->type != VG_TYPE_E4M3 && cache->type != d->type) return VG_ERR_INVALID_ARG;
  for (int i = 0; i < 3; ++i)
    if (d->q_stride[i] % 8) return VG_ERR_ALIGNMENT;
  if (!aligned16(d->q) || !aligned16(d->out)) return VG_ERR_ALIGNMENT;
  if (d->q_heads / cache->heads > 4096) return VG_ERR_UNSUPPORTED;
  int sms = 0;
  if (vg_status s = device_sms(&sms)) return s;
  if (sms > kMaxGrid) return VG_ERR_UNSUPPORTED;
  const int rows = d->n * (d->q_heads / cache->heads);
  const int type = cache_type(*cache);
  const Variant &v = pick(type, cache->head_dim, rows);
  if (!workspace || workspace_bytes < workspace_bytes_of(v, sms)) return VG_ERR_WORKSPACE;
  if (!aligned16(workspace)) return VG_ERR_ALIGNMENT;
  AttnParams p;
  p.q = d->q;
  p.out = d->out;
  p.lse = d->lse;
  p.lens = d->lens;
  p.counts = d->counts;
  p.tree = d->tree;
  for (int i = 0; i < 3; ++i) p.qs[i] = d->q_stride[i];
  p.cache = cache_view(*cache);
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  p.error = reinterpret_cast<int *>(ws);
  p.arrived = reinterpret_cast<uint32_t *>(ws + kHeader);
  p.partial = reinterpret_cast<float *>(ws + kHeader + 3 * kMaxGrid * sizeof(uint32_t));
  p.batch = cache->batch;
  p.n = d->n;
  p.hq = d->q_heads;
  p.hkv = cache->heads;
  p.d = cache->head_dim;
  p.q_f16 = d->type == VG_TYPE_FP16;
  p.rows = rows;
  p.group = d->q_heads / cache->heads;
  p.group_magic = p.group == 1 ? 0 : uint32_t((uint64_t(1) << 32) / uint64_t(p.group)) + 1;
  p.blocks = (rows + v.rows - 1) / v.rows;
  p.box = cache_box_tokens(cache->page_size);
  // What a unit costs beside its tiles, in tiles, and half of it as the cut that
  // moves: less saves more than it unbalances.  Beginning and joining a unit
  // takes some 4 us.  The tcgen05 kernel's tiles take what a stream's chain of
  // scores, maxima and weights takes, whatever their bytes; the other's by their bytes (45 GB/s a block) but for
  // the smallest ones, and by the products from 64 rows on.  Measured over 1 to
  // 16 tiles of ragged batches: 18 sequences of 304 rows of 128, 6 tiles 100 us,
  // 8 106, 16 114; 30 units of 55 rows of 64 in E4M3, 26 us, 27, 32 and 40 with
  // 32; 50 units of 128 rows of 256, 2 tiles 36 us, 4 41.
  const bool wide = is_wide(p.d, rows);
  p.tile_log2 = wide ? 7 : 6;
  const int tile_bytes = (2 * p.d * (type == kE4M3 ? 1 : 2)) << p.tile_log2;
  p.least = std::max(1, 131072 / tile_bytes);
  p.extra = wide ? 6 : std::max(1, std::min({8, 16 * 16 / v.rows, 262144 / tile_bytes}));
  p.snap = p.extra / 2;
  p.c = d->scale * cache->k_scale * kLog2e;
  p.v_scale = cache->v_scale;
  // no more blocks than there can be tiles
  const int64_t most = int64_t(cache->batch) * cache->heads * p.blocks *
                       ((int64_t(cache->max_pages) * cache->page_size + d->n + kTile - 1) / kTile);
  const unsigned grid = unsigned(std::min<int64_t>(sms, most));
  alignas(64) CUtensorMap kmap, vmap;
  std::memcpy(&kmap, cache->opaque, sizeof kmap);
  std::memcpy(&vmap, cache->opaque + kCacheMapWords, sizeof vmap);
  if (vg_status s = allow_smem(v)) return s;
  v.fn<<<grid, v.threads, size_t(v.smem), as_cuda(stream)>>>(p, kmap, vmap);
  VG_LAUNCH_CHECK();
  return VG_OK;
}
