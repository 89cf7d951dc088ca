// vg_attention.cu -- vg_tree_attention's entry points: argument checks, the
// choice of a kernel variant and its launch.
#include <algorithm>
#include <cmath>

#include "vg_attention.cuh"
#include "vg_prefix.h"

namespace vg {
namespace {

using namespace attn;

// tcgen05 where mma.sync would set the pace.
bool is_wide(int d, int rows) { return d <= 128 && rows > 32; }

// Row groups: the fewest that hold the rows of a head, so that as many warps
// as can share out the keys; above 128 rows, blocks of 128.
int row_index(int rows) { return rows <= 16 ? 0 : rows <= 32 ? 1 : rows <= 64 ? 2 : 3; }

const Variant &pick(int type, int d, int rows, bool parts = false) {
  if (is_wide(d, rows)) return (parts ? kWideParts : kWide)[type][d <= 64 ? 0 : 1][rows <= 128 ? 0 : 1];
  const Variants &of = parts ? (type == kBf16 ? kPartsBf16 : type == kF16 ? kPartsF16 : kPartsE4M3)
                             : (type == kBf16 ? kVariantsBf16 : type == kF16 ? kVariantsF16 : kVariantsE4M3);
  const int r = row_index(rows);
  return of[d <= 64 ? 0 : d <= 128 ? 1 : d <= 192 && r >= 2 ? 2 : 3][r];
}

// The same for the rows of a whole batch over a prefix.  Under 1024 of them the tcgen05 kernel takes
// blocks of 128: 320 rows are 3 tiles of 128 and not 4 (65500 keys in E4M3: 156 us against 176), and
// 240 rows leave half the partial results (8003 keys of 8 heads, a decode of 48: 74 us against 76).  From
// there on blocks of 256, for which K and V are read half as often (4096 rows, 16384 keys: 290 us
// against 293).
const Variant &pick_prefix(int type, int d, int64_t rows) {
  return pick(type, d, is_wide(d, int(rows)) && rows < 1024 ? 128 : int(rows), true);
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

size_t workspace_bytes_of(int partial, int sms) {
  return kHeader + 3 * kMaxGrid * sizeof(uint32_t) + size_t(sms) * 2 * size_t(partial) * sizeof(float);
}

vg_status check_heads(int n, int q_heads, const vg_kv_cache *cache) {
  if (n < 1 || n > 64 || q_heads < 1) return VG_ERR_INVALID_ARG;
  if (vg_status s = cache_ready(cache)) return s;
  if (q_heads % cache->heads) return VG_ERR_INVALID_ARG;
  return q_heads / cache->heads > 4096 ? VG_ERR_UNSUPPORTED : VG_OK;
}

vg_status check_call(const vg_attention_desc *d, const vg_kv_cache *cache) {
  if (!d) return VG_ERR_INVALID_ARG;
  if (vg_status s = check_heads(d->n, d->q_heads, cache)) return s;
  if (!d->q || !d->out || !d->lens || !std::isfinite(d->scale)) return VG_ERR_INVALID_ARG;
  if (d->type != VG_TYPE_BF16 && d->type != VG_TYPE_FP16) return VG_ERR_INVALID_ARG;
  if (cache->type != VG_TYPE_E4M3 && cache->type != d->type) return VG_ERR_INVALID_ARG;
  for (int i = 0; i < 3; ++i)
    if (d->q_stride[i] % 8) return VG_ERR_ALIGNMENT;
  if (!aligned16(d->q) || !aligned16(d->out)) return VG_ERR_ALIGNMENT;
  return VG_OK;
}

AttnParams params_of(const vg_attention_desc *d, const vg_kv_cache *cache, void *workspace) {
  AttnParams p{};
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
  p.group = d->q_heads / cache->heads;
  p.group_magic = p.group == 1 ? 0 : uint32_t((uint64_t(1) << 32) / uint64_t(p.group)) + 1;
  p.box = cache_box_tokens(cache->page_size);
  p.c = d->scale * cache->k_scale * kLog2e;
  p.v_scale = cache->v_scale;
  return p;
}

// One launch over p.batch sequences of p.n nodes; what it is cut into goes to p.
vg_status launch(AttnParams &p, const Variant &v, int type, const vg_kv_cache *cache, int sms, vg_stream_t stream,
                 int *blocks = nullptr) {
  p.rows = p.n * p.group;
  p.blocks = (p.rows + v.rows - 1) / v.rows;
  // What a unit costs beside its tiles, in tiles, and half of it as the cut that
  // moves: less saves more than it unbalances.  Beginning and joining a unit
  // takes some 4 us.  The tcgen05 kernel's tiles take what a stream's chain of
  // scores, maxima and weights takes, whatever their bytes; the other's by their bytes (45 GB/s a block) but for
  // the smallest ones, and by the products from 64 rows on.  Measured over 1 to
  // 16 tiles of ragged batches: 18 sequences of 304 rows of 128, 6 tiles 100 us,
  // 8 106, 16 114; 30 units of 55 rows of 64 in E4M3, 26 us, 27, 32 and 40 with
  // 32; 50 units of 128 rows of 256, 2 tiles 36 us, 4 41.
  const bool wide = is_wide(p.d, p.rows);
  p.tile_log2 = wide ? 7 : 6;
  const int tile_bytes = (2 * p.d * (type == kE4M3 ? 1 : 2)) << p.tile_log2;
  p.least = std::max(1, 131072 / tile_bytes);
  p.extra = wide ? 6 : std::max(1, std::min({8, 16 * 16 / v.rows, 262144 / tile_bytes}));
  p.snap = p.extra / 2;
  // no more blocks than there can be tiles
  const int64_t most = int64_t(p.batch) * p.hkv * p.blocks *
                       ((int64_t(p.cache.max_pages) * p.cache.page_size + p.n + kTile - 1) / kTile);
  const unsigned grid = unsigned(std::min<int64_t>(sms, most));
  alignas(64) CUtensorMap kmap, vmap;
  std::memcpy(&kmap, cache->opaque, sizeof kmap);
  std::memcpy(&vmap, cache->opaque + kCacheMapWords, sizeof vmap);
  if (vg_status s = allow_smem(v)) return s;
  if (blocks) *blocks = int(grid);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(unsigned(v.threads));
  cfg.dynamicSmemBytes = size_t(v.smem);
  cfg.stream = as_cuda(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.pass == kOwn;
  VG_CUDA(cudaLaunchKernelEx(&cfg, v.fn, p, kmap, vmap));
  return VG_OK;
}

// Prefix attention: the kernels of its first two launches and the parts of its workspace.
// (The two overlap: each has partial results of its own.)
struct Behind {
  const Variant *prefix, *own;
  size_t partial, prefix_part, own_part, bytes;    // where: the prefix's partial results, both launches' results
};
vg_status behind_prefix(int n, int q_heads, const vg_kv_cache *cache, int sms, Behind &b) {
  const int group = q_heads / cache->heads, type = cache_type(*cache);
  const int64_t nodes = int64_t(cache->batch) * n, rows = nodes * group;
  // (node_of and q_of divide by multiplying)
  if (rows * group >= int64_t(1) << 32 || nodes * n >= int64_t(1) << 32 || rows >= int64_t(1) << 31)
    return VG_ERR_UNSUPPORTED;
  b.prefix = &pick_prefix(type, cache->head_dim, rows);
  b.own = &pick(type, cache->head_dim, n * group, true);
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  const size_t all = size_t(nodes) * size_t(q_heads);
  const size_t part = up(all * size_t(cache->head_dim) * sizeof(float)) + up(all * sizeof(float));
  b.partial = up(workspace_bytes_of(b.own->partial, sms));
  b.prefix_part = up(b.partial + size_t(sms) * 2 * size_t(b.prefix->partial) * sizeof(float));
  b.own_part = b.prefix_part + part;
  b.bytes = b.own_part + part;
  return VG_OK;
}

}  // namespace
}  // namespace vg

using namespace vg;

extern "C" vg_status vg_tree_attention_workspace_size(int n, int q_heads, const vg_kv_cache *cache,
                                                      size_t *bytes) {
  if (!bytes) return VG_ERR_INVALID_ARG;
  if (vg_status s = check_heads(n, q_heads, cache)) return s;
  int sms = 0;
  if (vg_status s = device_sms(&sms)) return s;
  *bytes = workspace_bytes_of(pick(cache_type(*cache), cache->head_dim, n * (q_heads / cache->heads)).partial, sms);
  return VG_OK;
}

extern "C" vg_status vg_tree_attention(const vg_attention_desc *d, const vg_kv_cache *cache,
                                       void *workspace, size_t workspace_bytes,
                                       vg_stream_t stream) {
  if (vg_status s = check_call(d, cache)) return s;
  int sms = 0;
  if (vg_status s = device_sms(&sms)) return s;
  if (sms > kMaxGrid) return VG_ERR_UNSUPPORTED;
  const int type = cache_type(*cache);
  const Variant &v = pick(type, cache->head_dim, d->n * (d->q_heads / cache->heads));
  if (!workspace || workspace_bytes < workspace_bytes_of(v.partial, sms)) return VG_ERR_WORKSPACE;
  if (!aligned16(workspace)) return VG_ERR_ALIGNMENT;
  AttnParams p = params_of(d, cache, workspace);
  return launch(p, v, type, cache, sms, stream);
}

extern "C" vg_status vg_prefix_attention_workspace_size(int n, int q_heads, const vg_kv_cache *cache,
                                                        size_t *bytes) {
  if (!bytes) return VG_ERR_INVALID_ARG;
  if (vg_status s = check_heads(n, q_heads, cache)) return s;
  int sms = 0;
  if (vg_status s = device_sms(&sms)) return s;
  Behind b;
  if (vg_status s = behind_prefix(n, q_heads, cache, sms, b)) return s;
  *bytes = b.bytes;
  return VG_OK;
}

extern "C" vg_status vg_prefix_attention(const vg_attention_desc *d, const vg_kv_cache *cache,
                                         const int32_t *prefix, const int32_t *prefix_pages,
                                         int max_prefix_pages, void *workspace,
                                         size_t workspace_bytes, vg_stream_t stream) {
  if (vg_status s = check_call(d, cache)) return s;
  if (max_prefix_pages < 0 || !prefix || (max_prefix_pages && !prefix_pages)) return VG_ERR_INVALID_ARG;
  if (int64_t(max_prefix_pages) * cache->page_size > kCacheMaxSlots) return VG_ERR_UNSUPPORTED;
  if ((reinterpret_cast<uintptr_t>(prefix) | reinterpret_cast<uintptr_t>(prefix_pages)) & 3) return VG_ERR_ALIGNMENT;
  int sms = 0;
  if (vg_status s = device_sms(&sms)) return s;
  if (sms > kMaxGrid) return VG_ERR_UNSUPPORTED;
  Behind b;
  if (vg_status s = behind_prefix(d->n, d->q_heads, cache, sms, b)) return s;
  if (!workspace || workspace_bytes < b.bytes) return VG_ERR_WORKSPACE;
  if (!aligned16(workspace)) return VG_ERR_ALIGNMENT;
  const int type = cache_type(*cache);
  AttnParams own = params_of(d, cache, workspace);
  if (max_prefix_pages == 0)
    return launch(own, pick(type, cache->head_dim, own.n * own.group), type, cache, sms, stream);
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  const int64_t all = int64_t(own.batch) * own.n * own.hq;
  auto part_at = [&](AttnParams &p, size_t at) {
    p.part = reinterpret_cast<float *>(ws + at);
    p.part_lse = p.part + (all * p.d + 63) / 64 * 64;
  };
  own.pass = kOwn;
  own.prefix = prefix;
  own.prefix_pages = max_prefix_pages;
  AttnParams first = own;
  part_at(own, b.own_part);
  part_at(first, b.prefix_part);
  first.pass = kPrefix;
  first.inner = own.n;
  first.inner_magic = own.n == 1 ? 0 : uint32_t((uint64_t(1) << 32) / uint64_t(own.n)) + 1;
  first.batch = 1;
  first.n = own.batch * own.n;
  first.cache.table = prefix_pages;
  first.cache.table_stride = first.cache.max_pages = max_prefix_pages;
  first.partial = reinterpret_cast<float *>(ws + b.partial);
  PrefixJoin j{};
  if (vg_status s = launch(first, *b.prefix, type, cache, sms, stream, &j.grid)) return s;
  if (vg_status s = launch(own, *b.own, type, cache, sms, stream)) return s;
  j.wide = is_wide(own.d, first.rows);
  j.e4m3 = type == kE4M3;
  j.sms = sms;
  j.rows = b.prefix->rows;
  j.partial = b.prefix->partial;
  j.columns = (b.prefix->partial - 2 * j.rows) / j.rows;
  j.state = j.rows * j.columns;
  j.lift = type == kBf16 ? 0.f : j.wide ? 7.f : 15.f;
  VG_CUDA(launch_prefix_join(own, first, j, as_cuda(stream)));
  return VG_OK;
}
