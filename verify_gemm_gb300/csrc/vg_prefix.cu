// vg_prefix.cu -- the third launch of vg_prefix_attention: joins what the rows of all
// sequences got from the shared prefix to what each got from its own slots.
//
// With the parts' outputs o_i and l_i = log2 of their sums of exponentials,
//     l = log2 sum 2^l_i,   o = sum 2^(l_i - l) o_i.
// A prefix unit of 256 rows that 19 blocks share is 2.5 MB of partial results: the block
// that ended last, alone, read them for 20 us.  Here every row and group of four columns has a
// thread of its own, and the whole device reads.  Consecutive lanes are
// consecutive rows, which lie side by side in the tcgen05 kernel's partial results.
#include "vg_attention.cuh"
#include "vg_prefix.h"

namespace vg {
namespace attn {
namespace {

constexpr int kJoinRows = 32, kJoinCols = 8;   // threads of a block: rows, groups of four columns

__device__ __forceinline__ float4 scaled_sum(float4 a, float wa, float4 b, float wb) {
  return make_float4(a.x * wa + b.x * wb, a.y * wa + b.y * wb, a.z * wa + b.z * wb, a.w * wa + b.w * wb);
}

// Columns 4 c .. 4 c + 3 of a row in a partial result.
__device__ __forceinline__ float4 partial_at(const PrefixJoin &j, const float *part, int row, int c) {
  if (j.wide) return __ldg(reinterpret_cast<const float4 *>(part) + c * j.rows + row);
  // mma.sync fragments: [row group][tile of 8 columns][lane][4]
  const int tiles = j.columns / 8, half = row % 16 / 8;
  const int nt = j.e4m3 ? c / 4 * 2 : c / 2, t = j.e4m3 ? c % 4 : c % 2 * 2;
  const float2 *at = reinterpret_cast<const float2 *>(part) + (row / 16 * tiles + nt) * 64 + (row % 8 * 4 + t) * 2 + half;
  if (j.e4m3) {                                // even columns in one tile, odd ones in the next
    const float2 even = __ldg(at), odd = __ldg(at + 64);
    return make_float4(even.x, odd.x, even.y, odd.y);
  }
  const float2 a = __ldg(at), b = __ldg(at + 2);
  return make_float4(a.x, a.y, b.x, b.y);
}

__global__ void __launch_bounds__(kJoinRows *kJoinCols)
    prefix_join_kernel(const __grid_constant__ AttnParams own, const __grid_constant__ AttnParams first,
                       const __grid_constant__ PrefixJoin j) {
  const int row = blockIdx.x * kJoinRows + threadIdx.x, head = blockIdx.y;
  const int c = blockIdx.z * kJoinCols + threadIdx.y;
  const bool real = row < first.rows && 4 * c < own.d;
  // whatever the other launches do not write may be read before they end
  const int node = node_of(first, row), h = head * own.group + row - node * own.group;
  const int b = own.n == 1 ? node : node / own.n;
  bool shares = false;
  const int shared = shared_slots(own);
  if (real) {
    const int64_t room = int64_t(own.cache.max_pages) * own.cache.page_size;
    shares = shared > 0 && min(int64_t(max(own.lens[b], 0)), room) >= shared &&
             node - b * own.n < (own.counts ? own.counts[b] : own.n);
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (!real) return;
  const int64_t at = int64_t(node) * own.hq + h;
  float lse = __ldcg(own.part_lse + at);
  float4 o = __ldcg(reinterpret_cast<const float4 *>(own.part + at * own.d) + c);
  if (shares) {
    // the prefix's unit on its line, and the blocks that hold a part of it
    Line line;
    line.tiles = Line::tiles_for(first, shared);
    line.extra = first.extra;
    line.snap = first.snap;
    const int units = first.hkv * first.blocks, block = row / j.rows;
    line.total = int64_t(line.tiles + line.extra) * units;
    line.runs = line.runs_of(first, j.grid, units);
    line.unit0 = int64_t(line.tiles + line.extra) * (head * first.blocks + block);
    const int from = line.first(), to = line.final(), in = row - block * j.rows;
    float theirs;
    float4 v;
    if (from == to) {
      theirs = __ldcg(first.part_lse + at);
      v = __ldcg(reinterpret_cast<const float4 *>(first.part + at * own.d) + c);
    } else {
      auto place = [&](int blk) { return first.partial + (int64_t(blk) * 2 + (blk == from)) * j.partial; };
      auto state = [&](int blk) { return __ldg(reinterpret_cast<const float2 *>(place(blk) + j.state) + in); };
      float m = -INFINITY, l = 0.f;
#pragma unroll 8
      for (int blk = from; blk <= to; ++blk) m = fmaxf(m, state(blk).x);
      v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int blk = from; blk <= to; ++blk) {
        const float2 s = state(blk);
        const float w = s.x == -INFINITY ? 0.f : ex2(s.x - m);
        l += s.x == -INFINITY ? s.y : s.y * w; // (the NaN of a wait that ran out is kept)
        v = scaled_sum(v, 1.f, partial_at(j, place(blk), in, c), w);
      }
      const bool empty = m == -INFINITY && l == 0.f;
      theirs = empty ? -INFINITY : m - j.lift + log2f(l);
      const float inv = empty ? 0.f : own.v_scale / l;
      v = make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
    }
    if (theirs != -INFINITY) {
      const float top = fmaxf(theirs, lse);
      const float wa = ex2(theirs - top), wb = lse == -INFINITY ? 0.f : ex2(lse - top), sum = wa + wb;
      o = scaled_sum(v, wa / sum, o, lse == -INFINITY ? 0.f : wb / sum);
      lse = top + log2f(sum);
    }
  }
  if (*static_cast<volatile int *>(own.error)) {   // what a wait that ran out has left is no number
    const float nan = __int_as_float(0x7FFFFFFF);
    o = make_float4(nan, nan, nan, nan);
    lse = nan;
  }
  const bool f16 = own.q_f16 != 0;
  reinterpret_cast<uint2 *>(static_cast<uint16_t *>(own.out) + at * own.d)[c] =
      make_uint2(pack_out(o.x, o.y, f16), pack_out(o.z, o.w, f16));
  if (own.lse && c == 0) own.lse[at] = lse * kLn2;
}

}  // namespace

cudaError_t launch_prefix_join(const AttnParams &own, const AttnParams &first, const PrefixJoin &j, cudaStream_t st) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(unsigned((first.rows + kJoinRows - 1) / kJoinRows), unsigned(own.hkv),
                     unsigned((own.d / 4 + kJoinCols - 1) / kJoinCols));
  cfg.blockDim = dim3(kJoinRows, kJoinCols);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, &prefix_join_kernel, own, first, j);
}

}  // namespace attn
}  // namespace vg
