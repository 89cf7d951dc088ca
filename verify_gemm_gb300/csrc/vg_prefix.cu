// vg_prefix.cu -- the third launch of vg_prefix_attention: joins what the rows of all
// sequences got from the shared prefix to what each got from its own slots.
//
// With the parts' outputs o_i and l_i = log2 of their sums of exponentials,
//     l = log2 sum 2^l_i,   o = sum 2^(l_i - l) o_i.
// A prefix unit of 256 rows that 19 blocks share is 2.5 MB of partial results: the block
// that ended last, alone, read them for 20 us.  Here rows and groups of four columns are spread
// over the device.  Consecutive lanes are consecutive rows, which lie side by side in the
// tcgen05 kernel's partial results; for the rows' outputs, which lie by columns, they change over in
// shared memory.
//
// The grid may begin while the launches before still write what it reads: every load of that lies behind the
// wait for them, and none goes by the read-only path, which promises memory that is not written meanwhile.
// Plain loads, and not ones that pass by L1: a row's states are read twice and by each of its groups of
// columns (4 rows of 2 cache heads of 128 over 25643 keys 24.8 us, 29.1 past L1).  64 registers a thread, so
// that four blocks an SM begin as soon as an SM is left (64 trees of 8 nodes 279 us, with 76 registers 285).
//
// Measured (the whole of vg_prefix_attention): 48 sequences of 1 node, 40 query and 8 cache heads of
// 128 in BF16, 8003 + up to 1201 keys, 69 us (91 with the join at the end of the first launch); of that
// the prefix takes 24, the own keys 38, this launch some 7, and what overlaps is not
// counted twice.
#include "vg_attention.cuh"
#include "vg_prefix.h"

namespace vg {
namespace attn {
namespace {

constexpr int kJoinRows = 32, kJoinWarps = 8;  // a warp's lanes are rows

__device__ __forceinline__ float4 scaled_sum(float4 a, float wa, float4 b, float wb) {
  return make_float4(a.x * wa + b.x * wb, a.y * wa + b.y * wb, a.z * wa + b.z * wb, a.w * wa + b.w * wb);
}

// Columns 4 c .. 4 c + 3 of a row in a partial result.
__device__ __forceinline__ float4 partial_at(const PrefixJoin &j, const float *part, int row, int c) {
  if (j.wide) return reinterpret_cast<const float4 *>(part)[c * j.rows + row];
  // mma.sync fragments: [row group][tile of 8 columns][lane][4]
  const int tiles = j.columns / 8, half = row % 16 / 8;
  const int nt = j.e4m3 ? c / 4 * 2 : c / 2, t = j.e4m3 ? c % 4 : c % 2 * 2;
  const float2 *at = reinterpret_cast<const float2 *>(part) + (row / 16 * tiles + nt) * 64 + (row % 8 * 4 + t) * 2 + half;
  if (j.e4m3) {                                // even columns in one tile, odd ones in the next
    const float2 even = at[0], odd = at[64];
    return make_float4(even.x, odd.x, even.y, odd.y);
  }
  const float2 a = at[0], b = at[2];
  return make_float4(a.x, a.y, b.x, b.y);
}

// kSplit warps share out a row's partial results, and each takes kGroups groups of four columns.
template <int kSplit, int kGroups>
__global__ void __launch_bounds__(kJoinRows *kJoinWarps, 4)
    prefix_join_kernel(const __grid_constant__ AttnParams own, const __grid_constant__ AttnParams first,
                       const __grid_constant__ PrefixJoin j) {
  constexpr int kCols = kJoinWarps / kSplit * kGroups;         // groups of four columns of the block
  __shared__ float tops[kSplit > 1 ? kJoinWarps : 1][kJoinRows], totals[kSplit > 1 ? kJoinWarps : 1][kJoinRows];
  __shared__ float4 values[kSplit][kCols][kJoinRows + 1];
  __shared__ float2 weights[kJoinRows];                        // of the prefix's result and of the own one
  __shared__ int64_t places[kJoinRows];                        // a row's place among all, -1: none
  __shared__ int2 blocks_of[kJoinRows];                        // that hold a part of the row's unit; x > y: none
  const int row = blockIdx.x * kJoinRows + threadIdx.x, head = blockIdx.y, y = threadIdx.y;
  const int group0 = y / kSplit * kGroups, c0 = int(blockIdx.z) * kCols + group0, mine = y % kSplit;
  // what may be read and worked out before the other launches end, by one warp
  if (y == 0) {
    const bool real = row < first.rows;
    const int node = node_of(first, row), h = head * own.group + row - node * own.group;
    const int b = own.n == 1 ? node : node / own.n;
    const int shared = shared_slots(own);
    int2 span = make_int2(1, 0);
    if (real) {
      if (shared > 0 && own.lens[b] >= shared && node - b * own.n < (own.counts ? own.counts[b] : own.n)) {
        Line<true> line;                                         // the prefix's unit on its line
        line.tiles = Line<true>::tiles_for(first, shared);
        line.extra = first.extra;
        line.snap = first.snap;
        const int units = first.hkv * first.blocks;
        line.total = int64_t(line.tiles + line.extra) * units;
        line.runs = min(int64_t(j.grid), max(line.wanted(first), int64_t(units)));
        line.unit0 = int64_t(line.tiles + line.extra) * (head * first.blocks + row / j.rows);
        span = make_int2(line.first(), line.final());
      }
    }
    blocks_of[threadIdx.x] = span;
    places[threadIdx.x] = real ? int64_t(node) * own.hq + h : -1;
  }
  __syncthreads();
  const int64_t at = places[threadIdx.x];
  const int from = blocks_of[threadIdx.x].x, to = blocks_of[threadIdx.x].y, in = row % j.rows;
  const bool shares = from <= to, cut = from < to;
  launch_before_has_ended();
  float theirs = -INFINITY, l = 0.f;
  float4 v[kGroups];
#pragma unroll
  for (int g = 0; g < kGroups; ++g) v[g] = make_float4(0.f, 0.f, 0.f, 0.f);
  auto here = [&](int g) { return 4 * (c0 + g) < own.d; };
  if (shares && !cut && mine == 0) {
    theirs = __ldcg(first.part_lse + at);
#pragma unroll
    for (int g = 0; g < kGroups; ++g)
      if (here(g)) v[g] = __ldcg(reinterpret_cast<const float4 *>(first.part + at * own.d) + c0 + g);
  }
  auto place = [&](int blk) { return first.partial + (int64_t(blk) * 2 + (blk == from)) * j.partial; };
  auto state = [&](int blk) { return reinterpret_cast<const float2 *>(place(blk) + j.state)[in]; };
  const int end = cut ? to : -1;
  float m = -INFINITY;
#pragma unroll 4
  for (int blk = from + mine; blk <= end; blk += kSplit) m = fmaxf(m, state(blk).x);
  if constexpr (kSplit > 1) {
    tops[y][threadIdx.x] = m;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kSplit; ++k) m = fmaxf(m, tops[y - mine + k][threadIdx.x]);
  }
#pragma unroll 2
  for (int blk = from + mine; blk <= end; blk += kSplit) {
    const float2 s = state(blk);
    const float w = s.x == -INFINITY ? 0.f : ex2(s.x - m);
    l += s.x == -INFINITY ? s.y : s.y * w;                     // (the NaN of a wait that ran out is kept)
#pragma unroll
    for (int g = 0; g < kGroups; ++g)
      if (here(g)) v[g] = scaled_sum(v[g], 1.f, partial_at(j, place(blk), in, c0 + g), w);
  }
#pragma unroll
  for (int g = 0; g < kGroups; ++g) values[mine][group0 + g][threadIdx.x] = v[g];
  if constexpr (kSplit > 1) totals[y][threadIdx.x] = l;
  __syncthreads();
  if (y == 0) {
    // this row's weights: of sums over the blocks, or of outputs
#pragma unroll
    for (int k = 1; k < kSplit; ++k) l += totals[k][threadIdx.x];
    float inv = 1.f;
    if (cut) {
      const bool empty = m == -INFINITY && l == 0.f;
      theirs = empty ? -INFINITY : m - j.lift + log2f(l);
      inv = empty ? 0.f : own.v_scale / l;
    }
    float lse = at >= 0 ? __ldcg(own.part_lse + at) : 0.f;
    float2 w = make_float2(0.f, 1.f);
    if (theirs != -INFINITY) {
      const float top = fmaxf(theirs, lse);
      const float wa = ex2(theirs - top), wb = lse == -INFINITY ? 0.f : ex2(lse - top), sum = wa + wb;
      w = make_float2(wa / sum * inv, wb / sum);
      lse = top + log2f(sum);
    }
    if (*static_cast<volatile int *>(own.error)) {             // what a wait that ran out has left is no number
      lse = __int_as_float(0x7FFFFFFF);
      w = make_float2(lse, lse);
    }
    weights[threadIdx.x] = w;
    if (at >= 0 && own.lse && blockIdx.z == 0) own.lse[at] = lse * kLn2;
  }
  __syncthreads();
  // now lanes are columns
  const bool f16 = own.q_f16 != 0;
  for (int i = y * kJoinRows + threadIdx.x; i < kJoinRows * kCols; i += kJoinRows * kJoinWarps) {
    const int r = i / kCols, k = i % kCols, c = blockIdx.z * kCols + k;
    const int64_t to_row = places[r];
    if (to_row < 0 || 4 * c >= own.d) continue;
    float4 theirs4 = values[0][k][r];
#pragma unroll
    for (int q = 1; q < kSplit; ++q) theirs4 = scaled_sum(theirs4, 1.f, values[q][k][r], 1.f);
    const float4 o = scaled_sum(theirs4, weights[r].x, __ldcg(reinterpret_cast<const float4 *>(own.part + to_row * own.d) + c),
                                weights[r].y);
    reinterpret_cast<uint2 *>(static_cast<uint16_t *>(own.out) + to_row * own.d)[c] =
        make_uint2(pack_out(o.x, o.y, f16), pack_out(o.z, o.w, f16));
  }
}

}  // namespace

cudaError_t launch_prefix_join(const AttnParams &own, const AttnParams &first, const PrefixJoin &j, cudaStream_t st) {
  cudaLaunchConfig_t cfg{};
  // As many warps a row as there are some partial results of it, and blocks enough to fill the device
  // twice: 132 parts of 12 rows of 256 columns, 64 blocks of a group of columns a warp 29 us for
  // the whole call, 16 blocks of four 42.
  const int64_t tiles = int64_t((first.rows + kJoinRows - 1) / kJoinRows) * own.hkv;
  const bool many = j.grid >= int64_t(4) * first.hkv * first.blocks, few = many && tiles * (own.d / 16) < 2 * j.sms;
  const int cols = few ? 4 : many ? 16 : 128;
  cfg.gridDim = dim3(unsigned((first.rows + kJoinRows - 1) / kJoinRows), unsigned(own.hkv),
                     unsigned((own.d + cols - 1) / cols));
  cfg.blockDim = dim3(kJoinRows, kJoinWarps);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, few ? &prefix_join_kernel<kJoinWarps, 1> : many ? &prefix_join_kernel<kJoinWarps, 4> : &prefix_join_kernel<1, 4>, own, first, j);
}

}  // namespace attn
}  // namespace vg
