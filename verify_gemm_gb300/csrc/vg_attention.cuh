// vg_attention.cuh -- the kernel of vg_tree_attention: the nodes of each sequence's tree
// over its paged cache.
//
// The rows that share a cache head (n nodes x the query heads of the group,
// node-major) are one operand; a unit is (sequence, cache head, block of up
// to 16 RW rows), and its keys are cut into tiles of 64.  With scores in
// base 2, x = c q.k (c = scale log2 e), each row keeps a running maximum m,
// sum l and output o:
//     m' = max(m, x),  l' = l 2^(m - m') + 2^(x - m'),  o' = o 2^(m - m') + v 2^(x - m').
//
// Keys and values are read once from HBM, which bounds long 16-bit caches under up
// to 32 rows a head (0.9 of a copy's rate; of 36 us for 164 MB some 9 are beginnings,
// cuts and joining).  One block per SM, because a ring that fills its
// shared memory is what keeps HBM busy: two warps, one for K and one for V,
// copy tiles by TMA (a box of a page at a time, 128-byte swizzle) into its
// slots; eight consumer warps share out rows (RW groups of 16) and keys (32 at
// a time, 16 for heads of 256), each with a softmax state of its own, and are
// joined in shared memory at the end of a unit.  Keys and not only rows are
// shared out because a chain of 8 nodes with 2 query heads a cache head has 16
// rows in all, one fragment of mma.sync, which carries the products: at
// 16 rows they take a fifth of the time that the bytes take.
//
// A warp that waits for a step's dependent chain (scores, maximum, weights,
// output) leaves its slots held, so with more rows the warps' latency and not
// the bytes sets the pace.  Measured (heads of 128, a kernel by itself):
//     8003 keys of 40 heads, 8 rows, BF16        164 MB   34.5 us  4.75 TB/s
//     262001 keys of 8 heads, 20 rows, E4M3      537 MB  155 us    3.5 TB/s
//     131000 keys of 8 heads, 20 rows, BF16      537 MB   93 us    5.8 TB/s
//     130 keys of 8 heads of 64, 4 rows: 6.6 us, a launch and a chain of waits
// (With 16 keys a step, one copying warp and a page number fetched for each
// tile the second took 227 us.  Two row groups a warp, which read each key once
// and not twice for 20 rows, made it 194 us: q no longer stays in registers.)
//
// The tiles of all units form one line that is cut into equal runs, one a
// block, from the lengths in device memory: ragged lengths and long single
// sequences fill the device alike, and the host need not know a length.  A
// unit that is cut leaves partial results in the workspace; the block that
// arrives last joins them in block order, so the bits do not depend on which
// that is.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>

#include "vg_cache.h"
#include "vg_device.cuh"

namespace vg {
namespace attn {

constexpr int kTile = 64;                     // keys of a tile (mma.sync)
constexpr int kConsumers = 8;                 // warps
constexpr int kAttnThreads = (kConsumers + 4) * 32;   // three warpgroups, one warp of the last copies
// Registers a thread: 168 at the launch (384 x 168 = 64512); the producer's
// warpgroup gives up what the consumers' two take, 128 x 56 + 256 x 224 = 64512.
constexpr int kProducerRegs = 56, kConsumerRegs = 224;
constexpr int kHeader = 256;                  // workspace: error word, then ...
constexpr int kMaxGrid = 512;                 // ... three counters for each block
constexpr uint64_t kWaitNs = 2000000000ull;   // bound of every wait
constexpr int kErrAttnWait = 16;              // the error word of a wait that ran out
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

enum { kBf16 = 0, kF16 = 1, kE4M3 = 2 };

// Weights are 2^(x - m + lift).  FP16 holds them with 11 bits down to 2^-14
// only, so there they are lifted to the top of its range: a weight then loses
// bits from 2^-29 of the largest on.  o and l carry the same factor.
template <int kType>
constexpr float kLift = kType == kBf16 ? 0.f : 15.f;

struct AttnParams {
  const void *q;
  void *out;
  float *lse;
  const int32_t *lens, *counts;
  const uint64_t *tree;
  int64_t qs[3];
  CacheView cache;
  int *error;
  uint32_t *arrived;                // [3][kMaxGrid]: units', and groups' by their first block's place
  float *partial;                   // [grid][2] of (rows x (head_dim padded) + 2 rows)
  int batch, n, hq, hkv, d, q_f16;
  int rows, blocks;                 // rows that share a cache head, row blocks of a unit
  int group;                        // query heads that share a cache head
  uint32_t group_magic;             // 2^32 / group + 1
  int tile_log2;                    // keys of a tile
  int box, least, extra, snap;      // tokens of a TMA box; tiles: of a run at least, a unit costs, a cut moves
  float c, v_scale;                 // scale * k_scale * log2 e
};

// Divisions by numbers that only the launch knows take some 150 clocks, and a
// unit's beginning and end are a chain of them.
// row / group, exact for row < 2^32 / group (rows are below 2^20 / 4).
__device__ __forceinline__ int node_of(const AttnParams &p, int row) {
  return p.group == 1 ? row : int(__umulhi(uint32_t(row), p.group_magic));
}
// Cache head and row block of unit u of a sequence.
__device__ __forceinline__ int head_of(const AttnParams &p, int u) { return p.blocks == 1 ? u : u / p.blocks; }
__device__ __forceinline__ int block_of_rows(const AttnParams &p, int u) { return p.blocks == 1 ? 0 : u % p.blocks; }

// ------------------------------------------------------------------ joining
// The blocks first .. final of a cut unit leave partial results, and the one
// that arrives last joins them in the blocks' order.  Where that is much to
// read for one block (some 120 GB/s), groups of about the square root of them
// are joined first, each by its last, into its first block's place: 80 blocks
// of 256 rows, 10.6 MB, took 110 us to join.  A second step costs what half a
// megabyte does.
struct Join {
  int lo, hi, step;                 // the blocks that are joined now
  int group, first, final;          // blocks of a group (all, when there is one step)
  __device__ __forceinline__ Join(int first_, int final_, int block, int most)
      : first(first_), final(final_) {
    const int count = final - first + 1;
    group = count;
    if (count > most)
      for (group = 2; group * group < count;) ++group;
    lo = first + (block - first) / group * group;
    hi = min(lo + group - 1, final);
    step = 1;
  }
  __device__ __forceinline__ bool last() const { return lo == first && hi == final; }
  __device__ __forceinline__ void next() {
    lo = first;
    hi = final;
    step = group;
  }
  __device__ __forceinline__ uint32_t members() const { return uint32_t((hi - lo) / step) + 1; }
  // A block has a part in at most one unit that it is the first block of and
  // in one that it is not.
  __device__ __forceinline__ uint32_t *counter(const AttnParams &p) const {
    return p.arrived + (last() ? 0 : lo == first ? kMaxGrid : 2 * kMaxGrid) + lo;
  }
};
template <typename L>
constexpr int kJoinAtOnce = 131072 / L::kPartial > 12 ? 131072 / L::kPartial : 12;

// ----------------------------------------------------------------- layout
template <int kType, int DC, int RW>
struct Cfg {
  static constexpr int kSize = kType == kE4M3 ? 1 : 2;
  static constexpr int kKeys = kTile;
  // a key's row comes in chunks of 128 bytes (64 for E4M3 heads of 64): half
  // as many of twice the size move an E4M3 tile faster
  static constexpr int kRow = kType == kE4M3 && DC == 1 ? 64 : 128;
  static constexpr int kElems = kRow / kSize;
  static constexpr int kChunks = (DC * 64 + kElems - 1) / kElems;
  static constexpr int kChunk = kTile * kRow;
  static constexpr int kSlot = kChunks * kChunk;         // one tile of K or of V
  static constexpr int D = DC * 64;
  static constexpr int kRows = 16 * RW;
  // keys of a step: 32 halve the maxima, shuffles and waits of a key against
  // 16 and give the products twice the chains; o of 256 columns leaves room for 16
  static constexpr int SK = DC == 4 ? 16 : 32;
  static constexpr int KW = kConsumers / RW;             // key warps of a row group
  static constexpr int KT = KW < kTile / SK ? KW : kTile / SK;   // ... that share a tile
  static constexpr int NG = KW / KT;                     // groups that take tiles in turn
  static constexpr int kSub = kTile / SK / KT;           // steps of a warp in a tile
  static constexpr int NT = D / 8;                       // output tiles of 8 columns
  static constexpr bool kQReg = DC <= 2;                 // q fragments stay in registers
  static constexpr int kQRow = D * 2 + 16;               // q row in shared memory, padded
  static constexpr int kQBytes = kRows * kQRow;
  static constexpr int kWarpState = NT * 32 * 16;        // one warp's o
  // every warp's o is laid open for the joining, at most 64 KB at a time
  static constexpr int kPasses = DC >= 3 && KW > 1 ? 2 : 1;
  static constexpr int kScratch = KW == 1 ? 0 : kConsumers * kWarpState / kPasses;
  static constexpr int TPW = NT / KW;                    // tiles that a warp joins
  static constexpr int kState = kConsumers * 16 * 8;     // m, l of each warp's rows
  // header: barriers, flags and the tiles' page bits
  static constexpr int kMaxSlots = 16;
  static constexpr int kFixed = 1024 + kState + kRows * 4 + kQBytes + kScratch;
  static constexpr int kFit = (227 * 1024 - 1024 - kFixed) / kSlot;
  // A slot always serves the same group: a warp that waits for a slot's next
  // filling has then seen the one before (a phase's parity tells only
  // neighbours apart, and copies land in any order).
  static constexpr int kSlots = (kFit > kMaxSlots ? kMaxSlots : kFit) / (2 * NG) * (2 * NG);
  static constexpr int kSmem = 1024 + kFixed + kSlots * kSlot;
  static_assert(kSlots >= 2 * NG, "room for a tile of K and one of V of each group");
  // floats of a partial result: o in fragment order, then m and l
  static constexpr int kPartial = RW * NT * 32 * 4 + 2 * kRows;
};

// ------------------------------------------------------------- small pieces
template <int kType>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                    uint32_t b1) {
  if constexpr (kType == kBf16)
    mma_bf16(c, a[0], a[1], a[2], a[3], b0, b1);
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Four E4M3 codes as FP16 pairs, exact.
__device__ __forceinline__ void e4m3_f16(uint32_t w, uint32_t &lo, uint32_t &hi) {
  asm("{ .reg .b16 a, b; mov.b32 {a, b}, %2;\n"
      "cvt.rn.f16x2.e4m3x2 %0, a; cvt.rn.f16x2.e4m3x2 %1, b; }"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
template <int kType>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  uint32_t y;
  if constexpr (kType == kBf16)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(y) : "f"(b), "f"(a));
  else
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(y) : "f"(b), "f"(a));
  return y;
}
__device__ __forceinline__ uint32_t pack_out(float a, float b, bool f16) {
  return f16 ? pack2<kF16>(a, b) : pack2<kBf16>(a, b);
}
// The power of two that a row of q with this largest magnitude is divided by
// before it goes to FP16: it brings the row to the top of FP16's range.
__device__ __forceinline__ int q_exponent(float top) {
  int e = 0;
  if (top > 0.f && top < INFINITY) {
    frexpf(top, &e);
    e = min(max(e - 14, -100), 120);
  }
  return e;
}
// Nonzero where one of the cache's elements in a word is infinite or NaN: x 0
// is a NaN then, else a zero; of E4M3 codes only 0x7F and 0xFF are.
template <int kType>
__device__ __forceinline__ uint32_t nonfinite_bits(uint32_t w) {
  uint32_t y;
  if constexpr (kType == kE4M3) {
    y = ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
    return y;
  } else if constexpr (kType == kBf16) {
    asm("fma.rn.bf16x2 %0, %1, %2, %2;" : "=r"(y) : "r"(w), "r"(0u));
  } else {
    asm("fma.rn.f16x2 %0, %1, %2, %2;" : "=r"(y) : "r"(w), "r"(0u));
  }
  return y & 0x7FFF7FFFu;
}
template <int kType>
__device__ __forceinline__ uint32_t finite_mask(uint32_t w) {
  constexpr uint32_t e = kType == kBf16 ? 0x7F80u : 0x7C00u;
  return ((w & e) == e ? 0u : 0xFFFFu) | (((w >> 16) & e) == e ? 0u : 0xFFFF0000u);
}

// Byte offset in a slot of 16-byte piece `c` + `more` of key `key` (`more`
// stays in the chunk of `c`): TMA's 128-byte or 64-byte swizzle.
template <typename L>
__device__ __forceinline__ uint32_t spot(uint32_t key, uint32_t c, uint32_t more = 0) {
  constexpr uint32_t N = L::kRow / 16;
  const uint32_t in = c % N + more;
  return c / N * L::kChunk +
         (N == 8 ? key * 128 + ((in ^ (key & 7)) << 4) : key * 64 + ((in ^ ((key >> 1) & 3)) << 4));
}

__device__ __forceinline__ void tma_4d(uint32_t dst, const CUtensorMap *map, int x, int token,
                                       int head, int page, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(map), "r"(x), "r"(token), "r"(head), "r"(page), "r"(bar)
      : "memory");
}

// Bounded wait for a phase; gives up at once after another wait has failed.
__device__ __forceinline__ bool wait_phase(uint32_t bar, uint32_t parity, volatile int *failed,
                                           int *error) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t end = globaltimer() + kWaitNs;
  while (!mbar_try_wait(bar, parity)) {
    if (*failed) return false;
    if (globaltimer() > end) {
      atomicCAS(error, 0, kErrAttnWait);
      *failed = 1;
      return false;
    }
  }
  return true;
}

// ------------------------------------------------------------------ the line
// Where a block is on the line: unit u (= head * blocks + row block) of
// sequence b, and the unit's tiles [t0, t1) that are the block's.  A unit's
// place on the line is `extra` + its tiles long, as beginning and joining a
// unit costs about as much as `extra` tiles: without that, blocks with a
// second unit ended 7 us after the others (39 us in all).  A cut less than
// `snap` places from a unit's end moves there: it would cost a joining.
struct Line {
  int64_t total, end, unit0;        // the line's length, the run's end, where the unit begins
  int64_t runs;                     // blocks that have a run
  int b, u, units, extra, snap, tiles, t0, t1;
  int len, count;

  __device__ __forceinline__ static int used(const AttnParams &p, int b, int &len) {
    // no slot past the table exists: such lengths end with it
    const int64_t room = int64_t(p.cache.max_pages) * p.cache.page_size;
    len = int(min(int64_t(max(p.lens[b], 0)), room));
    return p.counts ? min(max(p.counts[b], 0), p.n) : p.n;
  }
  __device__ __forceinline__ static int tiles_for(const AttnParams &p, int tokens) {
    return max(1, (tokens + (1 << p.tile_log2) - 1) >> p.tile_log2);
  }
  __device__ __forceinline__ static int tiles_of(const AttnParams &p, int b) {
    int len;
    const int count = used(p, b, len);
    return tiles_for(p, len + count);
  }
  // The whole warp computes it.
  __device__ void init(const AttnParams &p, int units_) {
    const int lane = threadIdx.x % 32;
    units = units_;
    extra = p.extra;
    snap = p.snap;
    auto long_of = [&](int i) { return i < p.batch ? tiles_of(p, i) + extra : 0; };
    const int own = long_of(lane);              // of the first 32 sequences
    int64_t sum = own;
    for (int i = 32 + lane; i < p.batch; i += 32) sum += long_of(i);
#pragma unroll
    for (int w = 16; w; w /= 2) sum += __shfl_xor_sync(~0u, sum, w);
    total = sum * units;
    // a unit is cut into runs of at least 128 KB: shorter ones cost more in the
    // joining than they save
    const int64_t wanted = total < int64_t(1) << 32 ? uint32_t(total) / uint32_t(p.least) : total / p.least;
    runs = min(int64_t(gridDim.x), max(wanted, int64_t(p.batch) * units));
    const int64_t mine = min(int64_t(blockIdx.x), runs);
    int64_t at;
    if (total * runs < int64_t(1) << 32) {      // 64-bit divisions are slow
      at = uint32_t(total * mine) / uint32_t(runs);
      end = mine < runs ? uint32_t(total * (mine + 1)) / uint32_t(runs) : at;
    } else {
      at = total * mine / runs;
      end = mine < runs ? total * (mine + 1) / runs : at;
    }
    // the sequence that holds place `at`
    int64_t before = 0;
    int length = 1;
    b = 0;
    for (int i0 = 0; i0 < p.batch; i0 += 32) {
      const int each = i0 ? long_of(i0 + lane) : own;
      int64_t run = each;
#pragma unroll
      for (int w = 1; w < 32; w *= 2) {
        const int64_t y = __shfl_up_sync(~0u, run, w);
        if (lane >= w) run += y;
      }
      const uint32_t over = __ballot_sync(~0u, (before + run) * units > at);
      if (over) {
        const int f = __ffs(over) - 1;
        length = __shfl_sync(~0u, each, f);
        b = i0 + f;
        before += __shfl_sync(~0u, run, f) - length;
        break;
      }
      before += __shfl_sync(~0u, run, 31);
    }
    const int64_t in = at - before * units;
    u = in < int64_t(1) << 32 ? int(uint32_t(in) / uint32_t(length)) : int(in / length);
    tiles = length - extra;
    count = b < p.batch ? used(p, b, len) : 0;
    const int off = int(in - int64_t(u) * length);
    unit0 = at - off;
    t0 = off <= snap ? 0 : max(0, off - extra);
    if (off > snap && length - off <= snap)
      next(p);                                  // the run begins with the unit after
    else
      fill(p);
  }
  __device__ __forceinline__ void fill(const AttnParams &p) {
    const int64_t cut = end - unit0;            // where the run ends, from the unit's beginning
    const int length = tiles + extra;
    t1 = cut >= length ? tiles : cut <= snap ? 0 : length - cut <= snap ? tiles : max(0, int(cut) - extra);
  }
  __device__ __forceinline__ bool valid() const { return t0 < t1; }
  __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == tiles; }
  __device__ __forceinline__ void next(const AttnParams &p) {
    unit0 += tiles + extra;
    t0 = 0;
    t1 = 0;
    if (unit0 >= end) return;
    if (++u == units) {
      u = 0;
      ++b;
      count = used(p, b, len);
      tiles = tiles_for(p, len + count);
    }
    fill(p);
  }
  // The blocks that hold the unit's first tile and its last: a cut up to
  // max(snap, extra) begins a run at tile 0, and one in the last `snap` places
  // at the next unit.
  __device__ __forceinline__ int first() const { return block_of(unit0 + min(max(snap, extra), latest())); }
  __device__ __forceinline__ int final() const { return block_of(unit0 + latest()); }
  __device__ __forceinline__ int latest() const {
    return min(tiles + extra - 1, max(snap, tiles + extra - snap - 1));
  }
  // The last block whose run, before its cuts are moved, begins at place x or before.
  __device__ __forceinline__ int block_of(int64_t place) const {
    const int64_t x = (place + 1) * runs + total - 1;
    return (x < int64_t(1) << 32 ? int(uint32_t(x) / uint32_t(total)) : int(x / total)) - 1;
  }
};

// One warp copies the K (kv = 0) or V tiles of the block's run into the ring
// of NS slots, K and V in turn, and leaves for each tile a bit for every 16
// keys that there are in page_ok[tile of the run % 16].  What the error word
// says at the beginning goes to *stale before the first V tile can be seen.
// The page numbers of 32 boxes are fetched at a time, one a lane, and the
// next 32 while those are copied: a fetch for each tile cost 1200 clocks a
// tile, more than an E4M3 tile takes to arrive (2.8 TB/s).
template <typename L, int NS>
__device__ void copy_tiles(const AttnParams &p, Line at, const CUtensorMap *map, int kv,
                           uint32_t ring0, uint32_t full0, uint32_t empty0, uint32_t *page_ok,
                           volatile int *failed, volatile int *stale) {
  const int lane = threadIdx.x % 32;
  const int before = kv == 1 && lane == 0 ? *static_cast<volatile int *>(p.error) : 0;
  const int boxes = L::kKeys / p.box, copies = boxes * L::kChunks;
  const int page_boxes = p.cache.page_size / p.box;
  int s = kv, n = 0;
  uint32_t par = 1;                                      // slots start empty
  int pages = -1, ahead = -1, seq = -1, window = -1;     // the numbers held, of which sequence and window
  bool going = true;
  for (; going && at.valid(); at.next(p)) {
    const int head = head_of(p, at.u);
    const int total = at.len + at.count;
    const int32_t *table = p.cache.table + at.b * p.cache.table_stride;
    auto fetch = [&](int window) {
      const int box = window * 32 + lane, i = box / page_boxes;
      return box * p.box < total && i < p.cache.max_pages ? table[i] : -1;
    };
    if (at.b != seq || at.t0 * boxes / 32 != window) {   // (a sequence's heads have the same pages)
      seq = at.b;
      window = at.t0 * boxes / 32;
      pages = fetch(window);
      ahead = fetch(window + 1);
    }
    for (int t = at.t0; t < at.t1; ++t, ++n) {
      if (t * boxes / 32 != window) {
        pages = ahead;
        ahead = fetch(++window + 1);
      }
      // lane = box * chunks + chunk; a box without a page, or past the end,
      // is copied from outside the tensor: zeros, and no traffic
      const int box = lane / L::kChunks, chunk = lane % L::kChunks;
      const int number = t * boxes + box;
      int page = __shfl_sync(~0u, pages, number % 32);
      const bool ok = lane < copies && page >= 0 && page < p.cache.pages;
      if (!ok) page = int(p.cache.pages);
      const int token = ok ? number % page_boxes * p.box : 0;
      uint32_t bits = ok ? ((1u << (p.box / 16)) - 1) << (box * (p.box / 16)) : 0;
      bits = __reduce_or_sync(~0u, bits);
      // a slot that did not become free may still be filled or read: nothing more is copied
      going = __all_sync(~0u, wait_phase(empty0 + 8 * s, par, failed, p.error));
      if (!going) break;
      const uint32_t bar = full0 + 8 * s;
      if (lane == 0) {
        if (kv == 0) page_ok[n % 16] = bits;
        else if (n == 0) *stale = before;
        mbar_arrive_expect_tx(bar, L::kSlot);
      }
      __syncwarp();
      if (lane < copies)
        tma_4d(ring0 + s * L::kSlot + chunk * L::kChunk + box * p.box * L::kRow, map,
               chunk * L::kElems, token, head, page, bar);
      if ((s += 2) >= NS) {
        s = kv;
        par ^= 1;
      }
    }
  }
  // every copy has been read, so has landed, before the block may end; after
  // a failure they get 10 ms to land
  for (int k = 0; k < NS / 2; ++k) {
    wait_phase(empty0 + 8 * s, par, failed, p.error);
    if ((s += 2) >= NS) {
      s = kv;
      par ^= 1;
    }
  }
  if (*failed) {
    const uint64_t end = globaltimer() + 10000000;
    while (globaltimer() < end) __nanosleep(1000);
  }
}

// Joins another result of the same rows, o2 (tile i), (m2, l2), to o, m, l.
template <int NT, typename F>
__device__ __forceinline__ void merge(float (&o)[NT][4], float (&m)[2], float (&l)[2],
                                      const float2 (&other)[2], F &&o2) {
  float wa[2], wb[2];
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const float top = fmaxf(m[r], other[r].x);
    wa[r] = m[r] == -INFINITY ? 0.f : ex2(m[r] - top);
    wb[r] = other[r].x == -INFINITY ? 0.f : ex2(other[r].x - top);
    l[r] = l[r] * wa[r] + other[r].y * wb[r];
    m[r] = top;
  }
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const float4 v = o2(i);
    o[i][0] = o[i][0] * wa[0] + v.x * wb[0];
    o[i][1] = o[i][1] * wa[0] + v.y * wb[0];
    o[i][2] = o[i][2] * wa[1] + v.z * wb[1];
    o[i][3] = o[i][3] * wa[1] + v.w * wb[1];
  }
}

// Column of element e of output tile nt in thread t of a quad.  E4M3: the
// transposed load hands out pairs of columns, tile 2k has the even ones.
template <int kType>
__device__ __forceinline__ int out_col(int nt, int t, int e) {
  return kType == kE4M3 ? 16 * (nt / 2) + 4 * t + 2 * e + (nt & 1) : 8 * nt + 2 * t + e;
}

template <int kType, int DC, int RW>
__global__ void __launch_bounds__(kAttnThreads, 1)
    attention_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ CUtensorMap kmap,
                     const __grid_constant__ CUtensorMap vmap) {
  using L = Cfg<kType, DC, RW>;
  extern __shared__ uint8_t raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  uint8_t *ring = smem;
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::kSlots * L::kSlot);
  uint32_t *page_ok = reinterpret_cast<uint32_t *>(bars + 2 * L::kMaxSlots);   // [kMaxSlots]
  volatile int *failed = reinterpret_cast<volatile int *>(page_ok + L::kMaxSlots);
  int *last = const_cast<int *>(failed) + 1;
  volatile int *stale = failed + 2;
  float2 *state = reinterpret_cast<float2 *>(smem + L::kSlots * L::kSlot + 1024);   // [warp][16]
  float *q_unit = reinterpret_cast<float *>(state) + L::kState / 4;                  // [kRows]
  uint8_t *q_smem = reinterpret_cast<uint8_t *>(q_unit + L::kRows);
  uint8_t *scratch = q_smem + L::kQBytes;
  constexpr int NS = L::kSlots;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const uint32_t full0 = smem_addr(bars), empty0 = smem_addr(bars + L::kMaxSlots);
  if (tid == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(&kmap) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&vmap) : "memory");
    *failed = *stale = 0;
    for (int s = 0; s < NS; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, L::KT * RW);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  Line at;
  at.init(p, p.hkv * p.blocks);

  if (warp >= kConsumers) {
    // ------------------------------------------------------------ producer
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kProducerRegs));
    const int kv = warp - kConsumers;                    // one warp copies K, one V
    if (kv > 1) return;
    copy_tiles<L, NS>(p, at, kv ? &vmap : &kmap, kv, smem_addr(ring), full0, empty0, page_ok, failed,
                      stale);
    return;
  }

  // ------------------------------------------------------------- consumers
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kConsumerRegs));
  const int g = lane >> 2, t = lane & 3;
  const int rw = warp / L::KW, kg = warp % L::KW;        // row group, key warp
  const int grp = kg / L::KT, kt = kg % L::KT;
  const uint32_t ring0 = smem_addr(ring), q0 = smem_addr(q_smem);
  uint32_t tile_no = 0;                                  // tiles of the block so far
  // A unit's q goes to shared memory by way of registers, a warp a row.  With
  // up to 32 rows the next unit's is fetched before this one's results are
  // joined: under load a fetch takes 3 us.
  constexpr int kQn = L::kRows / kConsumers;
  // A unit of one tile occupies one group of key warps only; the others go on
  // to the next units meanwhile.  Each row group's KT warps are by themselves
  // then: their q lies in the first one's part of the scratch memory, and they
  // meet at a barrier of their own.  (1640 units of one tile 36.6 -> 17 us.)  Heads
  // above 128 have no room for it, and E4M3 heads above 64 no registers: their
  // long sequences would take 4 % more.
  constexpr bool kSolo = L::NG > 1 && L::kPasses == 1 && !(kType == kE4M3 && DC > 1);
  auto solo = [&](const Line &u) { return kSolo && u.valid() && u.tiles == 1; };
  const int pair = 2 + rw * L::NG + grp;
  uint8_t *solo_q = scratch + (rw * L::KW + grp * L::KT) * L::kWarpState;
  float *solo_unit = reinterpret_cast<float *>(solo_q + 16 * L::kQRow);
  static_assert(!kSolo || 16 * L::kQRow + 64 <= L::kWarpState * L::KT, "room for q");
  // (E4M3 has no registers for it: 156 -> 170 us over 262001 keys.)
  constexpr bool kAheadQ = L::kRows <= 32 && kType != kE4M3;
  uint4 qv[kQn];
  auto q_row = [&](const Line &u, int r) {
    const int row = block_of_rows(p, u.u) * L::kRows + r, node = node_of(p, row);
    if (row >= p.rows || lane * 8 >= p.d) return make_uint4(0, 0, 0, 0);
    return *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.q) + u.b * p.qs[0] + node * p.qs[1] +
                                            (head_of(p, u.u) * p.group + row - node * p.group) * p.qs[2] + lane * 8);
  };
  auto fetch_q = [&](const Line &u) {
#pragma unroll
    for (int k = 0; k < kQn; ++k) qv[k] = q_row(u, k * kConsumers + warp);
  };
  // E4M3: in FP16, each row brought to the top of its range by a power of two,
  // which keeps every bit of a BF16 row that counts (2^-29 of the row's
  // largest element and more)
  auto put_q = [&](uint4 v, uint8_t *to, float *unit) {
    if constexpr (kType == kE4M3) {
      float f[8];
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
      float top = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint16_t x = uint16_t(w[e / 2] >> (16 * (e & 1)));
        f[e] = p.q_f16 ? __half2float(__ushort_as_half(x)) : __bfloat162float(__ushort_as_bfloat16(x));
        top = fmaxf(top, fabsf(f[e]));
      }
#pragma unroll
      for (int m = 16; m; m /= 2) top = fmaxf(top, __shfl_xor_sync(~0u, top, m));
      const int e = q_exponent(top);
      const float down = ldexpf(1.f, -e);
      v = make_uint4(pack2<kF16>(f[0] * down, f[1] * down), pack2<kF16>(f[2] * down, f[3] * down),
                     pack2<kF16>(f[4] * down, f[5] * down), pack2<kF16>(f[6] * down, f[7] * down));
      if (lane == 0) *unit = ldexpf(1.f, e);
    }
    if (lane * 8 < L::D) *reinterpret_cast<uint4 *>(to + lane * 16) = v;
  };
  bool fetched = kAheadQ && at.valid() && !solo(at);
  if (fetched) fetch_q(at);
  for (; at.valid();) {
    Line after = at;
    after.next(p);
    const bool alone = solo(at);
    if (alone && tile_no % L::NG != uint32_t(grp)) {
      ++tile_no;
      fetched = false;
      at = after;
      continue;
    }
    const int head = head_of(p, at.u), row0 = block_of_rows(p, at.u) * L::kRows;
    uint32_t q_at = q0 + rw * 16 * L::kQRow;             // of this warp's rows
    const float *unit = q_unit + rw * 16;
    if (alone) {
      constexpr int kN = 16 / L::KT;
      uint4 v[kN];
#pragma unroll
      for (int k = 0; k < kN; ++k) v[k] = q_row(at, rw * 16 + k * L::KT + kt);
#pragma unroll
      for (int k = 0; k < kN; ++k)
        put_q(v[k], solo_q + (k * L::KT + kt) * L::kQRow, solo_unit + k * L::KT + kt);
      q_at = smem_addr(solo_q);
      unit = solo_unit;
      named_bar(pair, L::KT * 32);
    } else {
      if (!fetched) fetch_q(at);
#pragma unroll
      for (int k = 0; k < kQn; ++k) {
        const int r = k * kConsumers + warp;
        put_q(qv[k], q_smem + r * L::kQRow, q_unit + r);
      }
      named_bar(1, kConsumers * 32);
    }
    fetched = false;

    uint32_t qf[L::kQReg ? DC * 4 : 1][4];
    auto load_q = [&](uint32_t (&a)[4], int ks) {
      if constexpr (kType == kE4M3) {
        // k order of a step: thread t has elements 4t .. 4t + 3
        const uint32_t base = q_at + g * L::kQRow + ks * 32 + t * 8;
        const uint2 lo = lds64(base), hi = lds64(base + 8 * L::kQRow);
        a[0] = lo.x;
        a[1] = hi.x;
        a[2] = lo.y;
        a[3] = hi.y;
      } else {
        ldsm4(a, q_at + (lane & 15) * L::kQRow + ks * 32 + (lane >> 4) * 16);
      }
    };
    if constexpr (L::kQReg) {
#pragma unroll
      for (int ks = 0; ks < DC * 4; ++ks) load_q(qf[ks], ks);
    }
    float cr[2] = {p.c, p.c};
    if constexpr (kType == kE4M3) {
      cr[0] *= unit[g];
      cr[1] *= unit[g + 8];
    }
    // the drafted nodes that this thread's two rows attend to
    uint64_t word[2];
    const uint64_t used = at.count >= 64 ? ~0ull : (1ull << at.count) - 1;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int node = node_of(p, row0 + rw * 16 + g + 8 * r);
      word[r] = 0;
      if (node < p.n)
        word[r] = used & (p.tree ? p.tree[int64_t(at.b) * p.n + node] : ~0ull >> (63 - node));
    }
    float o[L::NT][4];
#pragma unroll
    for (int i = 0; i < L::NT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

    // a group of rows that do not exist leaves the tensor cores to the others
    const bool idle = row0 + rw * 16 >= p.rows;

    // ---------------------------------------------------------------- tiles
    for (int tile = at.t0; tile < at.t1; ++tile, ++tile_no) {
      if (tile_no % L::NG != uint32_t(grp)) continue;
      const uint32_t ik = 2 * tile_no, iv = ik + 1;
      const uint32_t sk = ik % NS, sv = iv % NS;
      wait_phase(full0 + 8 * sk, (ik / NS) & 1, failed, p.error);
      if (RW > 1 && idle) {
        wait_phase(full0 + 8 * sv, (iv / NS) & 1, failed, p.error);
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(empty0 + 8 * sk);
          mbar_arrive(empty0 + 8 * sv);
        }
        continue;
      }
      const uint32_t ok_bits = page_ok[tile_no % 16];
#pragma unroll
      for (int j = 0; j < L::kSub; ++j) {
        const int key0 = (j * L::KT + kt) * L::SK;       // within the tile
        const uint32_t kb = ring0 + sk * L::kSlot;
        constexpr int SN = L::SK / 8;
        // 16 keys: a second set of accumulators, for twice the chains
        constexpr int kSets = L::SK == 16 ? 2 : 1;
        float sc[kSets][SN][4] = {};
        uint32_t pf[L::SK / 16][4];
#pragma unroll
        for (int ks = 0; ks < DC * 4; ++ks) {
          uint32_t a[4];
          if constexpr (L::kQReg) {
#pragma unroll
            for (int e = 0; e < 4; ++e) a[e] = qf[ks][e];
          } else {
            load_q(a, ks);
          }
          auto &acc = sc[ks % kSets];
          if constexpr (kType == kE4M3) {
            // 16 codes of a key are one 16-byte chunk: matrices (keys 0-7),
            // (keys 8-15) of steps ks and ks + 1 come together
            if ((ks & 1) == 0) {
              uint32_t a2[4];
              if constexpr (L::kQReg) {
#pragma unroll
                for (int e = 0; e < 4; ++e) a2[e] = qf[ks + 1][e];
              } else {
                load_q(a2, ks + 1);
              }
#pragma unroll
              for (int h = 0; h < L::SK / 16; ++h) {
                uint32_t b[4];
                const uint32_t key = key0 + h * 16 + (lane & 15);
                ldsm4(b, kb + spot<L>(key, ks, lane >> 4));
                uint32_t k0[4], k1[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) e4m3_f16(b[e], k0[e], k1[e]);
                mma<kType>(sc[0][2 * h], a, k0[0], k1[0]);
                mma<kType>(sc[0][2 * h + 1], a, k0[1], k1[1]);
                mma<kType>(sc[kSets - 1][2 * h], a2, k0[2], k1[2]);
                mma<kType>(sc[kSets - 1][2 * h + 1], a2, k0[3], k1[3]);
              }
            }
          } else {
#pragma unroll
            for (int h = 0; h < L::SK / 16; ++h) {
              uint32_t b[4];
              const uint32_t key = key0 + h * 16 + (lane & 7) + ((lane >> 4) << 3);
              ldsm4(b, kb + spot<L>(key, 2 * ks, (lane >> 3) & 1));
              mma<kType>(acc[2 * h], a, b[0], b[1]);
              mma<kType>(acc[2 * h + 1], a, b[2], b[3]);
            }
          }
        }
        // scores in base 2; masks where a key is not everybody's
        const int s0 = tile * kTile + key0;
        constexpr uint32_t kAll = (1u << (L::SK / 16)) - 1;
        const uint32_t there = ok_bits >> (key0 / 16);
        const bool open = (there & kAll) == kAll && s0 + L::SK <= at.len;
        float x[SN][4];
#pragma unroll
        for (int nt = 0; nt < SN; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            x[nt][e] = (kSets == 2 ? sc[0][nt][e] + sc[kSets - 1][nt][e] : sc[0][nt][e]) * cr[e >> 1];
        // bit k of sees[r]: row r attends to key s0 + k
        uint32_t sees[2] = {~0u, ~0u};
        if (!open) {
          const int rel = s0 - at.len;                   // of the first key to the drafted ones
          uint32_t exist = 0;
#pragma unroll
          for (int h = 0; h < L::SK / 16; ++h) exist |= (there >> h & 1) ? 0xFFFFu << (16 * h) : 0u;
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            uint32_t w = rel <= -32 ? ~0u
                       : rel < 0   ? (uint32_t(word[r]) << -rel) | ((1u << -rel) - 1)
                       : rel < 64  ? uint32_t(word[r] >> rel) : 0u;
            sees[r] = w & exist;
          }
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const uint32_t w = sees[r] >> (2 * t);
#pragma unroll
            for (int nt = 0; nt < SN; ++nt)
#pragma unroll
              for (int e = 0; e < 2; ++e)
                if (!(w >> (8 * nt + e) & 1)) x[nt][2 * r + e] = -INFINITY;
          }
        }
        float m2[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          float top = fmaxf(x[0][2 * r], x[0][2 * r + 1]);
#pragma unroll
          for (int nt = 1; nt < SN; ++nt) top = fmaxf(top, fmaxf(x[nt][2 * r], x[nt][2 * r + 1]));
          top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
          top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
          m2[r] = fmaxf(m[r], top);
        }
        // rescale where a row's maximum has moved, which is rare after the first tiles
        if (__any_sync(~0u, m2[0] > m[0] || m2[1] > m[1])) {
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float keep = m[r] == -INFINITY ? 0.f : ex2(m[r] - m2[r]);
            l[r] *= keep;
#pragma unroll
            for (int i = 0; i < L::NT; ++i) {
              o[i][2 * r] *= keep;
              o[i][2 * r + 1] *= keep;
            }
            m[r] = m2[r];
          }
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          // the weights meet v in the products' 16 bits, l sums them as they are:
          // a rounding of each by 2^-8 of it at most in BF16, 2^-11 in FP16, for
          // one product where FP32's bits would take three
          const float base = m[r] == -INFINITY ? 0.f : m[r] - kLift<kType>;
#pragma unroll
          for (int nt = 0; nt < SN; ++nt) {
            const float a0 = ex2(x[nt][2 * r] - base), a1 = ex2(x[nt][2 * r + 1] - base);
            l[r] += a0 + a1;
            pf[nt / 2][r + 2 * (nt & 1)] = pack2<kType>(a0, a1);
          }
        }
        if (j == L::kSub - 1) {
          __syncwarp();
          if (lane == 0) mbar_arrive(empty0 + 8 * sk);
        }

        // ----------------------------------------------------------- p . v
        if (j == 0) wait_phase(full0 + 8 * sv, (iv / NS) & 1, failed, p.error);
        const uint32_t vb = ring0 + sv * L::kSlot;
        // Keys that some row does not attend to: a weight of 0 does not keep an
        // infinity or NaN of v out of the product, so v is looked through first
        bool plain = true;
        if (!open) {
          uint32_t odd = 0;
#pragma unroll
          for (int h = 0; h < L::SK / 16; ++h)
#pragma unroll
            for (int c = 0; c < L::kChunks * (L::kRow / 16); c += 2) {
              uint32_t b[4];
              ldsm4(b, vb + spot<L>(key0 + h * 16 + (lane & 15), c, lane >> 4));
#pragma unroll
              for (int e = 0; e < 4; ++e) odd |= nonfinite_bits<kType>(b[e]);
            }
          plain = !__any_sync(~0u, odd != 0);
        }
        if (plain) {
#pragma unroll
          for (int h = 0; h < L::SK / 16; ++h) {
            const uint32_t key = key0 + h * 16 + (lane & 15);
#pragma unroll
            for (int i = 0; i < L::NT / 2; ++i) {
              uint32_t b[4];
              if constexpr (kType == kE4M3) {
                // 16 columns: matrices (keys 0-7), (keys 8-15) of two blocks of 16
                if ((i & 1) == 0) {
                  ldsm4t(b, vb + spot<L>(key, i, lane >> 4));
#pragma unroll
                  for (int k = 0; k < 2; ++k) {
                    uint32_t v0[2], v1[2];
                    e4m3_f16(prmt(b[2 * k], 0, 0x3120), v0[0], v1[0]);
                    e4m3_f16(prmt(b[2 * k + 1], 0, 0x3120), v0[1], v1[1]);
                    mma<kType>(o[2 * (i + k)], pf[h], v0[0], v0[1]);
                    mma<kType>(o[2 * (i + k) + 1], pf[h], v1[0], v1[1]);
                  }
                }
              } else {
                ldsm4t(b, vb + spot<L>(key, 2 * i, lane >> 4));
                mma<kType>(o[2 * i], pf[h], b[0], b[1]);
                mma<kType>(o[2 * i + 1], pf[h], b[2], b[3]);
              }
            }
          }
        } else {
          // ... and what is not finite is left out of the product and added to
          // the rows that do attend to it
#pragma unroll 1
          for (int h = 0; h < L::SK / 16; ++h) {
            uint32_t pp[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) pp[e] = h == 0 ? pf[0][e] : pf[L::SK / 16 - 1][e];
            const uint32_t key = key0 + h * 16 + (lane & 15);
#pragma unroll
            for (int i = 0; i < L::NT / 2; ++i) {
              uint32_t b[4];
              if constexpr (kType == kE4M3) {
                ldsm4t(b, vb + spot<L>(key, i));
                e4m3_f16(prmt(b[0], 0, 0x3120), b[0], b[2]);
                e4m3_f16(prmt(b[1], 0, 0x3120), b[1], b[3]);
              } else {
                ldsm4t(b, vb + spot<L>(key, 2 * i, lane >> 4));
              }
#pragma unroll
              for (int e = 0; e < 4; ++e) b[e] &= finite_mask<kType>(b[e]);
              mma<kType>(o[2 * i], pp, b[0], b[1]);
              mma<kType>(o[2 * i + 1], pp, b[2], b[3]);
            }
          }
#pragma unroll 1
          for (int k = 0; k < L::SK; ++k) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              if (!(sees[r] >> k & 1)) continue;
#pragma unroll
              for (int i = 0; i < L::NT; ++i)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const int col = out_col<kType>(i, t, e);
                  const uint8_t *at16 = ring + sv * L::kSlot + spot<L>(key0 + k, col * L::kSize / 16);
                  float v;
                  if constexpr (kType == kE4M3) {
                    uint32_t lo, hi;
                    e4m3_f16(at16[col % 16], lo, hi);
                    v = __half2float(__ushort_as_half(uint16_t(lo)));
                  } else {
                    const uint16_t c = *reinterpret_cast<const uint16_t *>(at16 + (col % 8) * 2);
                    v = kType == kBf16 ? __bfloat162float(__ushort_as_bfloat16(c))
                                       : __half2float(__ushort_as_half(c));
                  }
                  if (!(fabsf(v) < INFINITY)) o[i][2 * r + e] += v;
                }
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty0 + 8 * sv);
    }

    // After a wait that ran out, in this call or in one before whose error nobody
    // has read, the sums are NaN, and with them what is made of them: the block
    // that joins other blocks' results, too, must not give out numbers.
    if (*failed | *stale) l[0] = l[1] = __int_as_float(0x7FFFFFFF);

    // What a row's result is, from `res` (tile_of(i): which tile of its columns
    // res[i] is) with maximum mm and sum ll.
    auto emit = [&](auto &res, const float (&mm)[2], const float (&ll)[2], bool first_warp, auto &&tile_of) {
      constexpr int N = sizeof(res) / sizeof(res[0]);
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int row = row0 + rw * 16 + g + 8 * r, node = node_of(p, row);
        if (row >= p.rows) continue;
        const int h = head * p.group + row - node * p.group;
        // NaN is not nothing
        const bool empty = node >= at.count || (mm[r] == -INFINITY && ll[r] == 0.f);
        const float inv = empty ? 0.f : p.v_scale / ll[r];
        const int64_t at_row = (int64_t(at.b) * p.n + node) * p.hq + h;
        uint16_t *out = static_cast<uint16_t *>(p.out) + at_row * p.d;
        const bool f16 = kType == kF16 || (kType == kE4M3 && p.q_f16);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const int nt = tile_of(i);
          const float v0 = empty ? 0.f : res[i][2 * r] * inv, v1 = empty ? 0.f : res[i][2 * r + 1] * inv;
          if constexpr (kType == kE4M3) {
            // columns 4t + 2e of even tiles, 4t + 2e + 1 of odd ones: an even
            // tile's lane stores for both where it has both
            if constexpr (N >= 2) {
              if (i % 2 == 0 && 8 * nt < p.d) {
                const float u0 = empty ? 0.f : res[i + 1][2 * r] * inv;
                const float u1 = empty ? 0.f : res[i + 1][2 * r + 1] * inv;
                *reinterpret_cast<uint2 *>(out + 8 * nt + 4 * t) =
                    make_uint2(pack_out(v0, u0, f16), pack_out(v1, u1, f16));
              }
            } else if (8 * (nt & ~1) < p.d) {
              const uint32_t both = pack_out(v0, v1, f16);
              out[out_col<kType>(nt, t, 0)] = uint16_t(both);
              out[out_col<kType>(nt, t, 1)] = uint16_t(both >> 16);
            }
          } else if (8 * nt < p.d) {
            *reinterpret_cast<uint32_t *>(out + 8 * nt + 2 * t) = pack_out(v0, v1, f16);
          }
        }
        if (p.lse && t == 0 && first_warp)
          p.lse[at_row] = empty ? -INFINITY : (mm[r] - kLift<kType> + log2f(ll[r])) * kLn2;
      }
    };
    if constexpr (kSolo) {
      if (alone) {
        // the KT warps join shares of the columns among themselves
        constexpr int TS = L::NT / L::KT;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          l[r] += __shfl_xor_sync(~0u, l[r], 1);
          l[r] += __shfl_xor_sync(~0u, l[r], 2);
        }
        named_bar(pair, L::KT * 32);                     // q has been read
        const int warp0 = rw * L::KW + grp * L::KT;
        float4 *box = reinterpret_cast<float4 *>(scratch) + warp0 * (L::NT * 32) + lane;
#pragma unroll
        for (int i = 0; i < L::NT; ++i)
          box[(kt * L::NT + i) * 32] = make_float4(o[i][0], o[i][1], o[i][2], o[i][3]);
        if (t == 0) {
          state[warp * 16 + g] = make_float2(m[0], l[0]);
          state[warp * 16 + g + 8] = make_float2(m[1], l[1]);
        }
        named_bar(pair, L::KT * 32);
        float res[TS][4], mj[2] = {-INFINITY, -INFINITY}, lj[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < TS; ++i) res[i][0] = res[i][1] = res[i][2] = res[i][3] = 0.f;
#pragma unroll
        for (int k = 0; k < L::KT; ++k) {
          const float2 st[2] = {state[(warp0 + k) * 16 + g], state[(warp0 + k) * 16 + g + 8]};
          merge<TS>(res, mj, lj, st, [&](int i) { return box[(k * L::NT + kt * TS + i) * 32]; });
        }
        emit(res, mj, lj, kt == 0, [&](int i) { return kt * TS + i; });
        named_bar(pair, L::KT * 32);                     // scratch is free again
        at = after;
        continue;
      }
    }
    if constexpr (kAheadQ) {
      fetched = after.valid() && !solo(after);
      if (fetched) fetch_q(after);
    }

    // ------------------------------------- join the key warps, then the blocks
    const bool whole = at.whole();
    const int first = whole ? 0 : at.first(), final = whole ? 0 : at.final();
    // a block's partial result: its unit's first block has it in its second place
    auto place = [&](int block) {
      return p.partial + (int64_t(block) * 2 + (block == first ? 1 : 0)) * L::kPartial;
    };
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      l[r] += __shfl_xor_sync(~0u, l[r], 1);
      l[r] += __shfl_xor_sync(~0u, l[r], 2);
    }
    // Every warp lays its result open in shared memory, and each then joins
    // a share of the columns of its row group: TPW output tiles, all key warps'.
    constexpr int TPW = L::TPW, NT = L::NT;
    float res[TPW][4], mj[2] = {m[0], m[1]}, lj[2] = {l[0], l[1]};
    if constexpr (L::KW == 1) {
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) res[i][e] = o[i][e];
    } else {
      float4 *box = reinterpret_cast<float4 *>(scratch);
      constexpr int NP = NT / L::kPasses;                // tiles of a pass
      if (t == 0) {
        state[warp * 16 + g] = make_float2(m[0], l[0]);
        state[warp * 16 + g + 8] = make_float2(m[1], l[1]);
      }
      float w[L::KW][2];
#pragma unroll
      for (int pass = 0; pass < L::kPasses; ++pass) {
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          const auto &x = o[pass * NP + i];
          box[(warp * NP + i) * 32 + lane] = make_float4(x[0], x[1], x[2], x[3]);
        }
        named_bar(1, kConsumers * 32);
        if (pass == 0) {
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            float2 st[L::KW];
            float top = -INFINITY, sum = 0.f;
#pragma unroll
            for (int k = 0; k < L::KW; ++k) {
              st[k] = state[(rw * L::KW + k) * 16 + g + 8 * r];
              top = fmaxf(top, st[k].x);
            }
#pragma unroll
            for (int k = 0; k < L::KW; ++k) {
              w[k][r] = st[k].x == -INFINITY ? 0.f : ex2(st[k].x - top);
              sum += st[k].y * w[k][r];
            }
            mj[r] = top;
            lj[r] = sum;
          }
        }
        constexpr int TP = TPW / L::kPasses;             // this warp's tiles of a pass
#pragma unroll
        for (int i = 0; i < TP; ++i) {
          float (&y)[4] = res[pass * TP + i];
          y[0] = y[1] = y[2] = y[3] = 0.f;
#pragma unroll
          for (int k = 0; k < L::KW; ++k) {
            const float4 v = box[((rw * L::KW + k) * NP + kg * TP + i) * 32 + lane];
            y[0] += v.x * w[k][0];
            y[1] += v.y * w[k][0];
            y[2] += v.z * w[k][1];
            y[3] += v.w * w[k][1];
          }
        }
        if (pass + 1 < L::kPasses) named_bar(1, kConsumers * 32);
      }
    }
    // tile of the head's columns that res[i] is
    auto tile_of = [&](int i) {
      constexpr int TP = TPW / L::kPasses;
      return (i / TP) * (NT / L::kPasses) + kg * TP + i % TP;
    };
    bool done = whole;
    if (!whole) {
      Join join(first, final, blockIdx.x, kJoinAtOnce<L>);
      float *to = place(blockIdx.x);
#pragma unroll 1
      while (true) {
        float4 *cols = reinterpret_cast<float4 *>(to) + rw * (NT * 32) + lane;
#pragma unroll
        for (int i = 0; i < TPW; ++i)
          cols[tile_of(i) * 32] = make_float4(res[i][0], res[i][1], res[i][2], res[i][3]);
        if (kg == 0 && t == 0) {
          float2 *st = reinterpret_cast<float2 *>(to + RW * NT * 32 * 4) + rw * 16;
          st[g] = make_float2(mj[0], lj[0]);
          st[g + 8] = make_float2(mj[1], lj[1]);
        }
        __threadfence();
        named_bar(1, kConsumers * 32);
        if (tid == 0) {
          uint32_t *counter = join.counter(p);
          *last = atomicAdd(counter, 1u) + 1 == join.members();
          if (*last) *counter = 0;
          __threadfence();
        }
        named_bar(1, kConsumers * 32);
        if (!*last) break;
#pragma unroll
        for (int i = 0; i < TPW; ++i) res[i][0] = res[i][1] = res[i][2] = res[i][3] = 0.f;
        mj[0] = mj[1] = -INFINITY;
        lj[0] = lj[1] = 0.f;
        constexpr int kAhead = TPW <= 2 ? 8 : TPW <= 4 ? 4 : 2;   // blocks fetched at a time
#pragma unroll 1
        for (int blk = join.lo; blk <= join.hi; blk += kAhead * join.step) {
          float4 v[kAhead][TPW];
          float2 st[kAhead][2];
#pragma unroll
          for (int k = 0; k < kAhead; ++k) {
            const int from_block = blk + k * join.step;
            const float *part = place(from_block <= join.hi ? from_block : blk);
            const float2 *sp = reinterpret_cast<const float2 *>(part + RW * NT * 32 * 4) + rw * 16;
            st[k][0] = __ldcg(sp + g);
            st[k][1] = __ldcg(sp + g + 8);
            const float4 *from = reinterpret_cast<const float4 *>(part) + rw * (NT * 32) + lane;
#pragma unroll
            for (int i = 0; i < TPW; ++i) v[k][i] = __ldcg(from + tile_of(i) * 32);
          }
#pragma unroll
          for (int k = 0; k < kAhead; ++k) {
            if (blk + k * join.step > join.hi) break;
            merge<TPW>(res, mj, lj, st[k], [&](int i) { return v[k][i]; });
          }
        }
        done = join.last();
        if (done) break;
        named_bar(1, kConsumers * 32);                   // everybody has read the group's
        to = place(join.lo);
        join.next();
      }
    }

    // -------------------------------------------------------------- results
    if (done) emit(res, mj, lj, kg == 0, tile_of);
    named_bar(1, kConsumers * 32);                       // scratch, q and *last are free again
    at = after;
  }
}

// -------------------------------------------------------------------- host
using Kernel = void (*)(AttnParams, CUtensorMap, CUtensorMap);

struct Variant {
  Kernel fn;
  int smem, rows, partial, threads;
  std::atomic<uint64_t> *allowed;   // bit d: device d lets fn have its shared memory
};

template <int kType, int DC, int RW>
Variant variant() {
  using L = Cfg<kType, DC, RW>;
  static std::atomic<uint64_t> allowed{0};
  return {reinterpret_cast<Kernel>(&attention_kernel<kType, DC, RW>), L::kSmem, L::kRows, L::kPartial,
          kAttnThreads, &allowed};
}

// The variants of one cache type, by head_dim up to 64, 128, 192, 256 and by
// row groups 1, 2, 4, 8: a translation unit each.
using Variants = Variant[4][4];
extern const Variants kVariantsBf16, kVariantsF16, kVariantsE4M3;

// The tcgen05 kernel (vg_attention_wide.cuh): by cache type, head_dim up to 64
// and 128, one and two row tiles of 128.
using WideVariants = Variant[3][2][2];
extern const WideVariants kWide;

// (Heads up to 128 go to the tcgen05 kernel above 32 rows.  Up to 32 the bytes
// and not the products bound heads of 192, and those of 256 serve.)
#define VG_ATTENTION_VARIANTS(T)                      \
  {{variant<T, 1, 1>(), variant<T, 1, 2>()},           \
   {variant<T, 2, 1>(), variant<T, 2, 2>()},           \
   {{}, {}, variant<T, 3, 4>(), variant<T, 3, 8>()},  \
   {variant<T, 4, 1>(), variant<T, 4, 2>(), variant<T, 4, 4>(), variant<T, 4, 8>()}}

}  // namespace attn
}  // namespace vg
