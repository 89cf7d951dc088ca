// vg_attention_wide.cuh -- the attention kernel for many rows a cache head:
// tcgen05 products with the scores, the weights and the output in TMEM.
//
// From some 32 rows a head on, mma.sync (0.5 PFLOP/s here) and not the cache's
// bytes bounds the kernel of vg_attention.cuh.  Here the products of 128 rows
// with 128 keys are
//     S = Q K^T        both operands in shared memory
//     P = 2^(c S - m)  one thread a row: TMEM -> registers -> TMEM, 16 bits
//     O = O + P V      P from TMEM, V in shared memory as it lies (its rows
//                      are the products' k, so it is the transposed operand)
// One warp issues the products, a warp each copies K and V, and two
// warpgroups do the softmax of two streams that take the tensor cores in
// turn: the products of one run under the softmax of the other.  With more
// than 128 rows the streams are two row tiles of the same keys; with fewer
// they are the even and the odd tiles of keys, joined at a unit's end (both
// outputs lie in the lanes of their row, so a thread reads both).
// TMEM holds S and O of both streams, 4 x 128 columns; P takes the place of S.
// 128 keys and not 64: an M = 128 product takes 64 clocks at N = 64 and at
// N = 128 alike (measured; 128 at N = 256).
// A row's maximum may lag by up to 2^8: O is rescaled, in TMEM by its softmax
// warpgroup, only when the true maximum is more than 8 above the one in use,
// and l carries the same factor.
// Codes of an E4M3 cache are copied as they are and turned into FP16 by a
// fourth warpgroup, tile by tile, into the slots that the products read; q is
// brought to FP16 by a power of two for each row, which goes into its c.
// The cutting of the line, the pages and the joining of blocks are those of
// vg_attention.cuh.
//
// Measured (heads of 128, a kernel by itself):
//     8 sequences of 8190 keys, 64 nodes, 8 query heads a cache head, BF16
//         512 rows: 124 us, 1.12 PFLOP/s.  Within a unit the tensor cores are
//         busy two thirds of the time (a stream's step takes 3094 clocks, the
//         two streams' products 2048); 9 us pass before the first scores and
//         12 in writing and joining the results of units that are cut
//     48 sequences of 1200 to 6007 keys, 16 nodes, 4 query heads a cache head
//         64 rows: 734 MB of FP16 in 133 us, 5.5 TB/s
//     the same over an E4M3 cache, half the bytes: 143 us, bound by the
//         warps that convert codes (two codes an instruction)
// The kernel of vg_attention.cuh took 458 us and 184 us for the first two, and
// 222 us for the third.
#pragma once

#include "vg_attention.cuh"

namespace vg {
namespace attn {

// Threads: two softmax warpgroups, one that copies and issues, and for E4M3
// one that converts.  Registers a thread: 168 at a launch of 384 (64512 in
// all), then 256 x 216 + 128 x 72 = 64512: a softmax thread holds a row of 128
// scores; 128 at a launch of 512 (65536), then 256 x 184 + 128 x 64 + 128 x 80
// = 65536, and the scores are read from TMEM twice instead.
template <bool kF8>
struct WideThreads {
  static constexpr int kThreads = kF8 ? 512 : 384;
  static constexpr int kSoftmax = kF8 ? 184 : 216, kOther = kF8 ? 64 : 72, kConvert = 80;
};
constexpr float kLag = 8.f;                   // log2 of what a maximum may lag
// FP16 weights are at most 2^kLag times 2^lift: lifted to 2^15 in all.  Where the
// maximum does not lag, weights below 2^-21 of the largest lose bits (in the other
// kernel below 2^-29), 2^-32 of the largest at most each.  As there, the weights
// meet v in the products' 16 bits, and l sums them as they are.
template <int kType>
constexpr float kWideLift = kType == kBf16 ? 0.f : 7.f;

template <int kCache, int DC, int NQ>
struct WideCfg {
  static constexpr bool kF8 = kCache == kE4M3;
  static constexpr int kType = kF8 ? kF16 : kCache;      // of the products
  static constexpr int D = DC * 64;
  static constexpr int kRow = 128, kElems = 64, kChunks = DC, kKeys = 128;
  static constexpr int kChunk = kKeys * kRow;            // 16 KB
  static constexpr int kSlot = DC * kChunk;
  // an E4M3 tile as it is copied
  struct Stage {
    static constexpr int kRow = DC == 1 ? 64 : 128, kElems = kRow, kChunks = 1, kKeys = 128;
    static constexpr int kChunk = kKeys * kRow, kSlot = kChunk;
  };
  static constexpr int kQChunk = 128 * 128;              // 128 rows of 64 elements
  static constexpr int kQTile = DC * kQChunk;
  static constexpr int kRows = 128 * NQ;
  static constexpr int kFixed = 3 * 1024;
  static constexpr int kRoom = 227 * 1024 - kFixed - NQ * kQTile;
  static constexpr int kFit = kRoom / kSlot;
  static constexpr int kSlots = kF8 ? 4 : (kFit > 16 ? 16 : kFit) & ~1;
  static constexpr int kStageFit = (kRoom - kSlots * kSlot) / Stage::kSlot;
  static constexpr int kStages = kF8 ? (kStageFit > 8 ? 8 : kStageFit) & ~1 : 0;
  static constexpr int kSmem = kFixed + NQ * kQTile + kSlots * kSlot + kStages * Stage::kSlot;
  static_assert(!kF8 || kStages >= 2, "room for codes of K and of V");
  static constexpr int kPartial = kRows * (D + 2);       // floats of a partial result
  static constexpr uint32_t kO = 0, kS = 256;            // TMEM columns
};

// ------------------------------------------------------------- tcgen05 pieces
// True in one lane of the warp, the same each time.  Products are issued in a
// branch on this: under it the compiler keeps what they take in uniform
// registers and a product takes some 15 clocks to issue; under a branch on
// the lane's number it took 60, as long as the product itself.
__device__ __forceinline__ bool elect_one() {
  uint32_t y;
  asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(y));
  return y != 0;
}
__device__ __forceinline__ void tc_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
               : "memory");
}
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// D (TMEM) = A B (+ D): A and B in shared memory.
__device__ __forceinline__ void tc_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{ .reg .pred p; setp.ne.u32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(uint32_t(add))
      : "memory");
}
// A in TMEM.
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{ .reg .pred p; setp.ne.u32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p; }" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(uint32_t(add))
      : "memory");
}
// Shared-memory operand: 128-byte swizzle; `lead` and `stride` in bytes.
__device__ __forceinline__ uint64_t tc_desc(uint32_t addr, uint32_t lead, uint32_t stride) {
  return uint64_t((addr >> 4) & 0x3FFF) | uint64_t(lead >> 4) << 16 | uint64_t(stride >> 4) << 32 |
         uint64_t(1) << 46 | uint64_t(2) << 61;
}

// 32 columns of this thread's TMEM lane.
__device__ __forceinline__ void tc_ld32(uint32_t (&r)[32], uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tc_st32(uint32_t addr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
      "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]),
      "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
// (A load's registers must not be read before this: they are tied to it.)
__device__ __forceinline__ void tc_wait_ld(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),
                 "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]),
                 "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]),
                 "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]),
                 "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29])
               :
               : "memory");
  asm volatile("" : "+r"(r[30]), "+r"(r[31])::"memory");
}
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// (a0 c + b, a1 c + b), as one instruction.
__device__ __forceinline__ void fma2(float &y0, float &y1, uint32_t a0, uint32_t a1, float c, float b) {
  asm("{ .reg .b64 a, c, b, y; mov.b64 a, {%2, %3}; mov.b64 c, {%4, %4}; mov.b64 b, {%5, %5};\n"
      "fma.rn.f32x2 y, a, c, b; mov.b64 {%0, %1}, y; }"
      : "=f"(y0), "=f"(y1)
      : "r"(a0), "r"(a1), "f"(c), "f"(b));
}
__device__ __forceinline__ void add2(float &s0, float &s1, float a0, float a1) {
  asm("{ .reg .b64 s, a; mov.b64 s, {%0, %1}; mov.b64 a, {%2, %3};\n"
      "add.rn.f32x2 s, s, a; mov.b64 {%0, %1}, s; }"
      : "+f"(s0), "+f"(s1)
      : "f"(a0), "f"(a1));
}

template <int kCache, int DC, int NQ>
__global__ void __launch_bounds__(WideThreads<kCache == kE4M3>::kThreads, 1)
    wide_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ CUtensorMap kmap,
                const __grid_constant__ CUtensorMap vmap) {
  using L = WideCfg<kCache, DC, NQ>;
  using W = WideThreads<L::kF8>;
  constexpr int kType = L::kType;
  extern __shared__ __align__(1024) uint8_t wide_smem[];
  if (smem_addr(wide_smem) & 1023) {                     // the swizzles need it
    if (threadIdx.x == 0) atomicCAS(p.error, 0, kErrAttnWait);
    return;
  }
  uint8_t *ring = wide_smem;
  uint8_t *q_smem = ring + L::kSlots * L::kSlot;
  uint8_t *stage = q_smem + NQ * L::kQTile;
  uint8_t *fixed = stage + L::kStages * L::Stage::kSlot;
  uint64_t *bars = reinterpret_cast<uint64_t *>(fixed);
  // barriers: slots full, slots free; of each stream: scores there, weights there
  // (halves), product done; q there; everything done
  const uint32_t full0 = smem_addr(bars), empty0 = smem_addr(bars + 16), s_full = smem_addr(bars + 32),
                 p_full = smem_addr(bars + 34), o_full = smem_addr(bars + 38), q_full = smem_addr(bars + 40),
                 finished = smem_addr(bars + 41), stage_full = smem_addr(bars + 42),
                 stage_empty = smem_addr(bars + 50);
  uint32_t *page_ok = reinterpret_cast<uint32_t *>(fixed + 512);        // [16]
  volatile int *failed = reinterpret_cast<volatile int *>(fixed + 576);
  int *last = reinterpret_cast<int *>(fixed + 580);
  uint32_t *tmem_at = reinterpret_cast<uint32_t *>(fixed + 584);
  volatile int *keep_o = reinterpret_cast<volatile int *>(fixed + 588); // [stream]
  volatile int *stale = reinterpret_cast<volatile int *>(fixed + 596);
  uint32_t *odd_at = reinterpret_cast<uint32_t *>(fixed + 608);         // [2][4]: bits of keys
  int8_t *q_exp = reinterpret_cast<int8_t *>(fixed + 640);              // E4M3: [unit % 2][row]
  float2 *state = reinterpret_cast<float2 *>(fixed + 1024);             // keys split: [stream][row]: (m, l)
  constexpr int NS = L::kSlots;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  if (tid == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(&kmap) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&vmap) : "memory");
    *failed = *stale = 0;
    for (int i = 0; i < 8; ++i) odd_at[i] = 0;
    for (int s = 0; s < NS; ++s) {
      mbar_init(full0 + 8 * s, L::kF8 ? 128 : 1);
      mbar_init(empty0 + 8 * s, 1);
    }
    for (int s = 0; s < L::kStages; ++s) {
      mbar_init(stage_full + 8 * s, 1);
      mbar_init(stage_empty + 8 * s, 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(s_full + 8 * i, 1);
      mbar_init(p_full + 16 * i, 128);
      mbar_init(p_full + 16 * i + 8, 128);
      mbar_init(o_full + 8 * i, 1);
    }
    mbar_init(q_full, 256);
    mbar_init(finished, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     smem_addr(tmem_at))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    tc_before();
  }
  __syncthreads();
  tc_after();
  const uint32_t tmem = *tmem_at;
  Line at;
  at.init(p, p.hkv * p.blocks);

  if (L::kF8 && warp >= 12) {
    // -------------------------------------------------------- conversions
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(W::kConvert));
    if constexpr (L::kF8) {
      using G = typename L::Stage;
      constexpr int kPieces = G::kRow / 16;              // 16 codes each
      const int me = tid - 384;
      uint32_t i = 0;                                    // K and V tiles so far
      for (; at.valid(); at.next(p)) {
        for (uint32_t n = 2 * uint32_t(at.t1 - at.t0); n; --n, ++i) {
          const uint32_t from = i % L::kStages, to = i % NS;
          wait_phase(stage_full + 8 * from, (i / L::kStages) & 1, failed, p.error);
          wait_phase(empty0 + 8 * to, (i / NS & 1) ^ 1, failed, p.error);
          const uint8_t *src = stage + from * G::kSlot;
          uint8_t *dst = ring + to * L::kSlot;
          // Eight lanes take four pieces of two keys whose numbers differ in bits
          // 0 and 2: then neither the loads nor the stores, of pieces 2c and
          // 2c + 1 of one 128-byte chunk, meet in a bank.
#pragma unroll 4
          for (int k = 0; k < G::kKeys * kPieces / 128; ++k) {
            const int set = k * 4 + me / 32;             // 8 keys, 4 pieces
            const int key = set / (kPieces / 4) * 8 + (lane / 8 ^ (lane & 4 ? 5 : 0));
            const int c = set % (kPieces / 4) * 4 + lane % 4;
            const uint4 v = *reinterpret_cast<const uint4 *>(src + spot<G>(key, c));
            uint4 a, b;
            e4m3_f16(v.x, a.x, a.y);
            e4m3_f16(v.y, a.z, a.w);
            e4m3_f16(v.z, b.x, b.y);
            e4m3_f16(v.w, b.z, b.w);
            *reinterpret_cast<uint4 *>(dst + spot<L>(key, 2 * c)) = a;
            *reinterpret_cast<uint4 *>(dst + spot<L>(key, 2 * c + 1)) = b;
          }
          fence_proxy_async();
          mbar_arrive(full0 + 8 * to);
          __syncwarp();
          if (lane == 0) mbar_arrive(stage_empty + 8 * from);
        }
      }
    }
  } else if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(W::kOther));
    if (warp == 8 || warp == 10) {
    // ------------------------------------------------------------- copies
    const int kv = warp == 10;
    if constexpr (L::kF8)
      copy_tiles<typename L::Stage, L::kStages>(p, at, kv ? &vmap : &kmap, kv, smem_addr(stage), stage_full,
                                                stage_empty, page_ok, failed, stale);
    else
      copy_tiles<L, NS>(p, at, kv ? &vmap : &kmap, kv, smem_addr(ring), full0, empty0, page_ok, failed, stale);
    } else if (warp == 9) {
    // ----------------------------------------------------------- products
    // Step w of a unit is stream w % 2's: tile w / 2 or, with the keys split, w.
    constexpr uint32_t kFmt = kType == kBf16 ? 1 : 0;
    constexpr uint32_t kIdesc = 1u << 4 | kFmt << 7 | kFmt << 10 | (128u / 16) << 24;
    constexpr uint32_t kQk = kIdesc | uint32_t(L::kKeys / 8) << 17;
    constexpr uint32_t kPv = kIdesc | 1u << 16 | uint32_t(L::D / 8) << 17;   // V: n runs along its rows
    const uint32_t tm = __shfl_sync(~0u, tmem, 0);
    const uint64_t k_ring = tc_desc(smem_addr(ring), 16, 1024), q_desc = tc_desc(smem_addr(q_smem), 16, 1024);
    const uint64_t v_ring = tc_desc(smem_addr(ring), L::kChunk, 1024);
    uint32_t n = 0, q_par = 0, c0 = 0, c1 = 0;           // tiles, units; steps of the streams so far
    for (; at.valid(); at.next(p)) {
      wait_phase(q_full, q_par, failed, p.error);
      q_par ^= 1;
      tc_after();
      const uint32_t tiles = __shfl_sync(~0u, uint32_t(at.t1 - at.t0), 0);
      const uint32_t steps = NQ == 2 ? 2 * tiles : tiles;
      auto scores = [&](uint32_t w) {
        const uint32_t q = w & 1, i = n + (NQ == 2 ? w / 2 : w), s = 2 * i % NS;
        if (NQ == 1 || q == 0) {
          wait_phase(full0 + 8 * s, (2 * i / NS) & 1, failed, p.error);
          tc_after();
        }
        const uint64_t kd = k_ring + s * (L::kSlot / 16);
        const uint64_t qd = q_desc + (NQ == 2 ? q : 0) * (L::kQTile / 16);
        if (elect_one()) {
#pragma unroll
          for (int ks = 0; ks < DC * 4; ++ks)
            tc_mma_ss(tm + L::kS + q * 128, qd + ((ks / 4) * L::kQChunk + (ks % 4) * 32) / 16,
                      kd + ((ks / 4) * L::kChunk + (ks % 4) * 32) / 16, kQk, ks > 0);
          tc_commit(s_full + 8 * q);
          if (NQ == 1 || q == 1) tc_commit(empty0 + 8 * s);
        }
        __syncwarp();
      };
      scores(0);
      if (steps > 1) scores(1);
      for (uint32_t w = 0; w < steps; ++w) {
        const uint32_t q = w & 1, i = n + (NQ == 2 ? w / 2 : w), s = (2 * i + 1) % NS;
        if (NQ == 1 || q == 0) wait_phase(full0 + 8 * s, ((2 * i + 1) / NS) & 1, failed, p.error);
        const uint32_t c = q ? c1++ : c0++;
        const uint64_t vd = v_ring + s * (L::kSlot / 16);
        // the first half of the weights goes ahead of the second
        wait_phase(p_full + 16 * q, c & 1, failed, p.error);
        tc_after();
        const bool fresh = w < 2 && !keep_o[q];          // O begins with this product
        if (elect_one()) {
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)
            tc_mma_ts(tm + L::kO + q * 128, tm + L::kS + q * 128 + ks * 8, vd + ks * 2048 / 16, kPv,
                      !fresh || ks > 0);
        }
        __syncwarp();
        wait_phase(p_full + 16 * q + 8, c & 1, failed, p.error);
        tc_after();
        if (elect_one()) {
#pragma unroll
          for (int ks = 4; ks < 8; ++ks)
            tc_mma_ts(tm + L::kO + q * 128, tm + L::kS + q * 128 + ks * 8, vd + ks * 2048 / 16, kPv, true);
          if (w + 2 >= steps) tc_commit(o_full + 8 * q);       // the stream's last of the unit
          if (NQ == 1 || q == 1) tc_commit(empty0 + 8 * s);
        }
        __syncwarp();
        if (w + 2 < steps) scores(w + 2);
      }
      n += tiles;
    }
    // nothing is in flight when TMEM is given back
    if (elect_one()) tc_commit(finished);
    __syncwarp();
    const uint64_t limit = globaltimer() + 10000000;
    while (!mbar_try_wait(finished, 0) && globaltimer() < limit) {
    }
    __syncwarp();
    }
  } else {
    // ------------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(W::kSoftmax));
    const int q = warp / 4, row_in = tid % 128;          // stream, lane of TMEM
    const uint32_t lanes = tmem + (uint32_t(warp % 4 * 32) << 16);
    const uint32_t o_at = lanes + L::kO + q * 128, s_at = lanes + L::kS + q * 128;
    // c > 0: its sign goes into q, so that the largest product is the largest score
    float c = fmaxf(fabsf(p.c), 1e-30f);
    const uint32_t flip = p.c < 0.f ? 0x80008000u : 0u;
    uint32_t n = 0, steps = 0, units = 0;                // tiles, this stream's steps and units so far
    auto sync_rows = [&] { named_bar(1, 256); };
    // q to shared memory, sixteen lanes a row, by way of registers: the next
    // unit's q is fetched and stored, and its first scores made, while this
    // unit's output is still written
    constexpr int kQn = L::kRows / 16;
    uint4 qv[kQn];
    const int piece = lane % 16;
    auto row_of = [&](int k) {                           // with two row tiles, the stream's own
      return NQ == 2 ? q * 128 + k * 8 + warp % 4 * 2 + lane / 16 : k * 16 + warp * 2 + lane / 16;
    };
    auto fetch_q = [&](const Line &u) {
      const int head = head_of(p, u.u), row0 = block_of_rows(p, u.u) * L::kRows;
#pragma unroll
      for (int k = 0; k < kQn; ++k) {
        const int rw = row0 + row_of(k), node = node_of(p, rw);
        qv[k] = make_uint4(0, 0, 0, 0);
        if (rw < p.rows && piece * 8 < p.d)
          qv[k] = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.q) + u.b * p.qs[0] +
                                                   node * p.qs[1] +
                                                   (head * p.group + rw - node * p.group) * p.qs[2] + piece * 8);
      }
    };
    auto store_q = [&](int8_t *exps) {
#pragma unroll
      for (int k = 0; k < kQn; ++k) {
        const int r = row_of(k);
        if constexpr (L::kF8) {
          float f[8], top = 0.f;
          const uint32_t w[4] = {qv[k].x, qv[k].y, qv[k].z, qv[k].w};
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const uint16_t x = uint16_t(w[e / 2] >> (16 * (e & 1)));
            f[e] = p.q_f16 ? __half2float(__ushort_as_half(x)) : __bfloat162float(__ushort_as_bfloat16(x));
            top = fmaxf(top, fabsf(f[e]));
          }
#pragma unroll
          for (int m = 8; m; m /= 2) top = fmaxf(top, __shfl_xor_sync(~0u, top, m));
          const int e = q_exponent(top);
          const float down = ldexpf(1.f, -e);
          qv[k] = make_uint4(pack2<kF16>(f[0] * down, f[1] * down), pack2<kF16>(f[2] * down, f[3] * down),
                             pack2<kF16>(f[4] * down, f[5] * down), pack2<kF16>(f[6] * down, f[7] * down));
          if (piece == 0) exps[r] = int8_t(e);
        }
        if (piece < DC * 8)
          *reinterpret_cast<uint4 *>(q_smem + (r / 128) * L::kQTile + (piece / 8) * L::kQChunk +
                                     (r % 128) * 128 + (((piece % 8) ^ (r & 7)) << 4)) =
              make_uint4(qv[k].x ^ flip, qv[k].y ^ flip, qv[k].z ^ flip, qv[k].w ^ flip);
      }
      fence_proxy_async();
      mbar_arrive(q_full);
    };
    uint32_t other = 0;                                  // the other stream's steps so far
    uint32_t unit = 0;
    if (at.valid()) {
      fetch_q(at);
      store_q(q_exp);
      if (L::kF8) sync_rows();                           // everybody's exponents are there
    }
    for (; at.valid(); ++unit) {
      if constexpr (L::kF8)
        c = fmaxf(fabsf(p.c) * ldexpf(1.f, q_exp[unit % 2 * L::kRows + (NQ == 2 ? q * 128 : 0) + row_in]),
                  1e-30f);
      Line after = at;
      after.next(p);
      const int head = head_of(p, at.u), rb = block_of_rows(p, at.u);
      const int row0 = rb * L::kRows, row = row0 + (NQ == 2 ? q * 128 : 0) + row_in;
      const int node = node_of(p, row), h = head * p.group + row - node * p.group;
      const bool real = row < p.rows;
      uint64_t word = 0;
      if (real)
        word = (at.count >= 64 ? ~0ull : (1ull << at.count) - 1) &
               (p.tree ? p.tree[int64_t(at.b) * p.n + node] : ~0ull >> (63 - node));
      float m = -INFINITY, l = 0.f;                      // the maximum in use
      const int tiles = at.t1 - at.t0;

      for (int k0 = NQ == 2 ? 0 : q; k0 < tiles; k0 += NQ == 2 ? 1 : 2, ++steps) {
        const int tile = at.t0 + k0;
        const uint32_t i = n + k0, sv = (2 * i + 1) % NS;
        const bool begin = k0 < (NQ == 2 ? 1 : 2);       // O has nothing yet
        wait_phase(s_full + 8 * q, steps & 1, failed, p.error);
        tc_after();
        const uint32_t ok_bits = page_ok[i % 16];
        const int rel = tile * L::kKeys - at.len;        // of the first key to the drafted ones
        const bool open = ok_bits == 255u && rel <= -L::kKeys;
        uint64_t sees[2] = {~0ull, ~0ull};
        if (!open) {
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            uint64_t exist = 0;
            const int rk = rel + 64 * k;
#pragma unroll
            for (int b = 0; b < 4; ++b) exist |= (ok_bits >> (4 * k + b) & 1) ? 0xFFFFull << (16 * b) : 0;
            sees[k] = exist & (rk <= -64 ? ~0ull
                               : rk < 0  ? (word << -rk) | ((1ull << -rk) - 1)
                               : rk < 64 ? word >> rk : 0);
          }
        }
        if (begin && row_in == 0) keep_o[q] = 0;
        if (!open) {
          // Keys that some row does not attend to: a weight of 0 does not keep an
          // infinity or NaN of v out of the product.  They are looked for, added
          // to the rows that attend to them and set to 0.  With two row tiles
          // both streams come here together; with the keys split, each alone.
          uint32_t *odd_keys = odd_at + (NQ == 2 ? i & 1 : q) * 4;
          auto sync_tile = [&] { named_bar(NQ == 2 ? 1 : 2 + q, NQ == 2 ? 256 : 128); };
          const int first = NQ == 2 ? tid : row_in;
          wait_phase(full0 + 8 * sv, ((2 * i + 1) / NS) & 1, failed, p.error);
          uint8_t *slot = ring + sv * L::kSlot;
          for (int k = first; k < L::kKeys * DC * 8; k += 128 * NQ) {
            const int key = k / (DC * 8);
            const uint4 v = *reinterpret_cast<const uint4 *>(slot + spot<L>(key, k % (DC * 8)));
            if (nonfinite_bits<kType>(v.x) | nonfinite_bits<kType>(v.y) | nonfinite_bits<kType>(v.z) |
                nonfinite_bits<kType>(v.w))
              atomicOr(odd_keys + key / 32, 1u << (key % 32));
          }
          sync_tile();
          const uint32_t odd[4] = {odd_keys[0], odd_keys[1], odd_keys[2], odd_keys[3]};
          if (NQ == 1) sync_tile();                      // the words are read before they change again
          if (odd[0] | odd[1] | odd[2] | odd[3]) {
            if (begin && row_in == 0) keep_o[q] = 1;
#pragma unroll 1
            for (int k = 0; k < L::D; k += 32) {
              uint32_t y[32];
              if (!begin) {
                tc_ld32(y, o_at + k);
                tc_wait_ld(y);
              } else {
#pragma unroll
                for (int e = 0; e < 32; ++e) y[e] = 0;
              }
#pragma unroll 1
              for (int key = 0; key < L::kKeys; ++key) {
                const uint32_t word32 = key < 32 ? odd[0] : key < 64 ? odd[1] : key < 96 ? odd[2] : odd[3];
                if (!(word32 >> (key % 32) & 1) || !((key < 64 ? sees[0] : sees[1]) >> (key % 64) & 1)) continue;
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                  const uint16_t b = *reinterpret_cast<const uint16_t *>(
                      slot + spot<L>(key, (k + e) / 8) + (k + e) % 8 * 2);
                  const float f = kType == kBf16 ? __bfloat162float(__ushort_as_bfloat16(b))
                                                 : __half2float(__ushort_as_half(b));
                  if (!(fabsf(f) < INFINITY)) y[e] = __float_as_uint(__uint_as_float(y[e]) + f);
                }
              }
              __syncwarp();
              tc_st32(o_at + k, y);
            }
            tc_wait_st();
            sync_tile();
            for (int k = first; k < L::kKeys * DC * 8; k += 128 * NQ) {
              uint4 *v = reinterpret_cast<uint4 *>(slot + spot<L>(k / (DC * 8), k % (DC * 8)));
              v->x &= finite_mask<kType>(v->x);
              v->y &= finite_mask<kType>(v->y);
              v->z &= finite_mask<kType>(v->z);
              v->w &= finite_mask<kType>(v->w);
            }
            fence_proxy_async();
            if (first < 4) odd_keys[first] = 0;
            sync_tile();
          }
        }
        // 32 columns of scores, masked
        auto scores = [&](uint32_t (&x)[32], int k) {
          if (!open) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!(sees[k / 2] >> (32 * (k % 2) + e) & 1)) x[e] = 0xFF800000u;
          }
        };
        uint32_t x[4][32];
        float t4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        constexpr int kAtOnce = L::kF8 ? 2 : 4;          // loads of 32 columns held
#pragma unroll
        for (int k0 = 0; k0 < 4; k0 += kAtOnce) {
#pragma unroll
          for (int k = 0; k < kAtOnce; ++k) tc_ld32(x[k], s_at + 32 * (k0 + k));
#pragma unroll
          for (int k = 0; k < kAtOnce; ++k) tc_wait_ld(x[k]);
#pragma unroll
          for (int k = 0; k < kAtOnce; ++k) {
            scores(x[k], k0 + k);
#pragma unroll
            for (int e = 0; e < 32; ++e) t4[e % 4] = fmaxf(t4[e % 4], __uint_as_float(x[k][e]));
          }
        }
        const float top = fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3])) * c;
        const bool raise = top > m + kLag || (m == -INFINITY && top > m);
        // (all lanes of the warp take part in the TMEM accesses)
        if (__any_sync(~0u, raise)) {
          const float m2 = raise ? top : m;
          const float keep = m == m2 ? 1.f : m == -INFINITY ? 0.f : ex2(m - m2);
          if (!begin) {
            // (the product before was made before these scores)
#pragma unroll 1
            for (int k = 0; k < L::D; k += 32) {
              uint32_t y[32];
              tc_ld32(y, o_at + k);
              tc_wait_ld(y);
#pragma unroll
              for (int e = 0; e < 32; ++e) y[e] = __float_as_uint(__uint_as_float(y[e]) * keep);
              tc_st32(o_at + k, y);
            }
            tc_wait_st();
          }
          l *= keep;
          m = m2;
        }
        const float base = m == -INFINITY ? 0.f : m - kWideLift<kType>;
        float l4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          if constexpr (L::kF8) {
            // (the first half's weights lie where its scores were)
            tc_ld32(x[0], s_at + 64 * half);
            tc_ld32(x[1], s_at + 64 * half + 32);
            tc_wait_ld(x[0]);
            tc_wait_ld(x[1]);
            scores(x[0], 2 * half);
            scores(x[1], 2 * half + 1);
          }
          uint32_t w[32];
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            const uint32_t *xs = &x[(L::kF8 ? 0 : 2 * half) + k / 16][k % 16 * 2];
            float a, b;
            fma2(a, b, xs[0], xs[1], c, -base);
            a = ex2(a);
            b = ex2(b);
            add2(l4[k % 2 * 2], l4[k % 2 * 2 + 1], a, b);
            w[k] = pack2<kType>(a, b);
          }
          tc_st32(s_at + 32 * half, w);
          tc_wait_st();
          tc_before();
          mbar_arrive(p_full + 16 * q + 8 * half);
        }
        l += (l4[0] + l4[1]) + (l4[2] + l4[3]);
      }
      n += tiles;
      if (NQ == 1) other += uint32_t(q ? (tiles + 1) / 2 : tiles / 2);
      if (after.valid()) {
        fetch_q(after);
        // both streams read the one row tile: the other's scores are made, too
        if (NQ == 1 && other) wait_phase(s_full + 8 * (1 - q), (other - 1) & 1, failed, p.error);
        store_q(q_exp + (unit + 1) % 2 * L::kRows);
      }

      // ----------------------------------------------------------- results
      const bool some = NQ == 2 || q == 0 || tiles > 1;  // whether the stream had a tile
      if (some) {
        wait_phase(o_full + 8 * q, units & 1, failed, p.error);
        ++units;
        tc_after();
      }
      // after a wait that ran out nothing passes for a number, as in the other kernel
      if (*failed | *stale) l = __int_as_float(0x7FFFFFFF);
      float w0 = 1.f, w1 = 0.f;                          // weights of the streams' outputs
      if constexpr (NQ == 1) {
        state[tid] = make_float2(m, l);
        tc_before();
        sync_rows();
        tc_after();
        const float2 a = state[row_in], b = state[128 + row_in];
        const float both = fmaxf(a.x, b.x);
        w0 = a.x == -INFINITY ? 0.f : ex2(a.x - both);
        w1 = b.x == -INFINITY ? 0.f : ex2(b.x - both);
        l = a.y * w0 + b.y * w1;
        m = both;
      }
      // this thread's columns of its row: all, or its stream's half of them
      const int col0 = NQ == 2 ? 0 : q * (L::D / 2), col1 = NQ == 2 ? L::D : col0 + L::D / 2;
      auto load = [&](int k, uint32_t (&y)[32]) {
        tc_ld32(y, lanes + L::kO + (NQ == 2 ? q * 128 : 0) + k);
        tc_wait_ld(y);
        if constexpr (NQ == 1) {
          // (a NaN of a stream whose rows weigh nothing is kept, too)
#pragma unroll
          for (int e = 0; e < 32; ++e) y[e] = __float_as_uint(__uint_as_float(y[e]) * w0);
          if (tiles > 1) {
            uint32_t z[32];
            tc_ld32(z, lanes + L::kO + 128 + k);
            tc_wait_ld(z);
#pragma unroll
            for (int e = 0; e < 32; ++e) y[e] = __float_as_uint(fmaf(__uint_as_float(z[e]), w1, __uint_as_float(y[e])));
          }
        }
      };
      const bool whole = at.whole();
      const int first = whole ? 0 : at.first(), final = whole ? 0 : at.final();
      const int64_t at_row = (int64_t(at.b) * p.n + node) * p.hq + h;
      uint16_t *out = static_cast<uint16_t *>(p.out) + at_row * p.d;
      auto store = [&](int c, const float (&y)[32], float inv, bool empty) {
        if (!real) return;
#pragma unroll
        for (int k = 0; k < 32; k += 8)
          if (c + k < p.d) {
            float z[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) z[e] = empty ? 0.f : y[k + e] * inv;
            const bool f16 = L::kF8 ? p.q_f16 != 0 : kType == kF16;
            *reinterpret_cast<uint4 *>(out + c + k) =
                make_uint4(pack_out(z[0], z[1], f16), pack_out(z[2], z[3], f16),
                           pack_out(z[4], z[5], f16), pack_out(z[6], z[7], f16));
          }
      };
      auto store_lse = [&](float mm, float ll, bool empty) {
        if (p.lse && real && (NQ == 2 || q == 0))
          p.lse[at_row] = empty ? -INFINITY : (mm - kWideLift<kType> + log2f(ll)) * kLn2;
      };
      if (whole) {
        const bool empty = node >= at.count || (m == -INFINITY && l == 0.f);   // NaN is not nothing
        const float inv = empty ? 0.f : p.v_scale / l;
#pragma unroll 1
        for (int k = col0; k < col1; k += 32) {
          uint32_t y[32];
          load(k, y);
          float f[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) f[e] = __uint_as_float(y[e]);
          store(k, f, inv, empty);
        }
        store_lse(m, l, empty);
      } else {
        // partial results: [4 columns][row], then (m, l) of each row
        const int mine_row = (NQ == 2 ? q * 128 : 0) + row_in;
        auto place = [&](int block) {
          return p.partial + (int64_t(block) * 2 + (block == first ? 1 : 0)) * L::kPartial;
        };
        auto state_of = [&](int block) {
          return __ldcg(reinterpret_cast<const float2 *>(place(block) + L::kRows * L::D) + mine_row);
        };
        Join join(first, final, blockIdx.x, kJoinAtOnce<L>);
        float *to = place(blockIdx.x);
#pragma unroll 1
        for (int k = col0; k < col1; k += 32) {
          uint32_t y[32];
          load(k, y);
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            reinterpret_cast<uint4 *>(to)[(k + e) / 4 * L::kRows + mine_row] =
                make_uint4(y[e], y[e + 1], y[e + 2], y[e + 3]);
        }
#pragma unroll 1
        while (true) {
          if (NQ == 2 || q == 0)
            reinterpret_cast<float2 *>(to + L::kRows * L::D)[mine_row] = make_float2(m, l);
          __threadfence();
          sync_rows();
          if (tid == 0) {
            uint32_t *counter = join.counter(p);
            *last = atomicAdd(counter, 1u) + 1 == join.members();
            if (*last) *counter = 0;
            __threadfence();
          }
          sync_rows();
          if (!*last) break;
          m = -INFINITY;
          l = 0.f;
#pragma unroll 4
          for (int blk = join.lo; blk <= join.hi; blk += join.step) m = fmaxf(m, state_of(blk).x);
#pragma unroll 4
          for (int blk = join.lo; blk <= join.hi; blk += join.step) {
            const float2 st = state_of(blk);
            l += st.y * (st.x == -INFINITY ? 0.f : ex2(st.x - m));
          }
          const bool all = join.last();
          to = place(join.lo);
          const bool empty = node >= at.count || (m == -INFINITY && l == 0.f);
          const float inv = empty ? 0.f : p.v_scale / l;
#pragma unroll 1
          for (int k = col0; k < col1; k += 32) {
            float f[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) f[e] = 0.f;
#pragma unroll 2
            for (int blk = join.lo; blk <= join.hi; blk += join.step) {
              const float mm = state_of(blk).x;
              const float wt = mm == -INFINITY ? 0.f : ex2(mm - m);
              const float4 *part = reinterpret_cast<const float4 *>(place(blk)) + mine_row;
#pragma unroll
              for (int e = 0; e < 32; e += 4) {
                const float4 v = __ldcg(part + (k + e) / 4 * L::kRows);
                f[e] += v.x * wt;
                f[e + 1] += v.y * wt;
                f[e + 2] += v.z * wt;
                f[e + 3] += v.w * wt;
              }
            }
            if (all) {
              store(k, f, inv, empty);
            } else {
              // (these columns of this row are read by no other thread)
#pragma unroll
              for (int e = 0; e < 32; e += 4)
                reinterpret_cast<float4 *>(to)[(k + e) / 4 * L::kRows + mine_row] =
                    make_float4(f[e], f[e + 1], f[e + 2], f[e + 3]);
            }
          }
          if (all) {
            store_lse(m, l, empty);
            break;
          }
          sync_rows();                                   // everybody has read the group's states
          join.next();
        }
      }
      // the outputs are read and *last is free before the next unit begins
      tc_before();
      sync_rows();
      at = after;
    }
  }
  tc_before();
  __syncthreads();
  if (warp == 9) {
    tc_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
  }
}

template <int kCache, int DC, int NQ>
Variant wide_variant() {
  using L = WideCfg<kCache, DC, NQ>;
  static std::atomic<uint64_t> allowed{0};
  return {reinterpret_cast<Kernel>(&wide_kernel<kCache, DC, NQ>), L::kSmem, L::kRows, L::kPartial,
          WideThreads<L::kF8>::kThreads, &allowed};
}

}  // namespace attn
}  // namespace vg
