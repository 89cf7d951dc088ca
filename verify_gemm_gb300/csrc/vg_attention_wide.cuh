// vg_attention_wide.cuh -- the attention kernel for many rows a cache head:
// tcgen05 products with the scores, the weights and the output in TMEM.
//
// From some 40 rows a head on, mma.sync (0.5 PFLOP/s here) and not the cache's
// bytes bounds the kernel of vg_attention.cuh.  Here a block takes one or two
// row tiles of 128 rows through the same keys:
//     S = Q K^T        128 x 64, both operands in shared memory
//     P = 2^(c S - m)  one thread a row: TMEM -> registers -> TMEM, 16 bits
//     O = O + P V      P from TMEM, V in shared memory as it lies (its rows
//                      are the products' k, so it is the transposed operand)
// One thread issues the products, a warpgroup does each row tile's softmax, a
// warp each copies K and V.  S has two buffers a row tile, and P takes the
// place of its S, so that the products of the next keys run under the softmax
// of these: TMEM holds 2 x 128 columns of O and 4 x 64 of S.
// A row's maximum may lag by up to 2^8: O is rescaled, in TMEM by its softmax
// warpgroup, only when the true maximum is more than 8 above the one in use,
// and l carries the same factor.
// The cutting of the line, the pages and the joining of blocks are those of
// vg_attention.cuh.
#pragma once

#include "vg_attention.cuh"

namespace vg {
namespace attn {

constexpr int kWideThreads = 384;
constexpr float kLag = 8.f;                   // log2 of what a maximum may lag
// FP16 weights are at most 2^kLag times 2^lift: lifted to 2^15 in all.
template <int kType>
constexpr float kWideLift = kType == kBf16 ? 0.f : 7.f;

template <int DC, int NQ>
struct WideCfg {
  static constexpr int D = DC * 64;
  static constexpr int kRow = 128, kElems = 64, kChunks = DC;
  static constexpr int kChunk = kTile * kRow;            // 8 KB
  static constexpr int kSlot = DC * kChunk;
  static constexpr int kQChunk = 128 * 128;              // 128 rows of 64 elements
  static constexpr int kQTile = DC * kQChunk;
  static constexpr int kRows = 128 * NQ;
  static constexpr int kFixed = 2048;
  static constexpr int kFit = (227 * 1024 - 1024 - kFixed - NQ * kQTile) / kSlot;
  static constexpr int kSlots = (kFit > 16 ? 16 : kFit) & ~1;
  static constexpr int kSmem = 1024 + kFixed + NQ * kQTile + kSlots * kSlot;
  static constexpr int kPartial = kRows * (D + 2);       // floats of a partial result
  static constexpr uint32_t kO = 0, kS = 256;            // TMEM columns
};

// ------------------------------------------------------------- tcgen05 pieces
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

template <int kType, int DC, int NQ>
__global__ void __launch_bounds__(kWideThreads, 1)
    wide_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ CUtensorMap kmap,
                const __grid_constant__ CUtensorMap vmap) {
  using L = WideCfg<DC, NQ>;
  extern __shared__ uint8_t raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  uint8_t *ring = smem;
  uint8_t *q_smem = smem + L::kSlots * L::kSlot;
  uint8_t *fixed = q_smem + NQ * L::kQTile;
  uint64_t *bars = reinterpret_cast<uint64_t *>(fixed);
  // barriers: slots full, slots free, scores there, weights there, product done, q there
  const uint32_t full0 = smem_addr(bars), empty0 = smem_addr(bars + 16), s_full = smem_addr(bars + 32),
                 p_full = smem_addr(bars + 36), o_full = smem_addr(bars + 40), q_full = smem_addr(bars + 44),
                 finished = smem_addr(bars + 45);
  uint32_t *page_ok = reinterpret_cast<uint32_t *>(fixed + 512);        // [16]
  volatile int *failed = reinterpret_cast<volatile int *>(fixed + 576);
  int *last = reinterpret_cast<int *>(fixed + 580);
  uint32_t *tmem_at = reinterpret_cast<uint32_t *>(fixed + 584);
  uint32_t *odd_at = reinterpret_cast<uint32_t *>(fixed + 592);         // [tile % 2][2]
  volatile int *keep_o = reinterpret_cast<volatile int *>(fixed + 608); // [row tile]
  constexpr int NS = L::kSlots;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  if (tid == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(&kmap) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&vmap) : "memory");
    *failed = 0;
    odd_at[0] = odd_at[1] = odd_at[2] = odd_at[3] = 0;
    for (int s = 0; s < NS; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(s_full + 8 * i, 1);
      mbar_init(p_full + 8 * i, 128);
      mbar_init(o_full + 8 * i, 1);
    }
    mbar_init(q_full, 128 * NQ);
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
  const int group = p.hq / p.hkv;

  if (warp == 8 || warp == 10) {
    // ------------------------------------------------------------- copies
    const int kv = warp == 10;
    copy_tiles<L, NS>(p, at, kv ? &vmap : &kmap, kv, smem_addr(ring), full0, empty0, page_ok, failed);
  } else if (warp == 9) {
    // ----------------------------------------------------------- products
    if (lane == 0) {
      constexpr uint32_t kFmt = kType == kBf16 ? 1 : 0;
      constexpr uint32_t kIdesc = 1u << 4 | kFmt << 7 | kFmt << 10 | (128u / 16) << 24;
      constexpr uint32_t kQk = kIdesc | (uint32_t(kTile) / 8) << 17;
      constexpr uint32_t kPv = kIdesc | 1u << 16 | (uint32_t(L::D) / 8) << 17;   // V: n runs along its rows
      const uint32_t ring0 = smem_addr(ring), q0 = smem_addr(q_smem);
      uint32_t n = 0, q_par = 0;                         // tiles so far
      auto scores = [&](uint32_t i) {                    // S of tile i, every row tile
        const uint32_t s = 2 * i % NS;
        wait_phase(full0 + 8 * s, (2 * i / NS) & 1, failed, p.error);
        tc_after();
#pragma unroll
        for (int q = 0; q < NQ; ++q) {
          const uint32_t d = tmem + L::kS + (q * 2 + (i & 1)) * kTile;
#pragma unroll
          for (int ks = 0; ks < DC * 4; ++ks)
            tc_mma_ss(d, tc_desc(q0 + q * L::kQTile + (ks / 4) * L::kQChunk + (ks % 4) * 32, 16, 1024),
                      tc_desc(ring0 + s * L::kSlot + (ks / 4) * L::kChunk + (ks % 4) * 32, 16, 1024), kQk,
                      ks > 0);
          tc_commit(s_full + 8 * (q * 2 + (i & 1)));
        }
        tc_commit(empty0 + 8 * s);
      };
      for (; at.valid(); at.next(p)) {
        wait_phase(q_full, q_par, failed, p.error);
        q_par ^= 1;
        tc_after();
        const uint32_t end = n + uint32_t(at.t1 - at.t0);
        scores(n);
        for (uint32_t i = n; i < end; ++i) {
          if (i + 1 < end) scores(i + 1);
          const uint32_t s = (2 * i + 1) % NS;
          wait_phase(full0 + 8 * s, ((2 * i + 1) / NS) & 1, failed, p.error);
#pragma unroll
          for (int q = 0; q < NQ; ++q) {
            const uint32_t buf = q * 2 + (i & 1);
            wait_phase(p_full + 8 * buf, (i / 2) & 1, failed, p.error);
            tc_after();
            const bool fresh = i == n && !keep_o[q];     // O begins with this product
#pragma unroll
            for (int ks = 0; ks < kTile / 16; ++ks)
              tc_mma_ts(tmem + L::kO + q * 128, tmem + L::kS + buf * kTile + ks * 8,
                        tc_desc(ring0 + s * L::kSlot + ks * 2048, L::kChunk, 1024), kPv,
                        !fresh || ks > 0);
            tc_commit(o_full + 8 * buf);
          }
          tc_commit(empty0 + 8 * s);
        }
        n = end;
      }
      // nothing is in flight when TMEM is given back
      tc_commit(finished);
      const uint64_t limit = globaltimer() + 10000000;
      while (!mbar_try_wait(finished, 0) && globaltimer() < limit) {
      }
    }
    __syncwarp();
  } else if (warp < 4 * NQ) {
    // ------------------------------------------------------------- softmax
    const int q = warp / 4, row_in = tid % 128;          // row tile, lane of TMEM
    const uint32_t lanes = tmem + (uint32_t(warp % 4 * 32) << 16);
    const uint32_t o_at = lanes + L::kO + q * 128;
    uint32_t n = 0;
    auto sync_rows = [&] { named_bar(1, 128 * NQ); };
    for (; at.valid(); at.next(p)) {
      const int head = at.u / p.blocks, rb = at.u % p.blocks;
      const int row0 = rb * L::kRows, row = row0 + q * 128 + row_in;
      const int node = row / group, h = head * group + row % group;
      const bool real = row < p.rows;
      // q to shared memory, sixteen lanes a row
      {
        const int piece = lane % 16;
#pragma unroll 4
        for (int r = warp % 4 * 2 + lane / 16; r < 128; r += 8) {
          const int rw = row0 + q * 128 + r;
          uint4 v = make_uint4(0, 0, 0, 0);
          if (rw < p.rows && piece * 8 < p.d)
            v = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.q) + at.b * p.qs[0] +
                                                 (rw / group) * p.qs[1] +
                                                 (head * group + rw % group) * p.qs[2] + piece * 8);
          if (piece < DC * 8)
            *reinterpret_cast<uint4 *>(q_smem + q * L::kQTile + (piece / 8) * L::kQChunk + r * 128 +
                                       (((piece % 8) ^ (r & 7)) << 4)) = v;
        }
        fence_proxy_async();
        mbar_arrive(q_full);
      }
      uint64_t word = 0;
      if (real)
        word = (at.count >= 64 ? ~0ull : (1ull << at.count) - 1) &
               (p.tree ? p.tree[int64_t(at.b) * p.n + node] : ~0ull >> (63 - node));
      float m = -INFINITY, l = 0.f;                      // the maximum in use

      for (int tile = at.t0; tile < at.t1; ++tile, ++n) {
        const uint32_t buf = q * 2 + (n & 1), s_at = lanes + L::kS + buf * kTile;
        const uint32_t sv = (2 * n + 1) % NS;
        wait_phase(s_full + 8 * buf, (n / 2) & 1, failed, p.error);
        tc_after();
        const uint32_t ok_bits = page_ok[n % 16];
        uint32_t x[2][32];
        tc_ld32(x[0], s_at);
        tc_ld32(x[1], s_at + 32);
        const int rel = tile * kTile - at.len;           // of the first key to the drafted ones
        const bool open = ok_bits == 15u && rel <= -kTile;
        uint64_t sees = ~0ull;
        if (!open) {
          uint64_t exist = 0;
#pragma unroll
          for (int k = 0; k < 4; ++k) exist |= (ok_bits >> k & 1) ? 0xFFFFull << (16 * k) : 0;
          sees = exist & (rel <= -64 ? ~0ull
                          : rel < 0  ? (word << -rel) | ((1ull << -rel) - 1)
                          : rel < 64 ? word >> rel : 0);
        }
        tc_wait_ld(x[0]);
        tc_wait_ld(x[1]);
        float top = -INFINITY;
        if (!open) {
#pragma unroll
          for (int k = 0; k < 64; ++k) {
            const float f = __uint_as_float(x[k / 32][k % 32]) * p.c;
            x[k / 32][k % 32] = __float_as_uint((sees >> k & 1) ? f : -INFINITY);
            top = fmaxf(top, __uint_as_float(x[k / 32][k % 32]));
          }
        } else {
          float t4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int k = 0; k < 64; ++k) {
            const float f = __uint_as_float(x[k / 32][k % 32]) * p.c;
            x[k / 32][k % 32] = __float_as_uint(f);
            t4[k % 4] = fmaxf(t4[k % 4], f);
          }
          top = fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3]));
        }
        const bool raise = top > m + kLag || (m == -INFINITY && top > m);
        // (all lanes of the warp take part in the TMEM accesses)
        if (__any_sync(~0u, raise)) {
          const float m2 = raise ? top : m;
          const float keep = m == m2 ? 1.f : m == -INFINITY ? 0.f : ex2(m - m2);
          if (tile > at.t0) {
            // the product before has been made, the next waits for these weights
            wait_phase(o_full + 8 * (q * 2 + ((n - 1) & 1)), ((n - 1) / 2) & 1, failed, p.error);
            tc_after();
#pragma unroll 1
            for (int c = 0; c < L::D; c += 32) {
              uint32_t y[32];
              tc_ld32(y, o_at + c);
              tc_wait_ld(y);
#pragma unroll
              for (int k = 0; k < 32; ++k) y[k] = __float_as_uint(__uint_as_float(y[k]) * keep);
              tc_st32(o_at + c, y);
            }
            tc_wait_st();
          }
          l *= keep;
          m = m2;
        }
        const float base = m == -INFINITY ? 0.f : m - kWideLift<kType>;
        float l4[4] = {0.f, 0.f, 0.f, 0.f};
        uint32_t w[32];
#pragma unroll
        for (int k = 0; k < 32; ++k) {
          const float a = ex2(__uint_as_float(x[k / 16][k % 16 * 2]) - base);
          const float b = ex2(__uint_as_float(x[k / 16][k % 16 * 2 + 1]) - base);
          l4[k % 4] += a + b;
          w[k] = pack2<kType>(a, b);
        }
        l += (l4[0] + l4[1]) + (l4[2] + l4[3]);
        tc_st32(s_at, w);
        if (tile == at.t0 && row_in == 0) keep_o[q] = 0;
        if (!open) {
          uint32_t *odd_keys = odd_at + (n & 1) * 2;
          // Keys that some row does not attend to: a weight of 0 does not keep an
          // infinity or NaN of v out of the product.  They are looked for, added
          // to the rows that attend to them and set to 0.
          wait_phase(full0 + 8 * sv, ((2 * n + 1) / NS) & 1, failed, p.error);
          uint8_t *slot = ring + sv * L::kSlot;
          for (int k = tid; k < kTile * DC * 8; k += 128 * NQ) {
            const int key = k / (DC * 8);
            const uint4 v = *reinterpret_cast<const uint4 *>(slot + spot<L>(key, k % (DC * 8)));
            if (nonfinite_bits<kType>(v.x) | nonfinite_bits<kType>(v.y) | nonfinite_bits<kType>(v.z) |
                nonfinite_bits<kType>(v.w))
              atomicOr(odd_keys + key / 32, 1u << (key % 32));
          }
          sync_rows();
          const uint64_t odd = uint64_t(odd_keys[1]) << 32 | odd_keys[0];
          if (odd) {
            if (tile > at.t0) {
              wait_phase(o_full + 8 * (q * 2 + ((n - 1) & 1)), ((n - 1) / 2) & 1, failed, p.error);
              tc_after();
            } else if (row_in == 0) {
              keep_o[q] = 1;
            }
            const uint64_t mine = odd & sees;
#pragma unroll 1
            for (int c = 0; c < L::D; c += 32) {
              uint32_t y[32];
              if (tile > at.t0) {
                tc_ld32(y, o_at + c);
                tc_wait_ld(y);
              } else {
#pragma unroll
                for (int k = 0; k < 32; ++k) y[k] = 0;
              }
#pragma unroll 1
              for (int key = 0; key < kTile; ++key) {
                if (!(mine >> key & 1)) continue;
#pragma unroll
                for (int k = 0; k < 32; ++k) {
                  const uint16_t e = *reinterpret_cast<const uint16_t *>(
                      slot + spot<L>(key, (c + k) / 8) + (c + k) % 8 * 2);
                  const float f = kType == kBf16 ? __bfloat162float(__ushort_as_bfloat16(e))
                                                 : __half2float(__ushort_as_half(e));
                  if (!(fabsf(f) < INFINITY)) y[k] = __float_as_uint(__uint_as_float(y[k]) + f);
                }
              }
              __syncwarp();
              tc_st32(o_at + c, y);
            }
            tc_wait_st();
            sync_rows();
            for (int k = tid; k < kTile * DC * 8; k += 128 * NQ) {
              uint4 *v = reinterpret_cast<uint4 *>(slot + spot<L>(k / (DC * 8), k % (DC * 8)));
              v->x &= finite_mask<kType>(v->x);
              v->y &= finite_mask<kType>(v->y);
              v->z &= finite_mask<kType>(v->z);
              v->w &= finite_mask<kType>(v->w);
            }
            fence_proxy_async();
            if (tid == 0) odd_keys[0] = odd_keys[1] = 0;
            sync_rows();
          }
        }
        tc_wait_st();
        tc_before();
        mbar_arrive(p_full + 8 * buf);
      }

      // ----------------------------------------------------------- results
      wait_phase(o_full + 8 * (q * 2 + ((n - 1) & 1)), ((n - 1) / 2) & 1, failed, p.error);
      tc_after();
      const int first = at.block_of(0), final = at.block_of(at.tiles - 1);
      const bool whole = first == final;
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
            *reinterpret_cast<uint4 *>(out + c + k) =
                make_uint4(pack2<kType>(z[0], z[1]), pack2<kType>(z[2], z[3]),
                           pack2<kType>(z[4], z[5]), pack2<kType>(z[6], z[7]));
          }
      };
      auto store_lse = [&](float mm, float ll, bool empty) {
        if (p.lse && real)
          p.lse[at_row] = empty ? -INFINITY : (mm - kWideLift<kType> + log2f(ll)) * kLn2;
      };
      if (whole) {
        const bool empty = node >= at.count || (m == -INFINITY && l == 0.f);   // NaN is not nothing
        const float inv = empty ? 0.f : p.v_scale / l;
#pragma unroll 1
        for (int c = 0; c < L::D; c += 32) {
          uint32_t y[32];
          tc_ld32(y, o_at + c);
          tc_wait_ld(y);
          float f[32];
#pragma unroll
          for (int k = 0; k < 32; ++k) f[k] = __uint_as_float(y[k]);
          store(c, f, inv, empty);
        }
        store_lse(m, l, empty);
      } else {
        // partial results: [4 columns][row], then (m, l) of each row
        const int mine_row = q * 128 + row_in;
        auto place = [&](int block) {
          return p.partial + (int64_t(block) * 2 + (block == first ? 1 : 0)) * L::kPartial;
        };
        float *mine = place(blockIdx.x);
#pragma unroll 1
        for (int c = 0; c < L::D; c += 32) {
          uint32_t y[32];
          tc_ld32(y, o_at + c);
          tc_wait_ld(y);
#pragma unroll
          for (int k = 0; k < 32; k += 4)
            reinterpret_cast<uint4 *>(mine)[(c + k) / 4 * L::kRows + mine_row] =
                make_uint4(y[k], y[k + 1], y[k + 2], y[k + 3]);
        }
        reinterpret_cast<float2 *>(mine + L::kRows * L::D)[mine_row] = make_float2(m, l);
        __threadfence();
        sync_rows();
        if (tid == 0) {
          const uint32_t before = atomicAdd(p.arrived + first, 1u);
          *last = before == uint32_t(final - first);
          if (*last) p.arrived[first] = 0;
          __threadfence();
        }
        sync_rows();
        if (*last) {
          float top = -INFINITY, sum = 0.f;
          for (int blk = first; blk <= final; ++blk)
            top = fmaxf(top, __ldcg(reinterpret_cast<const float2 *>(place(blk) + L::kRows * L::D) + mine_row).x);
          for (int blk = first; blk <= final; ++blk) {
            const float2 st = __ldcg(reinterpret_cast<const float2 *>(place(blk) + L::kRows * L::D) + mine_row);
            sum += st.y * (st.x == -INFINITY ? 0.f : ex2(st.x - top));
          }
          const bool empty = node >= at.count || (top == -INFINITY && sum == 0.f);
          const float inv = empty ? 0.f : p.v_scale / sum;
#pragma unroll 1
          for (int c = 0; c < L::D; c += 32) {
            float f[32];
#pragma unroll
            for (int k = 0; k < 32; ++k) f[k] = 0.f;
#pragma unroll 2
            for (int blk = first; blk <= final; ++blk) {
              const float *part = place(blk);
              const float mm = __ldcg(reinterpret_cast<const float2 *>(part + L::kRows * L::D) + mine_row).x;
              const float wt = mm == -INFINITY ? 0.f : ex2(mm - top);
#pragma unroll
              for (int k = 0; k < 32; k += 4) {
                const float4 v = __ldcg(reinterpret_cast<const float4 *>(part) + (c + k) / 4 * L::kRows + mine_row);
                f[k] += v.x * wt;
                f[k + 1] += v.y * wt;
                f[k + 2] += v.z * wt;
                f[k + 3] += v.w * wt;
              }
            }
            store(c, f, inv, empty);
          }
          store_lse(top, sum, empty);
        }
        sync_rows();                                     // *last is free again
      }
      tc_before();
    }
  }
  tc_before();
  __syncthreads();
  if (warp == 9) {
    tc_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
  }
}

template <int kType, int DC, int NQ>
Variant wide_variant() {
  using L = WideCfg<DC, NQ>;
  return {reinterpret_cast<Kernel>(&wide_kernel<kType, DC, NQ>), L::kSmem, L::kRows, L::kPartial};
}

}  // namespace attn
}  // namespace vg
