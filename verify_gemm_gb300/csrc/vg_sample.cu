// vg_sample.cu -- vg_probabilities (softmax of logits with a temperature per
// row) and vg_verify_tree (verification of drafted tokens).
#include <algorithm>
#include <cmath>

#include "vg_rows.cuh"

namespace vg {
namespace {

// ------------------------------------------------------------ probabilities
// A cluster of blocks a row.  Each thread copies its share of the row to
// shared memory (asynchronously, so every block of an SM has its whole share
// in flight) and reads it from there three times: each warp takes its largest
// logit m_w and, with c = log2 e / T and b_w = m_w c, s_w = sum 2^(x c - b_w);
// every block gets every warp's pair through distributed shared memory; and
// with B = max b_w, S = sum s_w 2^(b_w - B)
//     out = 2^(x c - b_w) 2^(b_w - B) / S.
// (b_w is one rounded number for the whole warp, so its rounding cancels.)
// A row is read once and written once, with one barrier of the cluster
// between, and bytes bound it.  A greedy row (T <= 0) exchanges (m_w, its
// first index) instead.
//
// 256 rows of 151936 BF16 logits (233 MB read and written): 52 us, 4.5 TB/s.
// An exponential is taken twice an element, which costs less than 4 bytes more
// of shared memory for each.  Shares of 80 KB, 512 threads a block and stores
// that stay in L2 measured the same, shares of 20 KB 60 us: all blocks of a wave
// copy, compute and store together, and HBM waits while they compute.  Stores
// of whole sectors, by way of shuffles, took 50 us, but one row 6.6.  One row:
// 4.6 us, of which the launch and the exchange are most.
//
// Elements go by units of 8 on the grid of the whole array, so that loads
// and stores are aligned whatever the row's length; the units at a row's two
// ends go element by element.
constexpr int kProbThreads = 256, kProbWarps = kProbThreads / 32;
constexpr int kProbShare = 40 * 1024;          // bytes of a row a block should hold at most ...
constexpr int kProbShareMax = 96 * 1024;       // ... and may
// kHeld: the block's share fits its shared memory; otherwise it is read from
// memory each time (rows of any length).
template <typename T, bool kHeld>
__global__ void __launch_bounds__(kProbThreads)
    probabilities_kernel(const T *x, int64_t V, const float *temperature, float *out) {
  extern __shared__ __align__(16) uint8_t held[];
  __shared__ __align__(16) ulonglong2 table[kMaxCluster * kProbWarps];
  const uint32_t rank = cluster_rank(), blocks = cluster_size();
  const int64_t row = blockIdx.x / blocks;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int64_t lo = row * V, hi = lo + V;
  const int64_t stride = int64_t(blocks) * kProbThreads;
  const int64_t u0 = lo / 8 + rank * kProbThreads + threadIdx.x, end = (hi + 7) / 8;
  // a block must have begun before others write to it: said here, waited for there
  if (blocks > 1) cluster_arrive();
  constexpr int kPart = sizeof(T) / 2;          // 16-byte parts of a unit, apart in shared memory
  Unit<T> *units = reinterpret_cast<Unit<T> *>(held);
  uint4 *parts = reinterpret_cast<uint4 *>(units) + threadIdx.x;
  if constexpr (kHeld) {
    uint4 *to = parts;
    for (int64_t u = u0; u < end; u += stride, to += kPart * kProbThreads) {
      if (u * 8 >= lo && u * 8 + 8 <= hi) {
#pragma unroll
        for (int k = 0; k < kPart; ++k)
          copy16(to + k * kProbThreads, reinterpret_cast<const uint4 *>(x + u * 8) + k);
      } else {
        const Unit<T> v = load_unit(x, u, lo, hi);
#pragma unroll
        for (int k = 0; k < kPart; ++k) to[k * kProbThreads] = v.w[k];
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");   // a thread reads only what it copied
  }
  const float t = temperature ? temperature[row] : 1.f;
  const bool greedy = t <= 0.f;
  // At the ends of T c is neither 0, which -infinity makes a NaN of, nor infinite,
  // which the maximum's 0 does: with 2^-149 every finite logit weighs 1, with the
  // largest number a logit 2^-121 below the maximum nothing.  A T of NaN stays one.
  float c = kLog2e / t;
  c = c == 0.f ? __uint_as_float(1) : c == INFINITY ? 0x1.fffffep127f : c;
  // units by the place of their first element in the row (-7 and up)
  const int first = int(u0 * 8 - lo), count = int(V), step = int(stride) * 8;
  auto each = [&](auto &&f) {
    const uint4 *from = parts;
#pragma unroll 2
    for (int r = first; r < count; r += step, from += kPart * kProbThreads) {
      Unit<T> v;
      if constexpr (kHeld) {
#pragma unroll
        for (int k = 0; k < kPart; ++k) v.w[k] = from[k * kProbThreads];
      } else {
        v = load_unit(x, (lo + r) / 8, lo, hi);
      }
      f(r, v);
    }
  };
  Largest<T> largest;
  each([&](int, const Unit<T> &v) { largest.take(v); });
  float m = largest.value();
#pragma unroll
  for (int w = 16; w; w /= 2) m = max_nan(m, __shfl_xor_sync(~0u, m, w));
  const float base = m == -INFINITY ? 0.f : m;
  // 2^((x - base) c) of a unit; the difference first, as x c may overflow
  auto weigh = [&](const Unit<T> &v, float2 (&e)[4]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 d = mul2(add2(v.pair(k), make_float2(-base, -base)), make_float2(c, c));
      e[k] = make_float2(ex2(d.x), ex2(d.y));
    }
  };
  uint64_t second = 0;                         // the sum, or the first index of the maximum
  if (greedy) {
    int at = count;
    each([&](int r, const Unit<T> &v) {
#pragma unroll
      for (int k = 3; k >= 0; --k) {
        const float2 p = v.pair(k);
        if (p.y == m && m != -INFINITY) at = min(at, r + 2 * k + 1);
        if (p.x == m && m != -INFINITY) at = min(at, r + 2 * k);
      }
    });
#pragma unroll
    for (int w = 16; w; w /= 2) at = min(at, __shfl_xor_sync(~0u, at, w));
    second = uint64_t(at);
  } else {
    float2 sums = make_float2(0.f, 0.f);
    each([&](int, const Unit<T> &v) {
      float2 e[4];
      weigh(v, e);
      sums = add2(sums, add2(add2(e[0], e[1]), add2(e[2], e[3])));
    });
    float sum = sums.x + sums.y;
#pragma unroll
    for (int w = 16; w; w /= 2) sum += __shfl_xor_sync(~0u, sum, w);
    second = __float_as_uint(sum);
  }
  if (blocks > 1) cluster_wait();
  if (lane < int(blocks))
    cluster_store(&table[rank * kProbWarps + warp], lane, __float_as_uint(m), second);
  if (blocks > 1) cluster_sync();
  else __syncthreads();
  const int entries = int(blocks) * kProbWarps;
  float top = -INFINITY;
  for (int i = lane; i < entries; i += 32) top = max_nan(top, __uint_as_float(uint32_t(table[i].x)));
#pragma unroll
  for (int w = 16; w; w /= 2) top = max_nan(top, __shfl_xor_sync(~0u, top, w));
  if (greedy) {
    int at = count;
    for (int i = lane; i < entries; i += 32)
      if (__uint_as_float(uint32_t(table[i].x)) == top) at = min(at, int(table[i].y));
#pragma unroll
    for (int w = 16; w; w /= 2) at = min(at, __shfl_xor_sync(~0u, at, w));
    for (int r = first; r < count; r += step) {
      float2 y[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        y[k] = make_float2(r + 2 * k == at ? 1.f : 0.f, r + 2 * k + 1 == at ? 1.f : 0.f);
      store_unit(out + lo, r, count, y);
    }
    return;
  }
  const float all = top == -INFINITY ? 0.f : top;
  float sum = 0.f;
  for (int i = lane; i < entries; i += 32) {
    const float mw = __uint_as_float(uint32_t(table[i].x));
    // a warp without a finite logit has summed from 0: its sum is 0, or NaN
    sum += __uint_as_float(uint32_t(table[i].y)) * ex2(((mw == -INFINITY ? all : mw) - all) * c);
  }
#pragma unroll
  for (int w = 16; w; w /= 2) sum += __shfl_xor_sync(~0u, sum, w);
  const float scale = (sum == 0.f ? 0.f : 1.f / sum) * ex2(m == -INFINITY ? 0.f : (base - all) * c);
  each([&](int r, const Unit<T> &v) {
    float2 y[4];
    weigh(v, y);
#pragma unroll
    for (int k = 0; k < 4; ++k) y[k] = mul2(y[k], make_float2(scale, scale));
    store_unit(out + lo, r, count, y);
  });
}

// Blocks a row: as few as hold it, up to 8 while the rows leave SMs idle, and
// 16, more than a portable cluster, for a few rows (151936 BF16 logits: one row
// 4.6 us against 5.9 with 8, eight rows 7.3 against 6.5).
template <typename T>
cudaError_t launch_probabilities(const T *x, int64_t rows, int64_t V, const float *temperature,
                                 float *out, int sms, cudaStream_t st) {
  const int64_t units = V / 8 + 2, size = 8 * sizeof(T);
  int c = 1;
  while (c < 8 &&
         (units * size > int64_t(kProbShare) * c || (rows * c < 2 * sms && units > kProbThreads * c)))
    c *= 2;
  if (c == 8 && units > 8 * kProbThreads && rows * 32 <= sms) c = kMaxCluster;
  const int64_t each = (units + int64_t(c) * kProbThreads - 1) / (int64_t(c) * kProbThreads);
  const int64_t share = each * kProbThreads * size;
  const unsigned grid = unsigned(rows) * unsigned(c);
  // (more than 48 KB, the kernel's own words included, have to be asked for)
  static std::atomic<uint64_t> allowed[2];
  const bool held = share <= kProbShareMax;
  void (*fn)(const T *, int64_t, const float *, float *) =
      held ? &probabilities_kernel<T, true> : &probabilities_kernel<T, false>;
  if (const cudaError_t e = allow(fn, held ? kProbShareMax : 0, allowed[held])) return e;
  return launch_clusters(fn, grid, kProbThreads, c, held ? int(share) : 0, st, x, V, temperature, out);
}

// -------------------------------------------------------------- verification
// All children of a node were drafted from one q, so the residual after its
// k-th refusal is max(p - a_k q, 0) with a_1 = 1 and a_(k+1) = a_k + S_k,
// S_k the residual's sum: max(max(p - a q, 0) - S q, 0) = max(p - (a + S) q, 0)
// because S q >= 0.  So a refusal costs one pass over two rows and leaves
// one number, and the rows of accepted nodes are never read whole.
//
// Fixed point: p, q and the sums S in units of 2^-60 (a row sums to less
// than 16), a in units of 2^-56, which hold up to 256.  1023 refusals can bring
// it to 1 + 16 * 1023, so it is counted beyond that, and from 256 on entries
// are taken with a in units of 2^-48: a cut of 2^-56 of it at most, as below.
//
// A cluster of blocks a sequence.  Every warp of it owns one run of the row:
// it adds up its run, and every block gets every warp's sum through
// distributed shared memory, so that each walks the tree by itself and alike;
// the warp whose run holds the drawn index finds it.
//
// A sequence's passes follow one another (what is read next depends on the
// last sum), and a pass is both rows' bytes over one cluster, some ten 64-bit
// integer operations an entry and a barrier: latency bounds a chain and the
// slowest tree a batch.  Over 151936 entries: a chain of 7 drafts 10.7 us; a
// batch of 48 trees of 15 drafts 43 us, set by the trees with the most refusals
// and by 38 sequences being resident at a time (8 blocks each, two blocks an SM);
// warps issue 39 % of the time.
constexpr int kVerThreads = 512, kVerWarps = kVerThreads / 32;
constexpr int kVerCluster = 16;                  // most blocks a sequence
constexpr int kMaxNodes = 1024;

// To [0, 1], NaN to 0.
__device__ __forceinline__ float as_probability(float x) { return __saturatef(x); }
// ... in units of 2^-60, rounded down: x = m 2^(e - 150), so m 2^37 >> (127 - e).
// (A conversion to 64 bits runs at 2 a clock and SM here: 13 us for a run of
// 25 000 entries.)
__device__ __forceinline__ uint64_t to_fixed(float x) {
  const uint32_t bits = __float_as_uint(as_probability(x)), e = bits >> 23;
  const uint64_t m = uint64_t(((bits & 0x7FFFFFu) | 0x800000u) << 5) << 32;
  uint64_t y;
  asm("shr.b64 %0, %1, %2;" : "=l"(y) : "l"(m), "r"(127u - e));   // 0 from 64 on
  return y;
}

constexpr uint64_t kOne = 1ull << 56;            // a = 1

// max(p - a q, 0) in units of 2^-60.  Modes: a = 0; a = 1; a < 8, where both
// factors of (y a) >> 56 fit 64 bits with the shift made beforehand; a < 256;
// any a, in units of 2^-48.
template <int kMode>
__device__ __forceinline__ uint64_t residual(float p, float q, uint64_t a) {
  const uint64_t x = to_fixed(p);
  if (kMode == 0) return x;
  uint64_t y = to_fixed(q);
  if (kMode == 2) y = __umul64hi(y << 3, a << 5);
  if (kMode >= 3) {
    constexpr int kShift = kMode == 3 ? 56 : 48;
    const uint64_t hi = __umul64hi(y, a), lo = y * a;
    y = hi >> kShift ? ~0ull : (hi << (64 - kShift)) | (lo >> kShift);
  }
  return x > y ? x - y : 0;
}
// a while the tree is walked: whole 256s and the rest in units of 2^-56.
struct Weight {
  uint64_t rest = 0;
  uint32_t whole = 0;
  __device__ __forceinline__ bool zero() const { return rest == 0 && whole == 0; }
  // one more refusal, after which the residual summed to S
  __device__ __forceinline__ void refuse(uint64_t S) {
    const uint64_t next = zero() ? kOne : rest + (S >> 4);
    whole += next < rest;
    rest = next;
  }
  // in the units that `residual` takes it in
  __device__ __forceinline__ uint64_t units() const { return whole ? uint64_t(whole) << 56 | rest >> 8 : rest; }
  __device__ __forceinline__ uint64_t left(float p, float q) const {
    return whole ? residual<4>(p, q, units()) : residual<3>(p, q, rest);
  }
};
// Calls f with the mode of `a` (in units of 2^-48: `coarse`) as a constant.
template <typename F>
__device__ __forceinline__ auto with_mode(uint64_t a, bool coarse, F &&f) {
  if (coarse) return f(std::integral_constant<int, 4>{});
  if (a == 0) return f(std::integral_constant<int, 0>{});
  if (a == kOne) return f(std::integral_constant<int, 1>{});
  if (a < 8 * kOne) return f(std::integral_constant<int, 2>{});
  return f(std::integral_constant<int, 3>{});
}

__device__ __forceinline__ uint64_t warp_sum(uint64_t x) {
#pragma unroll
  for (int w = 16; w; w /= 2) x += __shfl_xor_sync(~0u, x, w);
  return x;
}

struct VerifyParams {
  const float *p, *q;
  const int32_t *tokens, *parents, *counts;
  const float *u;
  int32_t *accepted, *path, *out;
  int64_t V;
  int n, q_rows;
};

// Four consecutive entries of a row, those at or past `last` as 0.
template <bool kVector>
__device__ __forceinline__ float4 load4(const float *row, int64_t e, int64_t last) {
  if (kVector) return e < last ? __ldg(reinterpret_cast<const float4 *>(row + e)) : make_float4(0, 0, 0, 0);
  float4 v;
  v.x = e < last ? __ldg(row + e) : 0.f;
  v.y = e + 1 < last ? __ldg(row + e + 1) : 0.f;
  v.z = e + 2 < last ? __ldg(row + e + 2) : 0.f;
  v.w = e + 3 < last ? __ldg(row + e + 3) : 0.f;
  return v;
}

template <int kMode>
__device__ __forceinline__ uint64_t four(const float4 &p, const float4 &q, uint64_t a) {
  return residual<kMode>(p.x, q.x, a) + residual<kMode>(p.y, q.y, a) +
         residual<kMode>(p.z, q.z, a) + residual<kMode>(p.w, q.w, a);
}

// kVector: vocab % 4 == 0, so every row is 16-byte aligned.
template <bool kVector>
__global__ void __launch_bounds__(kVerThreads, 2) verify_kernel(const VerifyParams v) {
  __shared__ float pt[kMaxNodes], qt[kMaxNodes], su[kMaxNodes];
  __shared__ int16_t par[kMaxNodes];             // -1: no node to try
  __shared__ __align__(16) ulonglong2 table[2][kVerCluster * kVerWarps];
  __shared__ uint64_t s_a;
  __shared__ int s_cur, s_more, s_kept, s_coarse;
  const uint32_t rank = cluster_rank(), blocks = cluster_size();
  const int b = blockIdx.x / blocks, tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int64_t V = v.V;
  const int n = v.counts ? min(max(v.counts[b], 0), v.n) : v.n;
  const float *prow = v.p + int64_t(b) * v.n * V;
  const float *qrow = v.q + int64_t(b) * v.q_rows * V;
  const int32_t *tokens = v.tokens + int64_t(b) * v.n;
  int32_t *path = v.path + int64_t(b) * v.n, *out = v.out + int64_t(b) * (v.n + 1);
  if (blocks > 1) cluster_arrive();
  for (int i = tid; i < v.n; i += kVerThreads) {
    su[i] = v.u[int64_t(b) * v.n + i];
    par[i] = -1;
    if (i > 0 && i < n) {
      const int f = v.parents[int64_t(b) * v.n + i], t = tokens[i];
      if (f >= 0 && f < i && f < v.q_rows && t >= 0 && t < V) {
        par[i] = int16_t(f);
        pt[i] = as_probability(prow[f * V + t]);
        qt[i] = as_probability(qrow[f * V + t]);
      }
    }
  }
  // Runs are whole steps of 128 entries (4 a lane) and follow each other in
  // the order of the warps: the sums of the warps before are the running sum.
  const int runs = int(blocks) * kVerWarps, mine = int(rank) * kVerWarps + warp;
  const int64_t run = ((V + runs - 1) / runs + 127) / 128 * 128;
  const int64_t first = min(run * mine, V), last = min(first + run, V);
  if (blocks > 1) cluster_wait();                // every block has begun ...
  __syncthreads();                               // ... and this one's nodes are there (written after its arrival)
  int i = 1, cur = 0, kept = 0;                  // thread 0's walk
  Weight a;
  uint64_t S = 1ull << 60, total = 0;
  bool summed = false;
  uint32_t pass = 0;
  while (true) {
    if (tid == 0) {
      s_more = 0;
      for (; i < n; ++i) {
        if (par[i] != cur) continue;
        const double left = double(su[i]) * double(qt[i]) * double(S);
        const bool ok = a.zero() ? left < double(pt[i]) * double(1ull << 60) : left < double(a.left(pt[i], qt[i]));
        if (ok) {
          if (rank == 0) {
            path[kept] = i;
            out[kept] = tokens[i];
          }
          ++kept;
          cur = i;
          a = Weight{};
          S = 1ull << 60;
          summed = false;
        } else {
          a.refuse(S);
          s_more = 1;
          ++i;
          break;
        }
      }
      // the end: the sums of p itself, where none or empty ones are at hand
      if (!s_more && (!summed || (total == 0 && !a.zero()))) {
        a = Weight{};
        s_more = 2;
      }
      s_cur = cur;
      s_a = a.units();
      s_coarse = a.whole != 0;
      s_kept = kept;
    }
    __syncthreads();
    const int more = s_more, node = s_cur;
    const uint64_t aa = s_a;
    const bool coarse = s_coarse;
    const float *pr = prow + node * V;
    const float *qr = qrow + (node < v.q_rows ? node : 0) * V;
    if (more) {
      ++pass;
      uint64_t sum = with_mode(aa, coarse, [&](auto mode) {
        constexpr int kMode = decltype(mode)::value;
        uint64_t sum = 0;
        for (int64_t e0 = first; e0 < last; e0 += 4 * 128) {
          float4 p4[4], q4[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int64_t e = e0 + k * 128 + lane * 4;
            p4[k] = load4<kVector>(pr, e, last);
            q4[k] = kMode ? load4<kVector>(qr, e, last) : make_float4(0, 0, 0, 0);
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) sum += four<kMode>(p4[k], q4[k], aa);
        }
        return sum;
      });
      sum = warp_sum(sum);
      // two tables in turn: a block may still read the one before
      if (lane < int(blocks)) cluster_store(&table[pass & 1][mine], lane, sum, 0);
      if (blocks > 1) cluster_sync();
      else __syncthreads();
      if (warp == 0) {
        uint64_t x = 0;
        for (int k = lane; k < runs; k += 32) x += table[pass & 1][k].x;
        total = warp_sum(x);
        S = total;
        summed = true;
      }
      if (more == 1) continue;
    }
    // draw: the warp whose run the threshold falls into looks it up
    uint64_t whole = 0, before = 0;
    for (int k = lane; k < runs; k += 32) {
      const uint64_t x = table[pass & 1][k].x;
      whole += x;
      if (k < mine) before += x;
    }
    whole = warp_sum(whole);
    before = warp_sum(before);
    const float u0 = fminf(fmaxf(su[0], 0.f), 0x1.fffffep-1f);
    const uint64_t mark = __umul64hi(uint64_t(double(u0) * 18446744073709551616.0), whole);
    const int at = s_kept;
    if (rank == 0) {
      if (tid == 0) v.accepted[b] = at;
      for (int k = at + tid; k < v.n; k += kVerThreads) path[k] = -1;
      for (int k = at + 1 + tid; k <= v.n; k += kVerThreads) out[k] = -1;
      if (tid == 0 && whole == 0) out[at] = -1;
    }
    if (whole != 0 && before <= mark && mark - before < table[pass & 1][mine].x) {
      const int64_t found = with_mode(aa, coarse, [&](auto mode) -> int64_t {
        constexpr int kMode = decltype(mode)::value;
        uint64_t c = before;
        for (int64_t e0 = first; e0 < last; e0 += 4 * 128) {
          float4 p4[4], q4[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int64_t e = e0 + k * 128 + lane * 4;
            p4[k] = load4<kVector>(pr, e, last);
            q4[k] = kMode ? load4<kVector>(qr, e, last) : make_float4(0, 0, 0, 0);
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint64_t own = four<kMode>(p4[k], q4[k], aa);
            uint64_t x = own;
#pragma unroll
            for (int w = 1; w < 32; w *= 2) {
              const uint64_t y = __shfl_up_sync(~0u, x, w);
              if (lane >= w) x += y;
            }
            const uint32_t over = __ballot_sync(~0u, c + x > mark);
            if (over) {
              // one of the four of the first lane that is over
              uint64_t y = c + x - own;
              const float pv[4] = {p4[k].x, p4[k].y, p4[k].z, p4[k].w};
              const float qv[4] = {q4[k].x, q4[k].y, q4[k].z, q4[k].w};
              int hit = 0;
#pragma unroll
              for (int j = 0; j < 3; ++j) {
                y += residual<kMode>(pv[j], qv[j], aa);
                if (y <= mark) hit = j + 1;
              }
              return e0 + k * 128 + lane * 4 + __shfl_sync(~0u, hit, __ffs(over) - 1) +
                     4 * (__ffs(over) - 1 - lane);
            }
            c += __shfl_sync(~0u, x, 31);
          }
        }
        return -1;
      });
      if (lane == 0) out[at] = int32_t(found);
    }
    return;
  }
}

}  // namespace
}  // namespace vg

using namespace vg;

extern "C" vg_status vg_probabilities(const void *x, int type, int64_t rows, int64_t vocab,
                                      const float *temperature, float *out, vg_stream_t stream) {
  if (!x || !out || rows < 1 || vocab < 1) return VG_ERR_INVALID_ARG;
  if (type != VG_TYPE_BF16 && type != VG_TYPE_FP16 && type != VG_TYPE_FP32)
    return VG_ERR_INVALID_ARG;
  if (vocab >= (int64_t(1) << 28) || rows >= (int64_t(1) << 27)) return VG_ERR_UNSUPPORTED;
  if (!aligned16(x) || !aligned16(out)) return VG_ERR_ALIGNMENT;
  int sms = 0;
  if (vg_status s = device_sms(&sms)) return s;
  cudaStream_t st = as_cuda(stream);
  if (type == VG_TYPE_BF16)
    VG_CUDA(launch_probabilities(static_cast<const __nv_bfloat16 *>(x), rows, vocab, temperature,
                                 out, sms, st));
  else if (type == VG_TYPE_FP16)
    VG_CUDA(launch_probabilities(static_cast<const __half *>(x), rows, vocab, temperature, out, sms,
                                 st));
  else
    VG_CUDA(launch_probabilities(static_cast<const float *>(x), rows, vocab, temperature, out, sms,
                                 st));
  VG_LAUNCH_CHECK();
  return VG_OK;
}

extern "C" vg_status vg_verify_tree(const float *p, const float *q, const int32_t *tokens,
                                    const int32_t *parents, const int32_t *counts, const float *u,
                                    int batch, int n, int q_rows, int64_t vocab,
                                    int32_t *accepted, int32_t *path, int32_t *out,
                                    vg_stream_t stream) {
  if (!p || !tokens || !parents || !u || !accepted || !path || !out || batch < 1 || n < 1 ||
      q_rows < 0 || q_rows > n || vocab < 1 || (n > 1 && (!q || q_rows < 1)))
    return VG_ERR_INVALID_ARG;
  if (n > kMaxNodes || vocab >= (int64_t(1) << 28) || batch >= (1 << 24)) return VG_ERR_UNSUPPORTED;
  if (!aligned16(p) || !aligned16(q)) return VG_ERR_ALIGNMENT;
  int sms = 0;
  if (vg_status s = device_sms(&sms)) return s;
  VerifyParams v;
  v.p = p;
  v.q = q;
  v.tokens = tokens;
  v.parents = parents;
  v.counts = counts;
  v.u = u;
  v.accepted = accepted;
  v.path = path;
  v.out = out;
  v.V = vocab;
  v.n = n;
  v.q_rows = q_rows;
  // Blocks a sequence: a power of two that fills the device twice over, up to 8
  // (48 trees over 151936 entries: 43 us with 8, 47 with 6, 50 with 4), and 16,
  // more than a portable cluster, for a few sequences (one: 10.7 us against
  // 12.4 with 8; 48: 57 us); each with a step of 128 entries a warp at least.
  int64_t c = 1;
  if (int64_t(batch) * 16 <= sms)
    c = kVerCluster;
  else
    while (c < 8 && c * batch < 2 * sms) c *= 2;
  c = std::max<int64_t>(1, std::min(c, vocab / (kVerWarps * 128)));
  const unsigned grid = unsigned(batch) * unsigned(c);
  void (*fn)(VerifyParams) = vocab % 4 ? &verify_kernel<false> : &verify_kernel<true>;
  static std::atomic<uint64_t> allowed[2];
  VG_CUDA(allow(fn, 0, allowed[vocab % 4 ? 0 : 1]));
  VG_CUDA(launch_clusters(fn, grid, kVerThreads, int(c), 0, as_cuda(stream), v));
  VG_LAUNCH_CHECK();
  return VG_OK;
}
