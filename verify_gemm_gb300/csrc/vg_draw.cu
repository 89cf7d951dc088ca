// vg_draw.cu -- vg_sample: draws from the softmax of logits with a temperature,
// truncated by top-k, top-p and min-p, from given random numbers.
//
// A row's tokens are ordered by logit, the largest first, equal ones by index.
// What a row keeps is a beginning of that order: at most k tokens, of these the
// fewest whose weights 2^-z, z = (max - x) log2 e / T, sum to p times theirs,
// of these the ones that weigh min_p and more.  So it is given by its last token:
// logit x_f, index i_f.  The token drawn is the first index whose running sum
// over what is kept exceeds u times the whole.
//
// Sums are integers, so that no order of addition changes what is kept or drawn, and weights are
// good to 2^-27.6 of themselves, rounded down to units of which V are 2^-28 of the largest or less: a draw
// is a comparison of u with the boundaries of 150000 tokens, and with sums good to 2^-22 one row in some
// hundred would end on the neighbour.
//
// A cluster of blocks a row; a block holds a run of it in shared memory, and
// each warp a run of that, so that the warps' order is the index order.  The
// last token is looked for in two steps: a histogram over z, 2048 bins of 1/64 of
// an octave, says in which bin it lies (of counts for top-k, of weights for
// top-p), and the tokens of that bin alone are sorted.  A top-k up to 200 goes without: all
// blocks know the largest logits of 256 groups of a row's threads, the k-th largest of those is
// at most the k-th largest of all, and the tokens down to it, few more than k, are sorted.
//
// What bounds it: for a few rows the exchanges between a cluster's blocks, some 1.7 us each (one row of
// 151936 BF16 logits, top-k 50 and top-p 0.95: 12.5 us, of which 3 to the largest, 3.5 to the list at the first block, 2 for its
// order and cut; top-p alone 28), and instructions that are fetched for the
// first time; for many rows, of some 45 instructions an element (issue 42 %), the
// barriers between steps of which the first block of a row does some alone.  256 rows with settings of
// their own 106 us (78 MB: 0.7 TB/s), 128 FP32 rows with their distributions 107 us (156 MB), 256 rows that
// all search for a top-p 218 us.
// (Two searches by codes alone, one level of bins after another, took 550 us and 1.7 ms: the
// bins of codes near zero are nearly empty and those of the body full.)
#include <algorithm>
#include <cmath>

#include "vg_rows.cuh"

namespace vg {
namespace {

constexpr int kDrawThreads = 512, kDrawWarps = kDrawThreads / 32;
constexpr int kBins = 2048;
constexpr int kDrawShare = 76 * 1024;         // bytes of a row a block should hold at most ...
constexpr int kDrawShareMax = 160 * 1024;     // ... and may
constexpr int kLocal = 1024, kSorted = 2048;  // tokens of a block, of the row, that a list holds
constexpr int kGroups = 256;                  // of which the largest logit is known to all blocks
static_assert(kMaxCluster * kDrawWarps == kGroups, "at least one group a warp");
// The largest top-k without a search: near 256 the groups' largest bound it badly, and the tokens to sort pass 512 and 1024.
// 138 rows of 151936 take 56 us at 200 and 78 at 201, 8 rows 22.7 at both; with a list up to 250, 138 rows of 250 would take
// 65 for 77, but 8 rows of 224 28 for 24 and of 248 35 for 24.
constexpr int kSmallK = 200;
constexpr int kListBytes = (kLocal + kSorted) * 8;   // (and the bins, which are read before a list is made)
static_assert(kListBytes >= 3 * kBins * 4, "room for the bins");

// A weight of 1 is 2^kOne and every weight is rounded down, so that the V of a row lose V 2^-kOne of the largest
// at most, 2^-28.  Rows of fewer than 2^18 tokens have sums of 64 bits, longer ones (kLong) of 96: there a pair of each thread of a
// warp, what a thread has of a row that is held, and a small top-k still sum to less than 2^64.  (151936
// tokens in 96 bits: 8 rows of top-p 44.6 us and not 40.8, 256 rows of mixed settings 110 and not 106.  2^27 tokens in 64
// bits left weights 35 of them: all that lay 35 octaves down, some 2^-9 of a row, was never drawn.)
using Wide = unsigned __int128;
constexpr int64_t kLongVocab = 1 << 18;
template <bool kLong>
using SumOf = std::conditional_t<kLong, Wide, uint64_t>;
template <bool kLong>
constexpr int kOne = kLong ? 56 : 46;
static_assert(kSmallK < 1 << 8 && kDrawShareMax / 2 / kDrawThreads < 1 << 8, "sums of 64 bits of weights of 2^56");

template <typename T>
struct alignas(2 * sizeof(T)) Pair {
  T x[2];
};
__device__ __forceinline__ float to_f(float x) { return x; }

struct DrawParams {
  const void *x;
  int64_t V, stride;
  const float *u, *temperature, *top_p, *min_p;
  const int32_t *top_k;
  int32_t *tokens;
  float *out;
  int draws, chunk;                  // units of a warp
  int rows;                          // at most one a thread, where those that take longest begin first
  int lead;                          // elements between the 16-byte border that x is and the first row
};

// 2^(30 - j / 64)
__constant__ uint32_t kPowers[64] = {
    1073741824, 1062175491, 1050733751, 1039415261, 1028218693, 1017142735, 1006186087, 995347464,
    984625594, 974019220, 963527098, 953147997, 942880699, 932724001, 922676710, 912737649,
    902905651, 893179563, 883558244, 874040567, 864625413, 855311680, 846098274, 836984114,
    827968132, 819049271, 810226483, 801498734, 792865000, 784324269, 775875538, 767517817,
    759250125, 751071493, 742980960, 734977579, 727060411, 719228525, 711481005, 703816941,
    696235434, 688735596, 681316545, 673977412, 666717336, 659535466, 652430958, 645402981,
    638450708, 631573326, 624770026, 618040012, 611382493, 604796689, 598281827, 591837143,
    585461881, 579155293, 572916640, 566745190, 560640218, 554601009, 548626854, 542717053};

// What a row's weights need: z in units of 1/64 is (top - h x) c, with top = h max.  h is a power of two: 1/4 for
// temperatures from 2^64 on, by which differences past FP32's range count, 2^64 for those below 2^-120, of which c = 64 log2 e
// / T itself is past it, and 1 for all others.
struct Scale {
  float top, minus;                  // minus: -h
  float c, c_low, cap;               // c as two floats; differences beyond cap weigh nothing
};
// A row's settings: read by its first block alone, as all blocks have to take the same way.
struct Settings {
  float temperature, top_p, min_p;
  int top_k;
  Scale scale;
  double min_at;                     // T ln(min_p)
};
static_assert(sizeof(Settings) == 48, "goes by 16 bytes");

// The weight of a finite logit x is w 2^(kOne - 30 - (bin >> 6)) (w some 2^30), rounded down.  With
// z = (k + r) / 64, k whole, |r| <= 1/2, it is 2^-(k / 64) from a table times
// 2^-(r / 64) by its series to the third power (the fourth is 2^-34).  What max - x loses in FP32 is carried along
// for FP32 logits.  It is exact for 16-bit ones but for those of less than 2^-16 (BF16) or 2^-13 (FP16) of the largest's
// magnitude, whose weights are off by up to 2^-24 (max - x) / T of themselves (carried along there, too: 256 mixed rows 111 us
// for 105).  The bin is k: the larger logit never has the larger one, as it goes by the rounded
// difference alone.
constexpr float kMagic = 12582912.f;           // 1.5 2^23: what is added to it is rounded to a whole number
constexpr int kMagicBits = 0x4B400000;
struct Weight {
  int w, k;
  __device__ __forceinline__ uint64_t value(int one) const { return uint64_t(uint32_t(w)) << (one - 30) >> min(k >> 6, 63); }
  __device__ __forceinline__ uint32_t bin() const { return min(uint32_t(k), uint32_t(kBins - 1)); }
  // w in the units of its bin: the last one has all weights below 2^-32
  __device__ __forceinline__ uint32_t in_bin() const { return uint32_t(w) >> min(max(k >> 6, 31) - 31, 31); }
};
// Of two logits at a time.
template <typename T>
__device__ __forceinline__ void weigh2(const Scale &s, const uint32_t *powers, float x0, float x1, Weight &w0, Weight &w1) {
  const float2 x = make_float2(x0, x1), minus = both(s.minus), all = fma2(x, minus, both(s.top));
  const float2 d = make_float2(fminf(all.x, s.cap), fminf(all.y, s.cap));
  float2 low = mul2(d, both(s.c_low));
  if constexpr (std::is_same_v<T, float>) {
    const float2 b = add2(all, both(-s.top)), c = add2(all, make_float2(-b.x, -b.y));
    const float2 e = add2(add2(both(s.top), make_float2(-c.x, -c.y)), fma2(x, minus, make_float2(-b.x, -b.y)));
    const float2 more = fma2(e, both(s.c), low);
    low = make_float2(all.x < s.cap ? more.x : low.x, all.y < s.cap ? more.y : low.y);
  }
  const float2 t = fma2(d, both(s.c), both(kMagic)), whole = add2(both(kMagic), make_float2(-t.x, -t.y));
  const float2 r = add2(fma2(d, both(s.c), whole), low);
  // 2^28 (2^-(r / 64) - 1)
  float2 q = fma2(r, both(-56.8362f), both(15743.4844f));
  q = fma2(r, q, both(-2907269.99f));
  q = fma2(r, q, both(kMagic));
  auto one = [&](Weight &w, float t, float q) {
    w.k = __float_as_int(t) - kMagicBits;
    const int p = int(powers[__float_as_int(t) & 63]);
    w.w = p + __mulhi(p, __float_as_int(q) * 16 - int(unsigned(kMagicBits) * 16u));
  };
  one(w0, t.x, q.x);
  one(w1, t.y, q.y);
}
// Its bin alone.
__device__ __forceinline__ uint32_t bin_of(const Scale &s, float x) {
  const float d = fminf(fmaf(x, s.minus, s.top), s.cap);
  return min(uint32_t(__float_as_int(fmaf(d, s.c, kMagic)) - kMagicBits), uint32_t(kBins - 1));
}

// Logits' codes in their order; logits of 16 bits have as many codes.
template <typename T>
constexpr int kCodeShift = std::is_same_v<T, float> ? 0 : std::is_same_v<T, __half> ? 13 : 16;
template <typename T>
__device__ __forceinline__ uint32_t code_of(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);           // (-0 is 0)
  return (b ^ (uint32_t(int32_t(b) >> 31) | 0x80000000u)) >> kCodeShift<T>;
}
template <typename T>
__device__ __forceinline__ float logit_of(uint32_t code) {
  uint32_t b = code << kCodeShift<T>;
  b = b & 0x80000000u ? b ^ 0x80000000u : ~(b | ((1u << kCodeShift<T>) - 1));
  return __uint_as_float(b);
}

// floor(a s) for 0 <= a < 1, and whether that is a s; s below 2^96
template <typename S>
__device__ __forceinline__ S part_of(float a, S s, bool &exact) {
  if (!(a > 0.f)) {
    exact = true;
    return 0;
  }
  const uint32_t b = __float_as_uint(a);
  const uint32_t e = b >> 23;
  const uint64_t m = e ? (b & 0x7FFFFF) | 0x800000 : b & 0x7FFFFF;
  const int right = 150 - int(e ? e : 1);      // a = m 2^-right, right >= 24
  if constexpr (sizeof(S) == 8) {
    const uint64_t lo = m * s, hi = __umul64hi(m, s);
    if (right >= 64) {
      exact = false;                           // (some bits are lost, or the product is 0)
      return right < 128 ? hi >> (right - 64) : 0;
    }
    exact = (lo & ((uint64_t(1) << right) - 1)) == 0;
    return hi << (64 - right) | lo >> right;
  } else {
    const Wide v = s * m, whole = right < 128 ? v >> right : Wide(0);
    exact = right < 128 && whole << right == v;
    return whole;
  }
}
// How many of weight w it takes to weigh `target`, if not more than 2^29.
template <typename S>
__device__ __forceinline__ uint64_t count_for(S target, uint64_t w) {
  uint32_t fewer = 0;                            // these weigh less
#pragma unroll 1
  for (uint32_t bit = 1u << 28; bit; bit /= 2)
    if (Wide(fewer | bit) * w < target) fewer |= bit;
  return target == 0 ? 0 : fewer + 1;
}

__device__ __forceinline__ uint64_t shuffle_up(uint64_t v, int lanes) { return __shfl_up_sync(~0u, v, lanes); }
__device__ __forceinline__ Wide shuffle_up(Wide v, int lanes) {
  return Wide(__shfl_up_sync(~0u, uint32_t(v >> 64), lanes)) << 64 | __shfl_up_sync(~0u, uint64_t(v), lanes);
}
template <typename S>
__device__ __forceinline__ S scan_up(S v, int lane) {
#pragma unroll
  for (int w = 1; w < 32; w *= 2) {
    const S y = shuffle_up(v, w);
    if (lane >= w) v += y;
  }
  return v;
}
// The sum of a warp, by 27 bits at a time.
template <typename S, typename V>
__device__ __forceinline__ S warp_sum(V v) {
  constexpr uint32_t k27 = (1u << 27) - 1;
  S sum = __reduce_add_sync(~0u, uint32_t(v) & k27) + (S(__reduce_add_sync(~0u, uint32_t(v >> 27) & k27)) << 27);
  if constexpr (sizeof(V) == 8) {
    sum += S(__reduce_add_sync(~0u, uint32_t(v >> 54))) << 54;
  } else {
    sum += S(__reduce_add_sync(~0u, uint32_t(v >> 54) & k27)) << 54;
    sum += S(__reduce_add_sync(~0u, uint32_t(v >> 81))) << 81;
  }
  return sum;
}
// A sum as two words.
__device__ __forceinline__ uint64_t upper(uint64_t) { return 0; }
__device__ __forceinline__ uint64_t upper(Wide v) { return uint64_t(v >> 64); }
template <typename S>
__device__ __forceinline__ S sum_of(const ulonglong2 &v) {
  if constexpr (sizeof(S) == 8) return v.x;
  else return Wide(v.y) << 64 | v.x;
}

// Sorts n (a power of two, at least 64) entries, the smallest first; the whole block.
// A thread holds entries 2 t and 2 t + 1 of every 1024: exchanges within a warp's 64
// entries go by shuffles, the others by shared memory.
__device__ __forceinline__ uint64_t other(uint64_t v, int lanes) { return __shfl_xor_sync(~0u, v, lanes); }
__device__ __forceinline__ Wide other(Wide v, int lanes) {
  return Wide(__shfl_xor_sync(~0u, uint32_t(v >> 64), lanes)) << 64 | __shfl_xor_sync(~0u, uint64_t(v), lanes);
}
__device__ __forceinline__ void sort_up(uint64_t *v, int n) {
#pragma unroll 1
  for (int size = 64; size <= n; size *= 2) {
#pragma unroll 1
    for (int stride = size / 2; stride >= 64; stride /= 2) {
      __syncthreads();
      for (int q = threadIdx.x; q < n / 2; q += kDrawThreads) {
        const int a = 2 * q - (q & (stride - 1)), b = a + stride;
        const uint64_t x = v[a], y = v[b];
        if ((x > y) == ((a & size) == 0)) {
          v[a] = y;
          v[b] = x;
        }
      }
    }
    __syncthreads();
    for (int at = 2 * int(threadIdx.x); at < n; at += 2 * kDrawThreads) {   // (whole warps)
      uint64_t a = v[at], b = v[at + 1];
      // the first time all sizes up to 64, then this one's last strides
#pragma unroll 1
      for (int inner = size == 64 ? 2 : size; inner <= size; inner *= 2) {
        const bool up = (at & inner) == 0;
#pragma unroll 1
        for (int lanes = min(inner, 64) / 4; lanes; lanes /= 2) {
          const uint64_t x = other(a, lanes), y = other(b, lanes);
          const bool small = ((threadIdx.x & lanes) == 0) == up;
          a = (x < a) == small ? x : a;
          b = (y < b) == small ? y : b;
        }
        const uint64_t x = a < b ? a : b, y = a < b ? b : a;
        a = up ? x : y;
        b = up ? y : x;
      }
      v[at] = a;
      v[at + 1] = b;
    }
  }
  __syncthreads();
}

// What the first block of a row tells the others.
template <typename S>
struct alignas(16) Found {
  uint32_t bin, code;                // the last token's bin; its logit
  int32_t index, state;              // its index
  S target, whole;                   // the count or weight wanted of the bin; the weight of what is kept
  float from, to;                    // the bin's logits
};
enum { kGo = 0, kAll = 1, kTooMany = 2 };      // state; kAll: nothing is left out
// Where a search by codes is: codes [lo, hi], bins of 2^shift of them from hi down, the last
// bin with all that is below; what is wanted of them.
template <typename S>
struct Search {
  uint32_t hi, lo;
  int shift, done;                   // 1: hi is the code, 2: there are fewer
  S target;
  uint64_t ties;                     // how many of the code
};
__device__ __forceinline__ int shift_for(uint32_t span) {
  // the smallest with span >> shift below the last bin
  int s = max(0, 21 - __clz(int(span | 1)));
  return (span >> s) < kBins - 1 ? s : s + 1;
}

template <typename T, bool kHeld, bool kOrdered, bool kLong>
__global__ void __launch_bounds__(kDrawThreads, 2) sample_kernel(const __grid_constant__ DrawParams p) {
  using Sum = SumOf<kLong>;
  using Found = vg::Found<Sum>;
  using Search = vg::Search<Sum>;
  constexpr int kOne = vg::kOne<kLong>;
  extern __shared__ __align__(16) uint8_t draw_smem[];
  __shared__ float tops[kGroups];
  __shared__ __align__(16) ulonglong2 sums[kMaxCluster * kDrawWarps];
  __shared__ __align__(16) Found told;
  __shared__ __align__(16) ulonglong2 shares[kMaxCluster];
  __shared__ uint32_t powers[64];
  __shared__ __align__(16) Settings settings;
  __shared__ Sum scan[kDrawWarps];
  __shared__ uint32_t listed;
  __shared__ int n_keep;
  __shared__ float list_floor;
  __shared__ uint64_t weights[kSmallK];
  uint32_t *bin_lo = reinterpret_cast<uint32_t *>(draw_smem), *bin_hi = bin_lo + kBins, *bin_top = bin_hi + kBins;
  uint64_t *local = reinterpret_cast<uint64_t *>(draw_smem), *list = local + kLocal;
  uint4 *held = reinterpret_cast<uint4 *>(draw_smem + kListBytes);
  const uint32_t rank = cluster_rank(), blocks = cluster_size();
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  int64_t row = blockIdx.x / blocks;
  if constexpr (kOrdered) {
    // The rows with a search over the bins before those without.  (The blocks of a row whose settings
    // change meanwhile may see other orders: each still has a row, and the first's settings.)
    bool slow = false;
    if (tid < p.rows) {
      const int k = p.top_k ? p.top_k[tid] : 0;
      const float q = p.top_p ? p.top_p[tid] : 1.f, t = p.temperature ? p.temperature[tid] : 1.f;
      slow = t > 0.f && (k > kSmallK || (k <= 0 && q > 0.f && q < 1.f));
    }
    const uint32_t those = __ballot_sync(~0u, slow);
    if (lane == 0) scan[warp] = __popc(those);
    __syncthreads();
    const int count = lane < kDrawWarps ? int(scan[lane]) : 0;
    const int before = __reduce_add_sync(~0u, lane < warp ? count : 0) + __popc(those & ((1u << lane) - 1));
    const int all = __reduce_add_sync(~0u, count), place = slow ? before : all + tid - before;
    if (place == int(row)) n_keep = tid;
    __syncthreads();
    row = n_keep;
  }
  const T *x = static_cast<const T *>(p.x);
  const int64_t lo = p.lead + row * p.stride, hi = lo + p.V;
  const int64_t end = (hi + 7) / 8;                      // units, on the grid of 16-byte borders
  const int64_t w0 = lo / 8 + int64_t(rank * kDrawWarps + warp) * p.chunk;
  const int mine = int(max(int64_t(0), min(int64_t(p.chunk), end - w0)));   // units of this warp
  if (blocks > 1) cluster_arrive();                      // a block must have begun before others write to it
  uint4 *run = held + int64_t(warp) * p.chunk * (sizeof(T) / 2);
  if constexpr (kHeld) {
    constexpr int kEach = 16 / sizeof(T);                // logits of a 16-byte piece
    for (int i = lane; i < mine * int(sizeof(T) / 2); i += 32) {
      const int64_t e = w0 * 8 + i * kEach;
      if (e >= lo && e + kEach <= hi) {
        copy16(run + i, x + e);
      } else {
        T t[kEach];
#pragma unroll
        for (int k = 0; k < kEach; ++k) t[k] = e + k >= lo && e + k < hi ? x[e + k] : T(-INFINITY);
        memcpy(run + i, t, 16);
      }
    }
  }
  if (warp == 0) {
    powers[lane] = kPowers[lane];
    powers[lane + 32] = kPowers[lane + 32];
    if (lane == 0) {
      listed = 0;
      if (rank == 0) {
        Settings now{};
        now.temperature = p.temperature ? p.temperature[row] : 1.f;
        now.top_p = p.top_p ? p.top_p[row] : 1.f;
        now.min_p = p.min_p ? p.min_p[row] : 0.f;
        now.top_k = p.top_k ? p.top_k[row] : 0;
        const float h = now.temperature >= 0x1p64f ? 0.25f : now.temperature < 0x1p-120f ? 0x1p64f : 1.f;
        const double c = 64 * 1.4426950408889634074 / double(now.temperature) / double(h);
        now.scale.minus = -h;
        now.scale.c = float(c);
        now.scale.c_low = float(c - double(now.scale.c));
        now.scale.cap = fminf(4096.f / now.scale.c, 3.4028234e38f);
        // (over an infinite temperature every finite logit weighs 1)
        now.min_at = !(now.min_p > 0.f)              ? 0.0
                     : now.temperature == INFINITY ? (now.min_p > 1.f ? 1e300 : -1e300)
                                                   : double(now.temperature) * log(double(now.min_p));
        settings = now;
      }
    }
  }
  if constexpr (kHeld) {
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncwarp();                                        // a warp reads only what it copied
  }
  const int64_t base = w0 * 8 - lo;                      // index of the warp's first element in the row
  // logits 2 j and 2 j + 1 of the warp's run as they came, -infinity beside the row
  auto pair_at = [&](int j) {
    if constexpr (kHeld) {
      return reinterpret_cast<const Pair<T> *>(run)[j];
    } else {
      Pair<T> v;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int64_t e = w0 * 8 + 2 * j + k;
        v.x[k] = e >= lo && e < hi ? x[e] : T(-INFINITY);
      }
      return v;
    }
  };
  auto unit_at = [&](int i) {
    Unit<T> v;
#pragma unroll
    for (int k = 0; k < int(sizeof(T) / 2); ++k) v.w[k] = run[i * int(sizeof(T) / 2) + k];
    return v;
  };
  // f(index of the first, two logits), over the warp's run; all lanes come along.
  // (Two at a time, and not the eight of a 16-byte piece: a row passes here but a
  // few times, and what the code of eight takes to be fetched is more than it saves.)
  auto each = [&](auto &&f) {
    const int count = mine * 4;
    int j0 = 0;
#pragma unroll 2
    for (; j0 + 32 <= count; j0 += 32) {
      const Pair<T> v = pair_at(j0 + lane);
      f(int(base) + 2 * (j0 + lane), to_f(v.x[0]), to_f(v.x[1]));
    }
    if (j0 < count) {
      const int j = j0 + lane;
      float a = -INFINITY, b = -INFINITY;
      if (j < count) {
        const Pair<T> v = pair_at(j);
        a = to_f(v.x[0]);
        b = to_f(v.x[1]);
      }
      f(int(base) + 2 * j, a, b);
    }
  };
  auto sync_all = [&] {
    if (blocks > 1) cluster_sync();
    else __syncthreads();
  };

  // ------------------------------------------------------------- the largest
  // Of each of 256 groups of threads: 16 / blocks in each warp.  All blocks get them all.
  float m = -INFINITY;
  if (kHeld && mine >= 32) {                             // (every thread has a unit)
    Largest<T> largest;
    for (int i = lane; i < mine; i += 32) largest.take(unit_at(i));
    m = largest.value();
  } else {
    for (int j = lane; j < mine * 4; j += 32) {
      const Pair<T> v = pair_at(j);
      m = max_nan(m, max_nan(to_f(v.x[0]), to_f(v.x[1])));
    }
  }
  const int groups = kGroups / kDrawWarps / int(blocks), wide = 32 / groups;
  for (int w = wide / 2; w; w /= 2) m = max_nan(m, __shfl_xor_sync(~0u, m, w));
  {
    const float v = __shfl_sync(~0u, m, lane % groups * wide);
    if (blocks > 1) cluster_wait();
    if (lane < kGroups / kDrawWarps) {
      float *to = tops + (rank * kDrawWarps + warp) * groups + lane % groups;
      asm volatile("{ .reg .b32 at; mapa.shared::cluster.u32 at, %0, %1; st.shared::cluster.f32 [at], %2; }" ::"r"(
                       static_cast<uint32_t>(__cvta_generic_to_shared(to))),
                   "r"(lane / groups), "f"(v)
                   : "memory");
    }
    if (rank == 0 && warp == 0) {
      __syncwarp();
      const uint64_t *from = reinterpret_cast<const uint64_t *>(&settings);
      if (lane && lane < int(blocks))
#pragma unroll
        for (int k = 0; k < int(sizeof(Settings) / 16); ++k)
          cluster_store(reinterpret_cast<ulonglong2 *>(&settings) + k, lane, from[2 * k], from[2 * k + 1]);
    }
  }
  sync_all();
  const float temperature = settings.temperature, top_p = settings.top_p, min_p = settings.min_p;
  const int top_k = settings.top_k;
  const int entries = int(blocks) * kDrawWarps, me = int(rank) * kDrawWarps + warp;
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < kGroups / 32; ++i) top = max_nan(top, tops[i * 32 + lane]);
#pragma unroll
  for (int w = 16; w; w /= 2) top = max_nan(top, __shfl_xor_sync(~0u, top, w));
  top += 0.f;
  float *out = p.out ? p.out + row * p.V : nullptr;
  // no token: a NaN, an infinity that weighs all, nothing but -infinity
  const bool cold = temperature <= 0.f;
  const bool bad = isnan(top) || isnan(temperature) || (top == INFINITY && !cold);
  if (bad || top == -INFINITY) {
    if (rank == 0)
      for (int i = tid; i < p.draws; i += kDrawThreads) p.tokens[row * p.draws + i] = -1;
    if (out) {
      const float v = bad && !cold ? __int_as_float(0x7FFFFFFF) : 0.f;
      for (int64_t i = rank * kDrawThreads + tid; i < p.V; i += int64_t(blocks) * kDrawThreads) out[i] = v;
    }
    return;
  }
  // stores the probabilities of elements r and r + 1
  const bool aligned = (reinterpret_cast<uintptr_t>(out + base) & 7) == 0;
  auto store = [&](int r, float a, float b) {
    if (aligned && r >= 0 && r + 2 <= p.V && r - int(base) < mine * 8) {
      __stcs(reinterpret_cast<float2 *>(out + r), make_float2(a, b));
    } else if (r - int(base) < mine * 8) {
      if (r >= 0 && r < p.V) out[r] = a;
      if (r + 1 >= 0 && r + 1 < p.V) out[r + 1] = b;
    }
  };

  // ---------------------------------------------------- the first largest alone
  if (cold || top_k == 1 || top_p <= 0.f || min_p > 1.f) {
    int first = INT32_MAX;
    each([&](int r, float a, float b) {
      if (b == top) first = min(first, r + 1);
      if (a == top) first = min(first, r);
    });
    first = __reduce_min_sync(~0u, first);
    if (lane < int(blocks)) cluster_store(&sums[rank * kDrawWarps + warp], lane, uint32_t(first), 0);
    sync_all();
    first = INT32_MAX;
    for (int i = lane; i < entries; i += 32) first = min(first, int(sums[i].x));
    first = __reduce_min_sync(~0u, first);
    if (rank == 0)
      for (int i = tid; i < p.draws; i += kDrawThreads) p.tokens[row * p.draws + i] = first;
    if (out)
      each([&](int r, float, float) { store(r, r == first ? 1.f : 0.f, r + 1 == first ? 1.f : 0.f); });
    return;
  }
  Scale scale = settings.scale;
  if (scale.minus < -1.f && fabsf(top) >= 0x1p60f) {       // 2^64 top would be past the range; what lies below it weighs nothing
    scale.minus = -1.f;
    scale.c = 0x1.fffffep127f;
    scale.c_low = 0.f;
    scale.cap = 4096.f / scale.c;
  }
  scale.top = -scale.minus * top;
  // What a draw's running sum has to exceed, of `all`.
  auto drawn = [&](int d, auto all) {
    const float u = p.u[row * p.draws + d];
    bool exact;
    return u >= 1.f ? all - 1 : part_of(u, all, exact);
  };
  auto weigh = [&](float y) {
    Weight a, b;
    weigh2<T>(scale, powers, y, y, a, b);
    return a.value(kOne);
  };

  // What is kept: y > x_f, and those equal to it up to index i_f.
  // (Elements beside the row, -infinity, have indices below 0.)
  float x_f = -INFINITY;
  int i_f = INT32_MIN;
  auto kept = [&](float y, int index) {
    bool k = y > x_f;
    if (i_f >= 0) k |= y == x_f && index <= i_f;
    return k;
  };
  // The block's 512 threads' sums of `v`, up to each and in all.
  auto scan_block = [&](auto v, Sum &whole) {
    const Sum in_warp = scan_up(v, lane);
    __syncthreads();                                     // (scan has been read)
    if (lane == 31) scan[warp] = in_warp;
    __syncthreads();
    Sum run = in_warp;
    whole = 0;
#pragma unroll
    for (int w = 0; w < kDrawWarps; ++w) {
      if (w < warp) run += scan[w];
      whole += scan[w];
    }
    return run;
  };
  // The warps' weights of what is kept, for all blocks.
  using Mass = SumOf<kLong && !kHeld>;
  auto tell_mass = [&](Mass mass) {
    const Sum sum = warp_sum<Sum>(mass);
    if (lane < int(blocks)) cluster_store(&sums[me], lane, uint64_t(sum), upper(sum));
  };
  // Tells the other blocks what this one has put into `what`.
  auto tell = [&](auto *what) {
    static_assert(sizeof(*what) % 16 == 0, "goes by 16 bytes");
    __syncthreads();
    if (tid < int(blocks) && tid != int(rank)) {
      const uint64_t *from = reinterpret_cast<const uint64_t *>(what);
#pragma unroll
      for (int k = 0; k < int(sizeof(*what) / 16); ++k)
        cluster_store(reinterpret_cast<ulonglong2 *>(what) + k, uint32_t(tid), from[2 * k], from[2 * k + 1]);
    }
  };
  // Which bin the running sum over all blocks' bins reaches the target in (0: of top_p of the
  // whole and `beyond`).  kOf: of counts, of weights in the bins' units, of weights.  A block
  // adds up a share of the bins, four a lane, one block's a lane, and the block whose share holds the
  // target tells the others.  (One block that took all bins of 16 blocks was at it for 5 us.)
  enum { kCounts, kScaled, kWeights };
  auto find = [&](auto of, Sum target, Sum beyond) {
    constexpr int kOf = decltype(of)::value, kWords = kOf == kCounts ? 1 : kOf == kWeights && kLong ? 3 : 2;
    using Bin = SumOf<kWords == 3>;
    using Part = SumOf<kLong && kOf != kCounts>;
    sync_all();
    const int quad = warp * (32 / int(blocks)) + lane / int(blocks), share = kBins / int(blocks);
    const uint32_t bin0 = rank * share + quad * 4;
    const uint32_t here = static_cast<uint32_t>(__cvta_generic_to_shared(bin_lo + bin0));
    Bin bin[4] = {};
#pragma unroll
    for (int k = 0; k < kWords; ++k) {
      uint32_t w[4];
      asm volatile("{ .reg .b32 at; mapa.shared::cluster.u32 at, %4, %5; ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [at]; }"
                   : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                   : "r"(here + k * kBins * 4), "r"(lane % blocks)
                   : "memory");
#pragma unroll
      for (int i = 0; i < 4; ++i) bin[i] |= Bin(w[i]) << (32 * k);
    }
    for (uint32_t w = 1; w < blocks; w *= 2)
#pragma unroll
      for (int k = 0; k < 4; ++k) bin[k] += other(bin[k], int(w));
    Part v[4], sum = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[k] = bin[k];
      if constexpr (kOf == kScaled) v[k] = v[k] << (kOne - 30) >> (bin0 >> 6);
      sum += v[k];
    }
    const bool counts = lane % blocks == 0;              // (all lanes of a quad have its sums)
    Sum mine_all, run = scan_block(counts ? sum : Part(0), mine_all), whole = 0;
    if (blocks > 1) {
      if (tid < int(blocks)) cluster_store(&shares[rank], uint32_t(tid), uint64_t(mine_all), upper(mine_all));
      sync_all();
      for (uint32_t r = 0; r < blocks; ++r) {
        const Sum part = sum_of<Sum>(shares[r]);
        if (r < rank) run += part;
        whole += part;
      }
    } else {
      whole = mine_all;
    }
    Found f{};
    f.whole = whole;
    if (target == 0) {
      bool exact;
      target = part_of(top_p, whole + beyond, exact);
      if (!exact || target == 0) ++target;
    }
    if (target > whole) {
      f.state = kAll;
      f.target = target - whole;
      sync_all();                                        // (the shares are read before they are written again)
      return f;
    }
    Sum before = run - sum;
    const bool it = counts && before < target && target <= run;
    if (it) {
      uint32_t k0 = 0;
#pragma unroll
      for (uint32_t k = 0; k < 3; ++k)
        if (k0 == k && before + v[k] < target) {
          before += v[k];
          ++k0;
        }
      f.bin = bin0 + k0;
      f.state = kGo;
      f.target = target - before;
      told = f;
    }
    if (__syncthreads_or(it)) {
      // the bin's logits, [from, to): the smallest code whose bin is at most this, and the one before
      if (warp < 2) {
        const uint32_t bin = told.bin - warp;
        uint32_t lo = code_of<float>(-INFINITY), hi = code_of<float>(top) + 1;   // not so; so, or top's next
#pragma unroll 1
        while (hi - lo > 1) {                          // 32 codes between at a time
          const uint32_t step = (hi - lo) / 33 + 1, code = min(hi, lo + uint32_t(lane + 1) * step);
          const uint32_t so = __ballot_sync(~0u, code == hi || bin_of(scale, logit_of<float>(code)) <= bin);
          const uint32_t n = so ? uint32_t(__ffs(int(so)) - 1) : 32;
          hi = min(hi, lo + (n + 1) * step);
          lo = lo + n * step;
        }
        const bool none = warp && told.bin == 0;
        if (lane == 0) (warp ? told.to : told.from) = none ? INFINITY : logit_of<float>(hi);
      }
      tell(&told);
    }
    sync_all();
    return told;
  };
  auto clear_bins = [&](int words) {
    for (int i = tid; i < words * kBins; i += kDrawThreads) bin_lo[i] = 0;
    if (tid == 0) listed = 0;
    __syncthreads();
  };
  // Those of two tokens that `wanted` says go to the block's list; the first block's `list` then has
  // all of the row's in order, and how many there are.
  uint64_t *const to_list = blocks == 1 ? list : local;
  const uint32_t room = blocks == 1 ? kSorted : kLocal;
  auto push = [&](float a, float b, int r, auto &&wanted) {
    const bool wa = wanted(a, r), wb = wanted(b, r + 1);
    if (wa || wb) {
      uint32_t at = atomicAdd(&listed, uint32_t(wa) + uint32_t(wb));
      if (wa && at < room) to_list[at] = uint64_t(~code_of<float>(a)) << 32 | uint32_t(r);
      at += wa;
      if (wb && at < room) to_list[at] = uint64_t(~code_of<float>(b)) << 32 | uint32_t(r + 1);
    }
  };
  auto count_list = [&](uint32_t &mine_n, uint32_t &mine_at) {   // lane r: block r's; -1: too many
    const uint32_t count_at = static_cast<uint32_t>(__cvta_generic_to_shared(&listed));
    mine_n = 0;
    if (lane < int(blocks))
      asm volatile("{ .reg .b32 at; mapa.shared::cluster.u32 at, %1, %2; ld.shared::cluster.u32 %0, [at]; }"
                   : "=r"(mine_n)
                   : "r"(count_at), "r"(lane)
                   : "memory");
    mine_at = uint32_t(scan_up(uint64_t(mine_n), lane)) - mine_n;
    const uint32_t n = __shfl_sync(~0u, mine_at + mine_n, 31);
    return n > kSorted || __any_sync(~0u, mine_n > room) ? -1 : int(n);
  };
  auto pad_list = [&](int n) {
    int size = 64;
    while (size < n) size *= 2;
    for (int i = n + tid; i < size; i += kDrawThreads) list[i] = ~uint64_t(0);
    __syncthreads();
  };
  auto gather_list = [&] {
    uint32_t mine_at, mine_n;
    const int n = count_list(mine_n, mine_at);
    if (n < 0) return -1;
    const uint32_t list_at = static_cast<uint32_t>(__cvta_generic_to_shared(local));
    if (blocks > 1) {                                    // a warp, or several, for each block
      const uint32_t share = kDrawWarps / blocks, r = warp / share;
      const uint32_t count = __shfl_sync(~0u, mine_n, r), to = __shfl_sync(~0u, mine_at, r);
      for (uint32_t i = warp % share * 32 + lane; i < count; i += share * 32) {
        uint64_t v;
        asm volatile("{ .reg .b32 at; mapa.shared::cluster.u32 at, %1, %2; ld.shared::cluster.u64 %0, [at]; }"
                     : "=l"(v)
                     : "r"(list_at + i * 8), "r"(r)
                     : "memory");
        list[to + i] = v;
      }
    }
    pad_list(n);
    return n;
  };
  auto sort_list = [&](int n, auto short_too) {
    int size = 64;
    while (size < n) size *= 2;
    if (!decltype(short_too)::value || size > 256) {
      sort_up(list, size);
      return;
    }
    // a short one, all different: each goes to where as many are before it, counted by 512 / size threads
    const int parts = kDrawThreads / size, i = tid / parts;
    const uint64_t v = i < n ? list[i] : 0;
    int before = 0;
#pragma unroll 4
    for (int j = tid % parts; j < n; j += parts) before += list[j] < v;
    for (int w = 1; w < parts; w *= 2) before += __shfl_xor_sync(~0u, before, w);
    __syncthreads();
    if (i < n && tid % parts == 0) list[before] = v;
    __syncthreads();
  };
  auto logit_at = [&](uint64_t e) { return logit_of<float>(~uint32_t(e >> 32)); };
  // The smallest logit that weighs min_p.
  const float f_min = min_p > 0.f ? fminf(__double2float_ru(double(top) + settings.min_at), top) : -INFINITY;
  // In the sorted list of n: how many are kept, with the target of what is before and in it
  // (limit: of tokens; target 0: no limit of weight).  Every thread has up to four entries.
  auto cut_list = [&](int n, int limit, Sum target, bool of_list) {
    uint64_t v[4], sum = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int i = tid * 4 + k;
      v[k] = i < min(n, limit) ? weigh(logit_at(list[i])) : 0;
      sum += v[k];
    }
    Sum whole, run = scan_block(sum, whole) - sum;
    if (of_list && top_p < 1.f) {
      bool exact;
      target = part_of(top_p, whole, exact);
      if (!exact || target == 0) ++target;
    }
    if (tid == 0) n_keep = 0;
    __syncthreads();
    int last = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int i = tid * 4 + k;
      if (i < min(n, limit) && (target == 0 || run < target) && logit_at(list[i]) >= f_min) last = i + 1;
      run += v[k];
    }
    if (last) atomicMax(&n_keep, last);
    __syncthreads();
  };
  bool too_many = false, done = false, summed = false;
  Sum whole = 0;
  if (top_k > 0 && top_k <= kSmallK && top_k < p.V) {
    // ----------------------------------------------------------- a small top-k
    // the upper 16 bits of the code of the top_k-th largest of the groups' largest, by one warp: the
    // others leave their turns to another row's block (186 rows of top-k 50: 46.7 us, all warps at it 49.4)
    if (warp == 0) {
      uint32_t code[kGroups / 32], least = 0;
#pragma unroll
      for (int i = 0; i < kGroups / 32; ++i) code[i] = code_of<float>(tops[i * 32 + lane]);
#pragma unroll 1
      for (uint32_t bit = 1u << 31; bit >= 1u << 16; bit /= 2) {
        uint32_t n = 0;
#pragma unroll
        for (int i = 0; i < kGroups / 32; ++i) n += code[i] >= (least | bit);
        if (int(__reduce_add_sync(~0u, n)) >= top_k) least |= bit;
      }
      if (lane == 0) list_floor = least > code_of<float>(-INFINITY) ? logit_of<float>(least) : -3.4028234e38f;
    }
    __syncthreads();
    const float floor = list_floor;
    if (kHeld && mine >= 32) {
      // (few units of eight have a logit that is wanted)
      for (int i = lane; i < mine; i += 32) {
        Largest<T> largest;
        largest.take(unit_at(i));
        if (!(largest.value() >= floor)) continue;
#pragma unroll 1
        for (int j = 4 * i; j < 4 * i + 4; ++j) {
          const Pair<T> v = pair_at(j);
          push(to_f(v.x[0]), to_f(v.x[1]), int(base) + 2 * j, [&](float y, int) { return y >= floor; });
        }
      }
    } else {
      each([&](int r, float a, float b) { push(a, b, r, [&](float y, int) { return y >= floor; }); });
    }
    // All blocks tell their counts, and those with few give the first their tokens, a place of its own
    // each, before they meet (fetched by it afterwards: a microsecond more).
    __syncthreads();
    const uint32_t few = kSorted / blocks, my_count = listed;
    if (tid < int(blocks)) cluster_store(&shares[rank], uint32_t(tid), my_count, 0);
    if (blocks > 1 && my_count <= few)
      for (uint32_t i = tid; i < my_count; i += kDrawThreads) {
        const uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(list + rank * few + i));
        asm volatile("{ .reg .b32 at; mapa.shared::cluster.u32 at, %0, 0; st.shared::cluster.u64 [at], %1; }" ::"r"(at),
                     "l"(local[i])
                     : "memory");
      }
    sync_all();
    const uint32_t count = lane < int(blocks) ? uint32_t(shares[lane].x) : 0;
    const int in_all = __reduce_add_sync(~0u, int(min(count, uint32_t(kSorted + 1))));
    const bool given = !__any_sync(~0u, count > few);
    too_many = in_all > kSorted || __any_sync(~0u, count > room);
    if (too_many) {
      sync_all();                                        // (the counts stay until all have read them)
    } else {
      // without a distribution the other blocks end when the first has their lists
      if (!out && rank) {
        if (!given) {
          cluster_arrive();
          cluster_wait();
        }
        return;
      }
      if (rank == 0) {
        int n = in_all;
        if (given && blocks > 1) {
          constexpr int kEach = kSorted / kDrawThreads;  // of a block's place, by the threads that are its own
          const uint32_t threads = kDrawThreads / blocks, r = uint32_t(tid) / threads, i0 = uint32_t(tid) % threads;
          const uint32_t there = __shfl_sync(~0u, count, int(r));
          const uint32_t to = __shfl_sync(~0u, uint32_t(scan_up(uint64_t(count), lane)) - count, int(r));
          uint64_t v[kEach];
#pragma unroll
          for (int k = 0; k < kEach; ++k)
            if (i0 + k * threads < there) v[k] = list[r * few + i0 + k * threads];
          __syncthreads();
#pragma unroll
          for (int k = 0; k < kEach; ++k)
            if (i0 + k * threads < there) list[to + i0 + k * threads] = v[k];
          pad_list(n);
        } else {
          n = gather_list();
          if (!out && blocks > 1) cluster_arrive();
        }
        sort_list(n, std::true_type{});
        cut_list(n, top_k, 0, true);
        const int keep = n_keep;
        // in the order of the indices: each token's sum before it
        uint64_t w = 0, before = 0, all = 0;
        const uint32_t index = tid < keep ? uint32_t(list[tid]) : 0;
        if (tid < keep) weights[tid] = w = weigh(logit_at(list[tid]));
        __syncthreads();
        if (warp * 32 < keep)
          for (int i = 0; i < keep; ++i) {
            const uint64_t v = weights[i];
            all += v;
            if (uint32_t(list[i]) < index) before += v;
          }
        for (int d = 0; d < p.draws; ++d) {
          const uint64_t want = drawn(d, all);
          if (tid < keep && want >= before && want < before + w) p.tokens[row * p.draws + d] = int32_t(index);
        }
        if (!out) {
          if (!given) cluster_wait();
          return;
        }
        if (tid == 0) {
          const uint64_t e = list[keep - 1];
          told = Found{0, ~uint32_t(e >> 32), int32_t(uint32_t(e)), kGo, 0, all, 0.f, 0.f};
        }
        tell(&told);
      }
      sync_all();
      done = true;
      x_f = logit_of<float>(told.code);
      i_f = told.index;
      whole = told.whole;
    }
  } else {
    // A round: the last token by counts (kMass: weights) among what is kept so far.
    auto round = [&](auto by_weight, Sum target) {
      constexpr bool kMass = decltype(by_weight)::value;
      clear_bins(2);
      each([&](int r, float y0, float y1) {
        const bool k0 = kept(y0, r), k1 = kept(y1, r + 1);
        if constexpr (kMass) {
          if (!k0 && !k1) return;
          Weight w[2];
          weigh2<T>(scale, powers, y0, y1, w[0], w[1]);
          auto add = [&](const Weight &w) {
            const uint32_t b = w.bin(), low = w.in_bin();
            if (atomicAdd(bin_lo + b, low) + low < low) atomicAdd(bin_hi + b, 1u);
          };
          if (k0) add(w[0]);
          if (k1) add(w[1]);
        } else {
          if (k0) atomicAdd(bin_lo + bin_of(scale, y0), 1u);
          if (k1) atomicAdd(bin_lo + bin_of(scale, y1), 1u);
        }
      });
      const Found f = find(std::integral_constant<int, kMass ? kScaled : kCounts>{}, target, 0);
      if (f.state == kAll) return;
      if (kMass && f_min >= f.to) return;                // min-p ends it before
      // kMass: what lies in the bins before is kept, and is weighed on the way
      Mass mass = 0;
      each([&](int r, float a, float b) {
        if constexpr (kMass) {
          const bool ka = a >= f.to, kb = b >= f.to;
          if (ka || kb) {
            Weight wa, wb;
            weigh2<T>(scale, powers, a, b, wa, wb);
            mass += (ka ? wa.value(kOne) : 0) + (kb ? wb.value(kOne) : 0);
          }
        }
        push(a, b, r, [&](float y, int i) { return y >= f.from && y < f.to && kept(y, i); });
      });
      if constexpr (kMass) tell_mass(mass);
      sync_all();
      if (rank == 0) {
        const int n = gather_list();
        if (n >= 0) {
          sort_list(n, std::false_type{});
          if constexpr (kMass) cut_list(n, n, f.target, false);
          else if (tid == 0) n_keep = int(f.target);
          __syncthreads();
          if constexpr (kMass) {
            // each kept token's weight to the sum of the warp that has it, and the sums to the other blocks
            for (int i = tid; i < n_keep; i += kDrawThreads) {
              const uint32_t warp_of = (uint32_t(list[i]) + uint32_t(lo & 7)) / uint32_t(8 * p.chunk);
              const uint64_t w = weigh(logit_at(list[i]));
              const uint64_t low = atomicAdd(reinterpret_cast<unsigned long long *>(&sums[warp_of].x), w) + w;
              if (kLong && low < w) atomicAdd(reinterpret_cast<unsigned long long *>(&sums[warp_of].y), 1ull);
            }
            __syncthreads();
            for (int i = entries + tid; i < entries * int(blocks); i += kDrawThreads)
              cluster_store(&sums[i % entries], uint32_t(i / entries), sums[i % entries].x, sums[i % entries].y);
          }
        }
        if (tid == 0) {
          if (n < 0) told.state = kTooMany;
          else if (n_keep == 0) told.state = kAll;       // min-p leaves out the whole bin
          else {
            const uint64_t e = list[n_keep - 1];
            told.code = ~uint32_t(e >> 32);
            told.index = int32_t(uint32_t(e));
          }
        }
        tell(&told);
      }
      sync_all();
      if (told.state == kTooMany) too_many = true;
      else if (told.state == kGo) {
        x_f = logit_of<float>(told.code);
        i_f = told.index;
      }
      summed = kMass && !too_many;
    };
    if (top_k > 0 && top_k < p.V) round(std::false_type{}, Sum(top_k));
    if (!too_many && top_p < 1.f) round(std::true_type{}, 0);
  }
  if (too_many) {
    // ------------------------------------------------- any row, by codes alone
    // Looks for the logit at which the running count (kMass: weight) of the order reaches the
    // target, among those above `floor`; kMass: the target is top_p of their sum and
    // `beyond`, the weight of what is kept of those equal to the floor.
    auto search = [&](auto mass, float floor, Sum target, Sum beyond) {
      constexpr bool kMass = decltype(mass)::value;
      Search s;
      s.hi = code_of<T>(top);
      s.lo = code_of<T>(floor) + 1;
      s.shift = shift_for(s.hi - s.lo);
      s.target = target;
      s.done = 0;
      bool first = true;
      while (true) {
        clear_bins(kLong ? 3 : 2);
        each([&](int, float y0, float y1) {
#pragma unroll 1
          for (int k = 0; k < 2; ++k) {
            const float y = k ? y1 : y0;
            const uint32_t code = code_of<T>(y);
            if (code > s.hi || code < s.lo) continue;
            const uint32_t b = min((s.hi - code) >> s.shift, uint32_t(kBins - 1));
            if constexpr (kMass) {
              const uint64_t w = weigh(y);
              const uint32_t low = uint32_t(w);
              const uint32_t more = uint32_t(w >> 32) + (atomicAdd(bin_lo + b, low) + low < low);
              if (more && atomicAdd(bin_hi + b, more) + more < more && kLong) atomicAdd(bin_top + b, 1u);
            } else {
              atomicAdd(bin_lo + b, 1u);
            }
          }
        });
        const Found f = find(std::integral_constant<int, kMass ? kWeights : kCounts>{}, first && kMass ? Sum(0) : s.target, beyond);
        first = false;
        s.target = f.target;
        if (f.state == kAll) {
          s.done = 2;
          return s;
        }
        s.hi -= f.bin << s.shift;
        if (f.bin < kBins - 1) {
          s.done = s.shift == 0;
          s.lo = max(s.lo, s.hi - ((1u << s.shift) - 1));
        }
        s.shift = shift_for(s.hi - s.lo);
        if (s.done) {
          const uint64_t w = kMass ? weigh(logit_of<T>(s.hi)) : 1;
          s.ties = count_for(s.target, w);
          return s;
        }
      }
    };
    x_f = -INFINITY;
    uint64_t ties = 0;                                   // how many equal to x_f are kept
    if (top_k > 0 && top_k < p.V) {
      const Search s = search(std::false_type{}, -INFINITY, Sum(top_k), 0);
      if (s.done == 1) {
        x_f = logit_of<T>(s.hi);
        ties = s.ties;
      }
    }
    if (top_p < 1.f) {
      const uint64_t w = ties ? weigh(x_f) : 0;
      const Search s = search(std::true_type{}, x_f, 0, Sum(ties) * w);
      if (s.done == 1) {
        x_f = logit_of<T>(s.hi);
        ties = s.ties;
      } else if (w) {
        ties = min(ties, count_for(s.target, w));
      }
    }
    // the index of the last of them
    uint32_t n = 0;
    each([&](int, float a, float b) {
      if (x_f > -INFINITY) n += uint32_t(a == x_f) + uint32_t(b == x_f);
    });
    n = __reduce_add_sync(~0u, n);
    if (lane < int(blocks)) cluster_store(&sums[me], lane, n, 0);
    sync_all();
    uint64_t before = 0;
    for (int i = lane; i < me; i += 32) before += sums[i].x;
#pragma unroll
    for (int w = 16; w; w /= 2) before += __shfl_xor_sync(~0u, before, w);
    if (ties > before && ties <= before + n) {
      uint32_t left = uint32_t(ties - before);
      each([&](int r, float a, float b) {
        const uint32_t here = uint32_t(a == x_f) + uint32_t(b == x_f);
        uint32_t run = uint32_t(scan_up(uint64_t(here), lane));
        const uint32_t all = __shfl_sync(~0u, run, 31);
        run -= here;
        if (left > run && left <= run + here) {
          const int its_index = a == x_f && left == run + 1 ? r : r + 1;
          for (uint32_t to = 0; to < blocks; ++to) cluster_store(&told.target, to, uint64_t(uint32_t(its_index)), 0);
        }
        left = left > all ? left - all : 0;
      });
    }
    sync_all();
    i_f = ties ? int(told.target) : INT32_MIN;
    sync_all();                                          // (sums are read before they are written again)
  }
  if (!done) {
    if (f_min > x_f) {
      x_f = f_min;
      i_f = INT32_MAX;
    }
    // -------------------------------------------------------------- the draw
    if (!summed) {
      Mass mass = 0;
      each([&](int r, float a, float b) {
        const bool ka = kept(a, r), kb = kept(b, r + 1);
        if (!ka && !kb) return;
        Weight wa, wb;
        weigh2<T>(scale, powers, a, b, wa, wb);
        mass += (ka ? wa.value(kOne) : 0) + (kb ? wb.value(kOne) : 0);
      });
      tell_mass(mass);
      sync_all();
    }
    const Sum mass = sum_of<Sum>(sums[me]);
    Sum my_mass = 0;                                     // of the warps before this one
    for (int i = lane; i < entries; i += 32) {
      const Sum part = sum_of<Sum>(sums[i]);
      whole += part;
      if (i < me) my_mass += part;
    }
    whole = warp_sum<Sum>(whole);
    my_mass = warp_sum<Sum>(my_mass);
    for (int d = 0; d < p.draws; ++d) {
      const Sum want = drawn(d, whole);
      if (want < my_mass || want >= my_mass + mass) continue;
      Sum run = my_mass;
      bool found = false;
      each([&](int r, float a, float b) {
        if (found) return;
        Weight w0, w1;
        weigh2<T>(scale, powers, a, b, w0, w1);
        const uint64_t wa = kept(a, r) ? w0.value(kOne) : 0, sum = wa + (kept(b, r + 1) ? w1.value(kOne) : 0);
        const uint64_t to = scan_up(sum, lane);
        const Sum from = run + (to - sum);
        if (want >= from && want < run + to) p.tokens[row * p.draws + d] = want < from + wa ? r : r + 1;
        run += __shfl_sync(~0u, to, 31);
        found = run > want;
      });
    }
  }
  if (!out) return;
  // ------------------------------------------------------- the distribution
  const float c = scale.c * (1.f / 64), inv = 1.f / (float(uint64_t(whole >> (kLong ? 20 : 0))) * exp2f(float((kLong ? 20 : 0) - kOne)));
  auto share = [&](float y, int r) { return kept(y, r) ? (y == top ? 1.f : ex2(fmaf(y, -scale.minus, -scale.top) * c)) * inv : 0.f; };
  each([&](int r, float a, float b) { store(r, share(a, r), share(b, r + 1)); });
}

template <typename T>
cudaError_t launch_sample(DrawParams p, int64_t rows, int sms, cudaStream_t st) {
  const int64_t units = p.V / 8 + 2, size = 8 * sizeof(T);
  // As few blocks a row as hold it in 76 KB each (two blocks an SM; 256 rows of 151936 BF16 logits
  // with settings of their own 106 us on 4 blocks of 76 KB, 148 on 8 of 38), and more while all rows'
  // fit the device about at once (41 such rows 60 us on 4, 42 on 8); 16, more than a portable cluster, for a
  // few rows alone (8 rows of top-p 40 us, 42 on 8).
  int c = 1;
  auto more = [&] { return units * size > int64_t(kDrawShare) * c; };
  while (c < 8 && (more() || (8 * rows * c <= 9 * sms && units > kDrawThreads * c))) c *= 2;
  if (c == 8 && (more() || (units > 8 * kDrawThreads && rows * 16 <= sms))) c = kMaxCluster;
  const int64_t warps = int64_t(c) * kDrawWarps;
  p.chunk = int((units + warps - 1) / warps);
  const int64_t share = int64_t(p.chunk) * kDrawWarps * size;
  const bool held = share <= kDrawShareMax;
  // In what order they begin: with more blocks than run at once the rows that take longest should not be
  // the last (256 rows of mixed settings 121 us, in their own order 141, 512 rows 224 and 240; rows of equal
  // ones, for which it is a search for nothing, 1.5 % more: 256 of top-p 217.5 and 214.5).  A thread looks at
  // one row, so more than 512 keep their order.  Rows of short blocks keep theirs: the settings take a
  // microsecond to read.
  const bool ordered = held && rows <= kDrawThreads && rows * c > 2 * sms && share >= 32 * 1024 && (p.top_k || p.top_p);
  p.rows = int(std::min<int64_t>(rows, kDrawThreads));
  static std::atomic<uint64_t> allowed[5];
  const bool is_long = p.V >= kLongVocab;
  static_assert(kMaxCluster * kDrawShareMax / 2 / 4 >= kLongVocab, "what is not held is long");
  using Kernel = void (*)(DrawParams);
  constexpr Kernel kernels[5] = {&sample_kernel<T, true, false, false>, &sample_kernel<T, true, true, false>,
                                 &sample_kernel<T, true, false, true>, &sample_kernel<T, true, true, true>,
                                 &sample_kernel<T, false, false, true>};
  const int which = held ? 2 * is_long + ordered : 4;
  const Kernel fn = kernels[which];
  if (const cudaError_t e = allow(fn, kListBytes + (held ? kDrawShareMax : 0), allowed[which])) return e;
  return launch_clusters(fn, unsigned(rows) * unsigned(c), kDrawThreads, c, kListBytes + (held ? int(share) : 0), st, p);
}

}  // namespace
}  // namespace vg

using namespace vg;

extern "C" vg_status vg_sample(const vg_sample_desc *d, vg_stream_t stream) {
  if (!d || !d->x || !d->u || !d->tokens || d->rows < 1 || d->vocab < 1 || d->draws < 1 || d->row_stride < d->vocab)
    return VG_ERR_INVALID_ARG;
  if (d->type != VG_TYPE_BF16 && d->type != VG_TYPE_FP16 && d->type != VG_TYPE_FP32) return VG_ERR_INVALID_ARG;
  const int size = d->type == VG_TYPE_FP32 ? 4 : 2;
  const uintptr_t at = reinterpret_cast<uintptr_t>(d->x);
  if (at % uintptr_t(size) || reinterpret_cast<uintptr_t>(d->out) & 3) return VG_ERR_ALIGNMENT;
  for (const void *p : {static_cast<const void *>(d->u), static_cast<const void *>(d->temperature),
                        static_cast<const void *>(d->top_k), static_cast<const void *>(d->top_p),
                        static_cast<const void *>(d->min_p), static_cast<const void *>(d->tokens)})
    if (reinterpret_cast<uintptr_t>(p) & 3) return VG_ERR_ALIGNMENT;
  if (d->vocab >= (int64_t(1) << 28) || d->rows >= (int64_t(1) << 26) || d->draws > 65536 ||
      d->row_stride >= kMaxElems / d->rows)
    return VG_ERR_UNSUPPORTED;
  int sms = 0;
  if (vg_status s = device_sms(&sms)) return s;
  DrawParams p{};
  p.x = reinterpret_cast<const void *>(at & ~uintptr_t(15));
  p.lead = int(at & 15) / size;
  p.V = d->vocab;
  p.stride = d->row_stride;
  p.u = d->u;
  p.temperature = d->temperature;
  p.top_p = d->top_p;
  p.min_p = d->min_p;
  p.top_k = d->top_k;
  p.tokens = d->tokens;
  p.out = d->out;
  p.draws = d->draws;
  cudaError_t e;
  if (d->type == VG_TYPE_BF16) e = launch_sample<__nv_bfloat16>(p, d->rows, sms, as_cuda(stream));
  else if (d->type == VG_TYPE_FP16) e = launch_sample<__half>(p, d->rows, sms, as_cuda(stream));
  else e = launch_sample<float>(p, d->rows, sms, as_cuda(stream));
  if (e != cudaSuccess) {
    set_cuda_error(e);
    return VG_ERR_CUDA;
  }
  return VG_OK;
}
