// vg_draw.cu -- vg_sample: draws from the softmax of logits with a temperature,
// truncated by top-k, top-p and min-p, from given random numbers.
//
// A row's tokens are ordered by logit, the largest first, equal ones by index.
// What a row keeps is a beginning of that order: at most k tokens, of these the
// fewest whose weights 2^-z, z = (max - x) log2 e / T, sum to p times theirs,
// of these the ones that weigh min_p and more.  So it is given by the last kept
// logit x_f and how many of the logits equal to it are kept, m_f, the first by
// index.  The token drawn is the first index whose running sum over what is
// kept exceeds u times the whole.
//
// Sums are integers (a weight of 1 is 2^s with sums below 2^62), so that no order
// of addition changes what is kept or drawn, and weights are exact to some
// 2^-29 of themselves: a draw is a comparison of u with the boundaries of 150000
// tokens, and with sums good to 2^-22 one row in some hundred would end on the
// neighbour.
//
// A cluster of blocks a row; a block holds a run of it in shared memory, and
// each warp a run of that, so that the warps' order is the index order.  x_f is
// looked for in histograms of 2048 bins over the logits' codes (ordered as
// integers): a level narrows the range to the codes of one bin.
#include <algorithm>
#include <cmath>

#include "vg_rows.cuh"

namespace vg {
namespace {

constexpr int kDrawThreads = 512, kDrawWarps = kDrawThreads / 32;
constexpr int kBins = 2048;
constexpr int kDrawShare = 72 * 1024;         // bytes of a row a block should hold at most ...
constexpr int kDrawShareMax = 160 * 1024;     // ... and may

struct DrawParams {
  const void *x;
  int64_t V, stride;
  const float *u, *temperature, *top_p, *min_p;
  const int32_t *top_k;
  int32_t *tokens;
  float *out;
  int draws, chunk, bits;            // units of a warp; a weight of 1 is 2^bits
};

// 2^(30 - j / 32)
__constant__ uint32_t kPowers[32] = {
    1073741824, 1050733751, 1028218693, 1006186087, 984625594, 963527098, 942880699, 922676710,
    902905651,  883558244,  864625413,  846098274,  827968132, 810226483, 792865000, 775875538,
    759250125,  742980960,  727060411,  711481005,  696235434, 681316545, 666717336, 652430958,
    638450708,  624770026,  611382493,  598281827,  585461881, 572916640, 560640218, 548626854};

// What a row's weights need: z in units of 1/32 is (max - x) c.
struct Scale {
  float top, c, c_low, cap;          // c as two floats; differences beyond cap weigh nothing
};

// The weight of logit x: 2^-z in units of 2^-bits (up = bits - 30).  With z = (k + r) / 32, k
// whole, |r| <= 1/2, it is 2^-(k / 32) from a table times 2^-(r / 32) by its series.
// max - x is exact in FP32 for 16-bit logits but for those that are 2^-16 of
// the largest or less; for FP32 ones what it loses is carried along.
template <typename T>
__device__ __forceinline__ uint64_t weight(const Scale &s, const uint32_t *powers, float x, int up) {
  constexpr float kMagic = 12582912.f;         // 1.5 2^23: what is added to it is rounded to a whole number
  const float d = fminf(s.top - x, s.cap);
  float low = d * s.c_low;
  if constexpr (std::is_same_v<T, float>) {
    const float a = s.top - x, b = a - s.top;
    const float e = (s.top - (a - b)) + (-x - b);
    low = a < s.cap ? fmaf(e, s.c, low) : low;
  }
  const float t = fmaf(d, s.c, kMagic);
  const int k = __float_as_int(t) - __float_as_int(kMagic);
  const float r = fmaf(d, s.c, -(t - kMagic)) + low;
  // 2^28 (2^-(r / 32) - 1)
  float q = fmaf(r, 2.46224105f, -454.689658f);
  q = fmaf(r, q, 62973.9374f);
  q = fmaf(r, q, -5814539.98f);
  const int f = __float_as_int(fmaf(r, q, kMagic)) - __float_as_int(kMagic);
  const int w = int(powers[k & 31]);
  const uint64_t v = uint64_t(uint32_t(w + __mulhi(w, f << 4))) << up;
  return x == -INFINITY ? 0 : v >> min(k >> 5, 63);
}

// Logits' codes in their order; logits of 16 bits have as many codes.
template <typename T>
constexpr int kCodeShift = std::is_same_v<T, float> ? 0 : std::is_same_v<T, __half> ? 13 : 16;
template <typename T>
__device__ __forceinline__ uint32_t code_of(float x) {
  const uint32_t b = __float_as_uint(x);
  return (b ^ (uint32_t(int32_t(b) >> 31) | 0x80000000u)) >> kCodeShift<T>;
}
template <typename T>
__device__ __forceinline__ float logit_of(uint32_t code) {
  uint32_t b = code << kCodeShift<T>;
  b = b & 0x80000000u ? b ^ 0x80000000u : ~(b | ((1u << kCodeShift<T>) - 1));
  return __uint_as_float(b);
}

// floor(a s) for 0 <= a < 1
__device__ __forceinline__ uint64_t part_of(float a, uint64_t s, bool &exact) {
  if (!(a > 0.f)) {
    exact = true;
    return 0;
  }
  const uint32_t b = __float_as_uint(a);
  const uint32_t e = b >> 23;
  const uint64_t m = e ? (b & 0x7FFFFF) | 0x800000 : b & 0x7FFFFF;
  const int right = 150 - int(e ? e : 1);      // a = m 2^-right, right >= 24
  const uint64_t lo = m * s, hi = __umul64hi(m, s);
  if (right >= 64) {
    const uint64_t v = right < 128 ? hi >> (right - 64) : 0;
    exact = false;                             // (some bits are lost, or the product is 0)
    return v;
  }
  exact = (lo & ((uint64_t(1) << right) - 1)) == 0;
  return hi << (64 - right) | lo >> right;
}

__device__ __forceinline__ uint64_t scan_up(uint64_t v, int lane) {
#pragma unroll
  for (int w = 1; w < 32; w *= 2) {
    const uint64_t y = __shfl_up_sync(~0u, v, w);
    if (lane >= w) v += y;
  }
  return v;
}

// Where a search is: codes [lo, hi], bins of 2^shift of them from hi down, the last
// bin with all that is below; what is wanted of them.
struct Search {
  uint32_t hi, lo;
  int shift, done;                   // 1: hi is the code, 2: there are fewer
  uint64_t target, ties;             // ties: of the code
};
__device__ __forceinline__ int shift_for(uint32_t span) {
  // the smallest with span >> shift below the last bin
  int s = max(0, 21 - __clz(int(span | 1)));
  return (span >> s) < kBins - 1 ? s : s + 1;
}

template <typename T, bool kHeld>
__global__ void __launch_bounds__(kDrawThreads, 1) sample_kernel(const __grid_constant__ DrawParams p) {
  extern __shared__ __align__(16) uint8_t draw_smem[];
  __shared__ __align__(16) ulonglong2 tops[kMaxCluster * kDrawWarps];
  __shared__ __align__(16) ulonglong2 sums[kMaxCluster * kDrawWarps];
  __shared__ __align__(16) Search told;
  __shared__ uint32_t powers[32];
  __shared__ Scale told_scale;
  __shared__ double min_at;          // T ln(min_p)
  __shared__ uint64_t scan[kDrawWarps];
  uint32_t *bin_lo = reinterpret_cast<uint32_t *>(draw_smem), *bin_hi = bin_lo + kBins;
  uint4 *held = reinterpret_cast<uint4 *>(bin_hi + kBins);
  const uint32_t rank = cluster_rank(), blocks = cluster_size();
  const int64_t row = blockIdx.x / blocks;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const T *x = static_cast<const T *>(p.x);
  const int64_t lo = row * p.stride, hi = lo + p.V;
  const int64_t end = (hi + 7) / 8;                      // units, on the grid of the whole array
  const int64_t w0 = lo / 8 + int64_t(rank * kDrawWarps + warp) * p.chunk;
  const int mine = int(max(int64_t(0), min(int64_t(p.chunk), end - w0)));   // units of this warp
  if (blocks > 1) cluster_arrive();                      // a block must have begun before others write to it
  constexpr int kPart = sizeof(T) / 2;
  const int part = kDrawWarps * p.chunk;                 // 16-byte parts of a unit lie apart
  uint4 *at = held + warp * p.chunk;
  if constexpr (kHeld) {
    for (int i = lane; i < mine; i += 32) {
      const int64_t e = (w0 + i) * 8;
      if (e >= lo && e + 8 <= hi) {
#pragma unroll
        for (int k = 0; k < kPart; ++k) copy16(at + k * part + i, reinterpret_cast<const uint4 *>(x + e) + k);
      } else {
        const Unit<T> v = load_unit(x, w0 + i, lo, hi);
#pragma unroll
        for (int k = 0; k < kPart; ++k) at[k * part + i] = v.w[k];
      }
    }
  }
  const float temperature = p.temperature ? p.temperature[row] : 1.f;
  const float min_p = p.min_p ? p.min_p[row] : 0.f, top_p = p.top_p ? p.top_p[row] : 1.f;
  const int top_k = p.top_k ? p.top_k[row] : 0;
  if (warp == 0) {
    powers[lane] = kPowers[lane];
    if (lane == 0) {
      const double c = 32 * 1.4426950408889634074 / double(temperature);
      told_scale.c = c > 3.4e38 ? 3.4028234e38f : float(c);
      told_scale.c_low = c > 3.4e38 ? 0.f : float(c - double(told_scale.c));
      told_scale.cap = fminf(2048.f / told_scale.c, 3.4028234e38f);
      // (over an infinite temperature every finite logit weighs 1)
      min_at = !(min_p > 0.f) ? 0.0 : temperature == INFINITY ? (min_p > 1.f ? 1e300 : -1e300)
                                                              : double(temperature) * log(double(min_p));
    }
  }
  if constexpr (kHeld) asm volatile("cp.async.wait_all;" ::: "memory");   // a thread reads only what it copied
  auto unit = [&](int i) {
    if constexpr (kHeld) {
      Unit<T> v;
#pragma unroll
      for (int k = 0; k < kPart; ++k) v.w[k] = at[k * part + i];
      return v;
    } else {
      return load_unit(x, w0 + i, lo, hi);
    }
  };
  // f(i, logits 8 i .. 8 i + 7 of the warp's run), 0 for -0; all lanes come along
  auto each = [&](auto &&f) {
#pragma unroll 1
    for (int i0 = 0; i0 < mine; i0 += 32) {
      const int i = i0 + lane;
      float y[8];
      if (i < mine) {
        const Unit<T> v = unit(i);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          y[2 * k] = v.pair(k).x + 0.f;
          y[2 * k + 1] = v.pair(k).y + 0.f;
        }
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) y[k] = -INFINITY;
      }
      f(i, y);
    }
  };

  // ------------------------------------------------------------- the largest
  Largest<T> largest;
  for (int i = lane; i < mine; i += 32) largest.take(unit(i));
  float m = largest.value();
#pragma unroll
  for (int w = 16; w; w /= 2) m = max_nan(m, __shfl_xor_sync(~0u, m, w));
  auto sync_all = [&] {
    if (blocks > 1) cluster_sync();
    else __syncthreads();
  };
  if (blocks > 1) cluster_wait();
  if (lane < int(blocks)) cluster_store(&tops[rank * kDrawWarps + warp], lane, __float_as_uint(m), 0);
  sync_all();
  const int entries = int(blocks) * kDrawWarps;
  float top = -INFINITY;
  for (int i = lane; i < entries; i += 32) top = max_nan(top, __uint_as_float(uint32_t(tops[i].x)));
#pragma unroll
  for (int w = 16; w; w /= 2) top = max_nan(top, __shfl_xor_sync(~0u, top, w));
  top += 0.f;
  const bool greedy = temperature <= 0.f;
  float *out = p.out ? p.out + row * p.V : nullptr;
  // no token: a NaN, an infinity that weighs all, nothing but -infinity
  const bool bad = isnan(top) || isnan(temperature) || (top == INFINITY && !greedy);
  if (bad || top == -INFINITY) {
    if (rank == 0)
      for (int i = tid; i < p.draws; i += kDrawThreads) p.tokens[row * p.draws + i] = -1;
    if (out) {
      const float v = bad && !greedy ? __int_as_float(0x7FFFFFFF) : 0.f;
      for (int64_t i = rank * kDrawThreads + tid; i < p.V; i += int64_t(blocks) * kDrawThreads) out[i] = v;
    }
    return;
  }
  Scale scale = told_scale;
  scale.top = top;
  const int up = p.bits - 30;
  auto weigh = [&](float y) { return weight<T>(scale, powers, y, up); };

  // ---------------------------------------------------------- what is kept
  // Kept are logits above x_f and the first m_f equal to it.
  float x_f = -INFINITY;
  uint64_t m_f = 0;
  // Looks for the logit at which the running count (kMass: weight) of the order reaches the
  // target, among those above `floor`; kMass: the target is top_p of their sum and
  // `beyond`, the weight of what is kept of those equal to the floor.
  auto search = [&](auto mass, float floor, uint64_t target, uint64_t beyond) {
    constexpr bool kMass = decltype(mass)::value;
    Search s;
    s.hi = code_of<T>(top);
    s.lo = code_of<T>(floor) + 1;
    // (beyond 40 octaves of weight the bins need not tell codes apart)
    const uint32_t guess = code_of<T>(fmaxf(top - 1280.f / scale.c, floor));
    s.shift = shift_for(s.hi - min(guess, s.hi));
    s.target = target;
    s.done = 0;
    bool first = true;
    while (true) {
      for (int i = tid; i < 2 * kBins; i += kDrawThreads) bin_lo[i] = 0;
      __syncthreads();
      each([&](int, const float (&y)[8]) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint32_t code = code_of<T>(y[k]);
          if (code > s.hi || code < s.lo) continue;
          const uint32_t b = min((s.hi - code) >> s.shift, uint32_t(kBins - 1));
          if constexpr (kMass) {
            const uint64_t w = weigh(y[k]);
            const uint32_t low = uint32_t(w);
            const uint32_t old = atomicAdd(bin_lo + b, low);
            const uint32_t more = uint32_t(w >> 32) + (old + low < old);
            if (more) atomicAdd(bin_hi + b, more);
          } else {
            atomicAdd(bin_lo + b, 1u);
          }
        }
      });
      sync_all();
      if (rank == 0) {
        // four bins a thread, of all blocks
        constexpr int kEach = kBins / kDrawThreads;
        uint64_t v[kEach] = {};
        for (uint32_t r = 0; r < blocks; ++r)
#pragma unroll
          for (int k = 0; k < kEach; ++k) {
            uint32_t a, b;
            const uint32_t here = static_cast<uint32_t>(__cvta_generic_to_shared(bin_lo + tid * kEach + k));
            asm volatile("{ .reg .b32 at; mapa.shared::cluster.u32 at, %2, %3; ld.shared::cluster.u32 %0, [at];\n"
                         "ld.shared::cluster.u32 %1, [at + %4]; }"
                         : "=&r"(a), "=&r"(b)
                         : "r"(here), "r"(r), "n"(kBins * 4)
                         : "memory");
            v[k] += uint64_t(b) << 32 | a;
          }
        uint64_t sum = 0;
#pragma unroll
        for (int k = 0; k < kEach; ++k) sum += v[k];
        uint64_t run = scan_up(sum, lane);
        if (lane == 31) scan[warp] = run;
        __syncthreads();
        uint64_t whole = 0;
#pragma unroll
        for (int w = 0; w < kDrawWarps; ++w) {
          if (w < warp) run += scan[w];
          whole += scan[w];
        }
        uint64_t before = run - sum;
        Search next = s;
        if (kMass && first) {
          bool exact;
          next.target = part_of(top_p, whole + beyond, exact);
          next.target = max(next.target + !exact, uint64_t(1));
        }
        if (next.target > whole) {
          if (tid == 0) {
            next.done = 2;
            next.target -= whole;
            told = next;
          }
        } else if (before < next.target && next.target <= run) {
          int b = 0;
#pragma unroll
          for (int k = 0; k < kEach - 1; ++k)
            if (b == k && before + v[k] < next.target) {
              before += v[k];
              ++b;
            }
          const uint32_t bin = uint32_t(tid * kEach + b);
          next.target -= before;
          const uint32_t above = s.hi - (bin << s.shift);
          if (bin < kBins - 1) {
            next.done = s.shift == 0;
            next.lo = max(s.lo, above - ((1u << s.shift) - 1));
          }
          next.hi = above;
          next.shift = shift_for(next.hi - next.lo);
          if (next.done) {
            const uint64_t w = kMass ? weigh(logit_of<T>(above)) : 1;
            next.ties = (next.target + w - 1) / w;
          }
          told = next;
        }
        __syncthreads();
        // to the other blocks
        if (blocks > 1 && tid < int(blocks)) {
          const uint64_t *from = reinterpret_cast<const uint64_t *>(&told);
          if (tid)
#pragma unroll
            for (int k = 0; k < int(sizeof(Search) / 16); ++k)
              cluster_store(reinterpret_cast<ulonglong2 *>(&told) + k, uint32_t(tid), from[2 * k], from[2 * k + 1]);
        }
      }
      sync_all();
      s = told;
      first = false;
      if (s.done) return s;
    }
  };
  if (greedy) {
    x_f = top;
    m_f = 1;
  } else {
    if (top_k > 0 && top_k < p.V) {
      const Search s = search(std::false_type{}, -INFINITY, uint64_t(top_k), 0);
      if (s.done == 1) {
        x_f = logit_of<T>(s.hi);
        m_f = s.ties;
      }
    }
    if (top_p < 1.f) {
      const uint64_t w = m_f ? weigh(x_f) : 0;
      const Search s = search(std::true_type{}, x_f, 0, m_f * w);
      if (s.done == 1) {
        x_f = logit_of<T>(s.hi);
        m_f = s.ties;
      } else if (w) {
        m_f = min(m_f, (s.target + w - 1) / w);
      }
    }
    if (min_p > 0.f) {
      // the smallest logit that weighs min_p: those below are left out
      const double least = double(top) + min_at;
      float f = __double2float_ru(least);
      if (!(f < top)) {
        if (f > top) m_f = x_f == top ? min(m_f, uint64_t(1)) : 1;   // (min_p above 1: the first token alone)
        else if (x_f < top) m_f = uint64_t(p.V);
        x_f = top;
      } else if (f > x_f) {
        x_f = f;
        m_f = uint64_t(p.V);
      }
    }
  }

  // ---------------------------------------------------------------- the draw
  // of each warp: the weight above x_f and how many are equal to it
  uint64_t mass = 0;
  uint32_t ties = 0;
  each([&](int, const float (&y)[8]) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (y[k] > x_f) mass += weigh(y[k]);
      ties += y[k] == x_f;
    }
  });
#pragma unroll
  for (int w = 16; w; w /= 2) {
    mass += __shfl_xor_sync(~0u, mass, w);
    ties += __shfl_xor_sync(~0u, ties, w);
  }
  if (lane < int(blocks)) cluster_store(&sums[rank * kDrawWarps + warp], lane, mass, ties);
  sync_all();
  const uint64_t w_f = x_f == top ? uint64_t(1) << p.bits : m_f ? weigh(x_f) : 0;
  // entries a lane: a run of the warps; how many ties and how much weight lie before it
  const int per = (entries + 31) / 32, first = lane * per;
  uint64_t t = 0;
  for (int i = first; i < min(first + per, entries); ++i) t += sums[i].y;
  const uint64_t t_before = scan_up(t, lane) - t;
  auto kept_ties = [&](uint64_t before, uint64_t n) { return before >= m_f ? 0 : min(n, m_f - before); };
  uint64_t here = 0, ties_run = t_before;
  for (int i = first; i < min(first + per, entries); ++i) {
    here += sums[i].x + kept_ties(ties_run, sums[i].y) * w_f;
    ties_run += sums[i].y;
  }
  const uint64_t upto = scan_up(here, lane);
  const uint64_t whole = __shfl_sync(~0u, upto, 31);
  // what lies before this warp
  const int me = rank * kDrawWarps + warp;
  uint64_t my_ties = t_before, my_mass = upto - here;
  for (int i = first; i < min(first + per, me); ++i) {
    my_mass += sums[i].x + kept_ties(my_ties, sums[i].y) * w_f;
    my_ties += sums[i].y;
  }
  my_ties = __shfl_sync(~0u, my_ties, me / per);
  my_mass = __shfl_sync(~0u, my_mass, me / per);
  const uint64_t my_end = my_mass + mass + kept_ties(my_ties, ties) * w_f;
  const int64_t base = w0 * 8 - lo;                      // index of the run's first element
  for (int d = 0; d < p.draws; ++d) {
    float u = p.u[row * p.draws + d];
    u = u >= 1.f ? 0x1.fffffep-1f : u;
    bool exact;
    const uint64_t want = part_of(u, whole, exact);      // the first running sum above it
    if (want < my_mass || want >= my_end) continue;
    uint64_t run = my_mass, tie = my_ties;
    bool found = false;
    each([&](int i, const float (&y)[8]) {
      if (found) return;
      uint32_t n = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) n += y[k] == x_f;
      uint32_t n_before = n;
#pragma unroll
      for (int w = 1; w < 32; w *= 2) {
        const uint32_t z = __shfl_up_sync(~0u, n_before, w);
        if (lane >= w) n_before += z;
      }
      const uint32_t n_all = __shfl_sync(~0u, n_before, 31);
      uint64_t t0 = tie + n_before - n, sum = 0, each_w[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        each_w[k] = y[k] > x_f ? weigh(y[k]) : 0;
        if (y[k] == x_f && t0++ < m_f) each_w[k] = w_f;
        sum += each_w[k];
      }
      const uint64_t to = scan_up(sum, lane);
      uint64_t from = run + to - sum;
      if (want >= from && want < run + to) {
        int at8 = 0;
        for (int k = 0; k < 8; ++k) {
          if (want >= from + each_w[k]) at8 = k + 1;
          else break;
          from += each_w[k];
        }
        p.tokens[row * p.draws + d] = int32_t(base + int64_t(i) * 8 + at8);
      }
      run += __shfl_sync(~0u, to, 31);
      tie += n_all;
      found = run > want;
    });
  }
  if (!out) return;
  // ------------------------------------------------------- the distribution
  const float c = scale.c * (1.f / 32), inv = 1.f / (float(whole) * exp2f(float(-p.bits)));
  uint64_t tie = my_ties;
  const bool aligned = ((row * p.V + base) & 3) == 0;
  each([&](int i, const float (&y)[8]) {
    uint32_t n = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) n += y[k] == x_f;
    uint32_t n_before = n;
    if (__any_sync(~0u, n != 0)) {
#pragma unroll
      for (int w = 1; w < 32; w *= 2) {
        const uint32_t z = __shfl_up_sync(~0u, n_before, w);
        if (lane >= w) n_before += z;
      }
    }
    uint64_t t0 = tie + n_before - n;
    tie += __shfl_sync(~0u, n_before, 31);
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const bool kept = y[k] > x_f || (y[k] == x_f && t0 < m_f && y[k] > -INFINITY);
      t0 += y[k] == x_f;
      v[k] = kept ? (y[k] == top ? 1.f : ex2((y[k] - top) * c)) * inv : 0.f;
    }
    if (i >= mine) return;
    const int64_t r = base + int64_t(i) * 8;
    if (aligned && r >= 0 && r + 8 <= p.V) {
      float4 *to = reinterpret_cast<float4 *>(out + r);
      __stcs(to, make_float4(v[0], v[1], v[2], v[3]));
      __stcs(to + 1, make_float4(v[4], v[5], v[6], v[7]));
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (r + k >= 0 && r + k < p.V) out[r + k] = v[k];
    }
  });
}

template <typename T>
cudaError_t launch_sample(DrawParams p, int64_t rows, int sms, cudaStream_t st) {
  const int64_t units = p.V / 8 + 2, size = 8 * sizeof(T);
  int c = 1;
  while (c < 8 &&
         (units * size > int64_t(kDrawShare) * c || (rows * c < 2 * sms && units > kDrawThreads * c)))
    c *= 2;
  if (c == 8 && (units * size > int64_t(kDrawShare) * c || (units > 8 * kDrawThreads && rows * 32 <= sms)))
    c = kMaxCluster;
  const int64_t warps = int64_t(c) * kDrawWarps;
  p.chunk = int((units + warps - 1) / warps);
  const int64_t share = int64_t(p.chunk) * kDrawWarps * size;
  static std::atomic<uint64_t> allowed[2];
  const bool held = share <= kDrawShareMax;
  void (*fn)(DrawParams) = held ? &sample_kernel<T, true> : &sample_kernel<T, false>;
  constexpr int kBinBytes = 2 * kBins * 4;
  if (const cudaError_t e = allow(fn, kBinBytes + (held ? kDrawShareMax : 0), allowed[held])) return e;
  return launch_clusters(fn, unsigned(rows) * unsigned(c), kDrawThreads, c, kBinBytes + (held ? int(share) : 0), st, p);
}

}  // namespace
}  // namespace vg

using namespace vg;

extern "C" vg_status vg_sample(const vg_sample_desc *d, vg_stream_t stream) {
  if (!d || !d->x || !d->u || !d->tokens || d->rows < 1 || d->vocab < 1 || d->draws < 1 || d->row_stride < d->vocab)
    return VG_ERR_INVALID_ARG;
  if (d->type != VG_TYPE_BF16 && d->type != VG_TYPE_FP16 && d->type != VG_TYPE_FP32) return VG_ERR_INVALID_ARG;
  if (!aligned16(d->x) || !aligned16(d->out)) return VG_ERR_ALIGNMENT;
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
  p.x = d->x;
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
  p.bits = 62;
  while ((int64_t(1) << (62 - p.bits)) < d->vocab) --p.bits;
  if (p.bits > 60) p.bits = 60;
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
