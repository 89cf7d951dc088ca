// vg_sample.cu -- vg_probabilities (softmax of logits with a temperature per
// row) and vg_verify_tree (verification of drafted tokens).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "vg_internal.h"

namespace vg {
namespace {

__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f(float x) { return x; }

// ------------------------------------------------------------ probabilities
// One block a row: the largest logit and its first place, the sum of
// exponentials, and the row again, divided.
constexpr int kProbThreads = 1024;
constexpr float kLog2e = 1.4426950408889634f;

template <typename T>
__global__ void __launch_bounds__(kProbThreads)
    probabilities_kernel(const T *x, int64_t V, const float *temperature, float *out) {
  __shared__ float red[32];
  __shared__ int64_t where[32];
  const int64_t row = blockIdx.x;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  x += row * V;
  out += row * V;
  const float t = temperature ? temperature[row] : 1.f;
  const bool greedy = t <= 0.f;
  float m = -INFINITY;
  int64_t at = V;
  for (int64_t i = tid; i < V; i += kProbThreads) {
    const float v = to_f(x[i]);
    if (v > m) {
      m = v;
      at = i;
    }
  }
#pragma unroll
  for (int w = 16; w; w /= 2) {
    const float m2 = __shfl_xor_sync(~0u, m, w);
    const int64_t a2 = __shfl_xor_sync(~0u, at, w);
    if (m2 > m || (m2 == m && a2 < at)) {
      m = m2;
      at = a2;
    }
  }
  if (lane == 0) {
    red[warp] = m;
    where[warp] = at;
  }
  __syncthreads();
  for (int w = 0; w < 32; ++w)
    if (red[w] > m || (red[w] == m && where[w] < at)) {
      m = red[w];
      at = where[w];
    }
  __syncthreads();
  if (greedy) {
    for (int64_t i = tid; i < V; i += kProbThreads) out[i] = i == at ? 1.f : 0.f;
    return;
  }
  const float c = kLog2e / t;
  if (m == -INFINITY) m = 0.f;
  float sum = 0.f;
  for (int64_t i = tid; i < V; i += kProbThreads) sum += exp2f((to_f(x[i]) - m) * c);
#pragma unroll
  for (int w = 16; w; w /= 2) sum += __shfl_xor_sync(~0u, sum, w);
  if (lane == 0) red[warp] = sum;
  __syncthreads();
  sum = 0.f;
  for (int w = 0; w < 32; ++w) sum += red[w];
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  for (int64_t i = tid; i < V; i += kProbThreads) out[i] = exp2f((to_f(x[i]) - m) * c) * inv;
}

// -------------------------------------------------------------- verification
// All children of a node were drafted from one q, so the residual after its
// k-th refusal is max(p - a_k q, 0) with a_1 = 1 and a_(k+1) = a_k + S_k,
// S_k the residual's sum: max(max(p - a q, 0) - S q, 0) = max(p - (a + S) q, 0)
// because S q >= 0.  So a refusal costs one pass over two rows and leaves
// one number, and the rows of accepted nodes are never read whole.
//
// Fixed point: p, q and the sums S in units of 2^-60 (a row sums to less
// than 16), a in units of 2^-56 (at most 1 + the number of refusals).
constexpr int kVerThreads = 1024, kVerWarps = kVerThreads / 32;
constexpr int kMaxNodes = 1024;
constexpr float kUnit = 1152921504606846976.f;                 // 2^60

__device__ __forceinline__ float as_probability(float x) { return x > 0.f ? fminf(x, 1.f) : 0.f; }
__device__ __forceinline__ uint64_t to_fixed(float x) { return __float2ull_rz(x * kUnit); }

// a q in units of 2^-60, rounded down; all ones where it does not fit.
__device__ __forceinline__ uint64_t scaled(uint64_t a, float q) {
  const uint32_t bits = __float_as_uint(q), e = bits >> 23;
  if (e == 0) return 0;                                        // 0, or below 2^-126
  const uint64_t m = (bits & 0x7FFFFFu) | 0x800000u;           // q = m 2^(e - 150)
  const uint64_t lo = m * a, hi = __umul64hi(m, a);
  const uint32_t s = 146u - e;                                 // 19..145, as q <= 1
  if (s >= 128) return 0;
  if (s >= 64) return hi >> (s - 64);
  if (hi >> s) return ~0ull;
  return (hi << (64 - s)) | (lo >> s);
}

__device__ __forceinline__ uint64_t residual(float p, float q, uint64_t a) {
  const uint64_t x = to_fixed(as_probability(p));
  const uint64_t y = a ? scaled(a, as_probability(q)) : 0;
  return x > y ? x - y : 0;
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

__global__ void __launch_bounds__(kVerThreads) verify_kernel(const VerifyParams v) {
  __shared__ float pt[kMaxNodes], qt[kMaxNodes], su[kMaxNodes];
  __shared__ int16_t par[kMaxNodes];             // -1: no node to try
  __shared__ uint64_t sums[kVerWarps];
  __shared__ uint64_t s_a;
  __shared__ int s_cur, s_more;
  const int b = blockIdx.x, tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int64_t V = v.V;
  const int n = v.counts ? min(max(v.counts[b], 0), v.n) : v.n;
  const float *prow = v.p + int64_t(b) * v.n * V;
  const float *qrow = v.q + int64_t(b) * v.q_rows * V;
  const int32_t *tokens = v.tokens + int64_t(b) * v.n;
  int32_t *path = v.path + int64_t(b) * v.n, *out = v.out + int64_t(b) * (v.n + 1);
  for (int i = tid; i < v.n; i += kVerThreads) {
    su[i] = v.u[int64_t(b) * v.n + i];
    par[i] = -1;
    path[i] = -1;
    if (i > 0 && i < n) {
      const int f = v.parents[int64_t(b) * v.n + i], t = tokens[i];
      if (f >= 0 && f < i && f < v.q_rows && t >= 0 && t < V) {
        par[i] = int16_t(f);
        pt[i] = as_probability(prow[f * V + t]);
        qt[i] = as_probability(qrow[f * V + t]);
      }
    }
  }
  for (int i = tid; i <= v.n; i += kVerThreads) out[i] = -1;
  __syncthreads();
  // each warp sums one run of the row: the warps' sums in order are the
  // running sum at the runs' ends
  const int64_t run = ((V + kVerWarps - 1) / kVerWarps + 31) / 32 * 32;
  const int64_t first = min(run * warp, V), last = min(first + run, V);
  int i = 1, cur = 0, kept = 0;                  // thread 0's walk
  uint64_t a = 0, S = 1ull << 60, total = 0;
  bool summed = false;
  while (true) {
    if (tid == 0) {
      s_more = 0;
      for (; i < n; ++i) {
        if (par[i] != cur) continue;
        const double left = double(su[i]) * double(qt[i]) * double(S);
        const uint64_t r = a ? residual(pt[i], qt[i], a) : 0;
        const bool ok = a ? left < double(r) : left < double(pt[i]) * double(1ull << 60);
        if (ok) {
          path[kept] = i;
          out[kept++] = tokens[i];
          cur = i;
          a = 0;
          S = 1ull << 60;
          summed = false;
        } else {
          a = a ? a + (S >> 4) : 1ull << 56;
          s_more = 1;
          ++i;
          break;
        }
      }
      // the end: the sums of p itself, where none or empty ones are at hand
      if (!s_more && (!summed || (total == 0 && a != 0))) {
        a = 0;
        s_more = 2;
      }
      s_cur = cur;
      s_a = a;
    }
    __syncthreads();
    const int more = s_more, node = s_cur;
    const uint64_t aa = s_a;
    const float *pr = prow + node * V;
    const float *qr = qrow + (node < v.q_rows ? node : 0) * V;
    if (more) {
      uint64_t sum = 0;
      for (int64_t e = first + lane; e < last; e += 32)
        sum += residual(pr[e], aa ? qr[e] : 0.f, aa);
      sum = warp_sum(sum);
      if (lane == 0) sums[warp] = sum;
      __syncthreads();
      if (tid == 0) {
        total = 0;
        for (int w = 0; w < kVerWarps; ++w) total += sums[w];
        S = total;
        summed = true;
      }
      if (more == 1) continue;
    }
    // draw: the warp whose run the threshold falls into looks it up
    uint64_t whole = 0, before = 0;
    for (int w = 0; w < kVerWarps; ++w) {
      if (w < warp) before += sums[w];
      whole += sums[w];
    }
    const float u0 = fminf(fmaxf(su[0], 0.f), 0x1.fffffep-1f);
    const uint64_t mark = __umul64hi(uint64_t(double(u0) * 18446744073709551616.0), whole);
    if (tid == 0) v.accepted[b] = kept, s_cur = kept;
    __syncthreads();
    if (whole != 0 && before <= mark && mark - before < sums[warp]) {
      uint64_t c = before;
      for (int64_t e0 = first; e0 < last; e0 += 32) {
        const int64_t e = e0 + lane;
        uint64_t x = e < last ? residual(pr[e], aa ? qr[e] : 0.f, aa) : 0;
#pragma unroll
        for (int w = 1; w < 32; w *= 2) {
          const uint64_t y = __shfl_up_sync(~0u, x, w);
          if (lane >= w) x += y;
        }
        const uint32_t over = __ballot_sync(~0u, c + x > mark);
        if (over) {
          if (lane == 0) out[s_cur] = int32_t(e0 + __ffs(over) - 1);
          break;
        }
        c += __shfl_sync(~0u, x, 31);
      }
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
  const unsigned grid = unsigned(rows);
  if (type == VG_TYPE_BF16)
    probabilities_kernel<<<grid, kProbThreads, 0, st>>>(static_cast<const __nv_bfloat16 *>(x),
                                                        vocab, temperature, out);
  else if (type == VG_TYPE_FP16)
    probabilities_kernel<<<grid, kProbThreads, 0, st>>>(static_cast<const __half *>(x), vocab,
                                                        temperature, out);
  else
    probabilities_kernel<<<grid, kProbThreads, 0, st>>>(static_cast<const float *>(x), vocab,
                                                        temperature, out);
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
  verify_kernel<<<unsigned(batch), kVerThreads, 0, as_cuda(stream)>>>(v);
  VG_LAUNCH_CHECK();
  return VG_OK;
}
