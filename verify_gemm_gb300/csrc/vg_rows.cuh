// vg_rows.cuh -- what the kernels over rows of a vocabulary share: clusters of
// blocks a row, exchanges through distributed shared memory, and units of 8
// logits.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <type_traits>

#include "vg_internal.h"
#include "vg_pairs.cuh"

namespace vg {
namespace {

__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }

// ------------------------------------------------------------ clusters
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.aligned;\nbarrier.cluster.wait.aligned;" ::: "memory");
}
// The two halves of the barrier: what is done between them overlaps the wait.
__device__ __forceinline__ void cluster_arrive() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  __syncwarp();
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
}
// Stores 16 bytes at the address that `p` has in block `rank` of the cluster.
__device__ __forceinline__ void cluster_store(void *p, uint32_t rank, uint64_t a, uint64_t b) {
  uint32_t at;
  asm("mapa.shared::cluster.u32 %0, %1, %2;"
      : "=r"(at)
      : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(p))), "r"(rank));
  asm volatile("st.shared::cluster.v2.b64 [%0], {%1, %2};" ::"r"(at), "l"(a), "l"(b) : "memory");
}

constexpr int kMaxCluster = 16;

// Launches `fn` with `grid` blocks in clusters of `cluster` (which divides it).
template <typename... P, typename... A>
cudaError_t launch_clusters(void (*fn)(P...), unsigned grid, int threads, int cluster, int smem,
                            cudaStream_t st, A... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(unsigned(threads));
  cfg.dynamicSmemBytes = size_t(smem);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = unsigned(cluster);
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fn, static_cast<P>(args)...);
}

// Lets `fn` have `bytes` of dynamic shared memory and clusters of more than
// eight blocks, once for each device (its bit in `allowed`; device_sms refuses
// devices above 63).
template <typename F>
cudaError_t allow(F *fn, int bytes, std::atomic<uint64_t> &allowed) {
  int dev = 0;
  if (const cudaError_t e = cudaGetDevice(&dev)) return e;
  const uint64_t bit = uint64_t(1) << (dev & 63);
  if (allowed.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  const void *f = reinterpret_cast<const void *>(fn);
  if (const cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)) return e;
  if (bytes)
    if (const cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes)) return e;
  allowed.fetch_or(bit, std::memory_order_relaxed);
  return cudaSuccess;
}

// ------------------------------------------------------------ logits
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void copy16(void *to, const void *from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                   static_cast<uint32_t>(__cvta_generic_to_shared(to))),
               "l"(from)
               : "memory");
}

template <typename T>
struct Unit {                      // 8 logits as they came
  uint4 w[sizeof(T) / 2];
  __device__ __forceinline__ uint32_t word(int k) const {
    const uint4 &v = w[k / 4];
    return k % 4 == 0 ? v.x : k % 4 == 1 ? v.y : k % 4 == 2 ? v.z : v.w;
  }
  __device__ __forceinline__ float2 pair(int k) const {       // logits 2k and 2k + 1
    if constexpr (std::is_same_v<T, float>) {
      return make_float2(__uint_as_float(word(2 * k)), __uint_as_float(word(2 * k + 1)));
    } else if constexpr (std::is_same_v<T, __nv_bfloat16>) {
      return make_float2(__uint_as_float(word(k) << 16), __uint_as_float(word(k) & 0xFFFF0000u));
    } else {
      __half2 h;
      const uint32_t v = word(k);
      memcpy(&h, &v, 4);
      return __half22float2(h);
    }
  }
};
// The largest of two, NaN where one of them is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}
// The largest of units, 16-bit logits two at a time; NaN where one of them is, so
// that the row is: no logit is the largest beside it.
template <typename T>
struct Largest {
  using Pair = std::conditional_t<std::is_same_v<T, __half>, __half2, __nv_bfloat162>;
  Pair top[2];
  __device__ __forceinline__ Largest() {
    const T low = T(-INFINITY);
    const T both[2] = {low, low};
    memcpy(&top[0], both, 4);
    top[1] = top[0];
  }
  __device__ __forceinline__ void take(const Unit<T> &v) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      Pair x;
      const uint32_t w = v.word(k);
      memcpy(&x, &w, 4);
      top[k % 2] = __hmax2_nan(top[k % 2], x);
    }
  }
  __device__ __forceinline__ float value() const {
    const Pair x = __hmax2_nan(top[0], top[1]);
    return max_nan(to_f(x.x), to_f(x.y));
  }
};
template <>
struct Largest<float> {
  float top = -INFINITY;
  __device__ __forceinline__ void take(const Unit<float> &v) {
#pragma unroll
    for (int k = 0; k < 4; ++k) top = max_nan(top, max_nan(v.pair(k).x, v.pair(k).y));
  }
  __device__ __forceinline__ float value() const { return top; }
};

// Unit u of a row whose elements are [lo, hi) of the array; elements outside
// the row read as -infinity.
template <typename T>
__device__ __forceinline__ Unit<T> load_unit(const T *x, int64_t u, int64_t lo, int64_t hi) {
  Unit<T> v;
  const int64_t e = u * 8;
  if (e >= lo && e + 8 <= hi) {
#pragma unroll
    for (int k = 0; k < int(sizeof(T) / 2); ++k) v.w[k] = __ldg(reinterpret_cast<const uint4 *>(x + e) + k);
  } else {
    T t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = e + i >= lo && e + i < hi ? x[e + i] : T(-INFINITY);
    memcpy(v.w, t, sizeof t);
  }
  return v;
}
// Stores elements r .. r + 7 of a row of V.
__device__ __forceinline__ void store_unit(float *row, int r, int V, const float2 (&y)[4]) {
  if (r >= 0 && r + 8 <= V) {
    float4 *to = reinterpret_cast<float4 *>(row + r);
    __stcs(to, make_float4(y[0].x, y[0].y, y[1].x, y[1].y));
    __stcs(to + 1, make_float4(y[2].x, y[2].y, y[3].x, y[3].y));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (r + i >= 0 && r + i < V) row[r + i] = i % 2 ? y[i / 2].y : y[i / 2].x;
  }
}

}  // namespace
}  // namespace vg
