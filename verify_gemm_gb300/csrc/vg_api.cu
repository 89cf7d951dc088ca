// vg_api.cu -- status strings, version and CUDA error capture of the C ABI.
#include <cuda_runtime.h>

#include <atomic>
#include <cstdio>
#include <mutex>

#include "vg_internal.h"

namespace vg {
namespace {
thread_local char g_last_error[256] = "";
}

void set_cuda_error(cudaError_t e) {
  const char *name = cudaGetErrorName(e);
  const char *msg = cudaGetErrorString(e);
  std::snprintf(g_last_error, sizeof g_last_error, "%s: %s", name ? name : "?", msg ? msg : "?");
}

PFN_cuTensorMapEncodeTiled_v12000 encode_tiled() {
  static std::once_flag once;
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  std::call_once(once, [] {
    void *ptr = nullptr;
    cudaDriverEntryPointQueryResult q{};
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    else
      cudaGetLastError();
  });
  return fn;
}

vg_status device_sms(int *sms) {
  // a property of the device, looked up once for each; 0: not looked up yet
  static std::atomic<int> known[64];
  int dev = 0;
  VG_CUDA(cudaGetDevice(&dev));
  if (dev < 0 || dev >= 64) return VG_ERR_UNSUPPORTED;
  int n = known[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    int major = 0, minor = 0;
    VG_CUDA(cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev));
    VG_CUDA(cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev));
    VG_CUDA(cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev));
    if (major * 10 + minor != 103) return VG_ERR_UNSUPPORTED;
    known[dev].store(n, std::memory_order_relaxed);
  }
  *sms = n;
  return VG_OK;
}
}  // namespace vg

extern "C" const char *vg_status_string(vg_status s) {
  switch (s) {
    case VG_OK: return "ok";
    case VG_ERR_INVALID_ARG: return "invalid argument";
    case VG_ERR_ALIGNMENT: return "device pointer not 16-byte aligned";
    case VG_ERR_UNSUPPORTED: return "unsupported device or size";
    case VG_ERR_CUDA: return "CUDA error";
    case VG_ERR_TIMEOUT: return "device-side wait timed out";
    case VG_ERR_WORKSPACE: return "workspace missing or too small";
  }
  return "unknown status";
}

extern "C" int vg_version(void) { return 100; }

extern "C" const char *vg_last_cuda_error(void) { return vg::g_last_error; }
