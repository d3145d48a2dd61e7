// Host-side helpers shared by the files that implement the C ABI.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <mutex>

#include "../../include/vsa.h"

namespace vsa {

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn get_encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  // The encoder fails in a host thread without a current context, which one
  // that has made no call of the runtime before is; cudaSetDevice makes it so.
  thread_local bool bound = false;
  int dev = 0;
  if (!bound) bound = cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(dev) == cudaSuccess;
  return fn;
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// A strided [B, heads, N, D] tensor of `elem`-byte elements.
inline vsa_status check_heads(const vsa_heads* x, int B, int N, int elem, bool written) {
  if (x->heads < 0) return VSA_ERR_SHAPE;
  if (x->heads > 65535) return VSA_ERR_UNSUPPORTED;
  if (!B || !N || !x->heads) return VSA_OK;
  if (!x->data) return VSA_ERR_INVALID_ARG;
  if (!aligned16(x->data)) return VSA_ERR_ALIGN;
  const int len[3] = {B, x->heads, N};
  const long long stride[3] = {x->s_b, x->s_h, x->s_n};
  for (int i = 0; i < 3; ++i)
    if (len[i] > 1) {
      if (stride[i] < 0 || (written && stride[i] == 0)) return VSA_ERR_INVALID_ARG;
      if (stride[i] >= (1LL << 40)) return VSA_ERR_UNSUPPORTED;
      if (stride[i] * elem % 16) return VSA_ERR_ALIGN;
    }
  return VSA_OK;
}

// SM count of the current device, or an error if it is not an sm_100 part.
// The attributes of a device are read once.
inline vsa_status current_device_sms(int* sms) {
  constexpr int kMaxDevices = 64;
  static std::atomic<int> known[kMaxDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return VSA_ERR_CUDA;
  if (dev >= 0 && dev < kMaxDevices && (*sms = known[dev].load(std::memory_order_relaxed)) > 0) return VSA_OK;
  int major = 0;
  if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess) return VSA_ERR_CUDA;
  if (major != 10) return VSA_ERR_DEVICE;
  if (cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return VSA_ERR_CUDA;
  if (dev >= 0 && dev < kMaxDevices) known[dev].store(*sms, std::memory_order_relaxed);
  return VSA_OK;
}

}  // namespace vsa
