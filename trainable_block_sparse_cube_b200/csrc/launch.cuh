// Launches of the projection side's kernels: with much shared memory, and
// closely behind one another (the second is launched while the first still
// runs, and waits for its results itself).
#pragma once
#include <cuda_runtime.h>

#include <atomic>

namespace vsa {
namespace ptx {

// Everything that the kernels before this one in the stream wrote is visible
// after it. Before it a kernel launched by launch_behind touches no memory
// but its own shared one.
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// The kernel behind may be launched once every block has come here.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

}  // namespace ptx

// Lets kernel K have `bytes` of dynamic shared memory on the current device;
// set once a device.
template <auto K>
cudaError_t allow_smem(int bytes) {
  constexpr int kMaxDevices = 64;
  static std::atomic<bool> ready[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < kMaxDevices && ready[dev].load(std::memory_order_relaxed)) return cudaSuccess;
  e = cudaFuncSetAttribute(K, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev < kMaxDevices) ready[dev].store(true, std::memory_order_relaxed);
  return e;
}

template <typename... P, typename... A>
cudaError_t launch_behind(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, A... args) {
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c{};
  c.gridDim = grid;
  c.blockDim = block;
  c.dynamicSmemBytes = smem;
  c.stream = st;
  c.attrs = &at;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, kernel, args...);
}

}  // namespace vsa
