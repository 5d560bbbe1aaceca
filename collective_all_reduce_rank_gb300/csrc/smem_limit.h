// smem_limit.h -- the dynamic shared memory limit of a kernel.  The runtime
// keeps it per device, so it is raised once on each device that launches the
// kernel; what is kept here says on which it was.
#pragma once

#include <cuda_runtime_api.h>

#include <atomic>

namespace rra {

class SmemLimit {
 public:
  // For the current device.  Two threads may both raise it: it is the same limit.
  cudaError_t raise(const void* kernel, int bytes) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const bool kept = dev >= 0 && dev < kDevices;
    if (kept && raised_[dev].load(std::memory_order_relaxed)) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && kept) raised_[dev].store(true, std::memory_order_relaxed);
    return e;
  }

 private:
  static constexpr int kDevices = 64;
  std::atomic<bool> raised_[kDevices] = {};
};

// One limit per kernel (K is the kernel itself).
template <auto K>
cudaError_t raise_smem(int bytes) {
  static SmemLimit limit;
  return limit.raise(reinterpret_cast<const void*>(K), bytes);
}

}  // namespace rra
