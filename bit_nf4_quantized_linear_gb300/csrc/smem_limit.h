// smem_limit.h -- a kernel's limit of dynamic shared memory, set once a device.
#pragma once

#include <cuda_runtime_api.h>

#include <atomic>
#include <cstdint>

namespace nf4 {

// One per kernel.  The limit belongs to the kernel in a device's context, so each device
// needs it once; devices past the 64 flags get it with every launch.  Threads may race: a
// flag is only up once its device's limit stands.
class SmemLimit {
 public:
  template <typename Kernel>
  cudaError_t allow(Kernel kern, int bytes) {
    int dev = 0;
    if (cudaError_t e = cudaGetDevice(&dev)) return e;
    const uint64_t flag = dev < 64 ? uint64_t{1} << dev : 0;
    if (set_.load(std::memory_order_relaxed) & flag) return cudaSuccess;
    if (cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void*>(kern), cudaFuncAttributeMaxDynamicSharedMemorySize, bytes))
      return e;
    set_.fetch_or(flag, std::memory_order_relaxed);
    return cudaSuccess;
  }

 private:
  std::atomic<uint64_t> set_{0};
};

}  // namespace nf4
