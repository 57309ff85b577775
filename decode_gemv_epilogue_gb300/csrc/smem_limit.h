// The shared memory that a kernel's launches may ask for.
#pragma once

#include <atomic>
#include <mutex>

#include <cuda_runtime.h>

namespace gf {

// One per kernel.  raise() lets the kernel's launches on the current device have all the shared
// memory that the device offers a block, once; nothing ever lowers it, whichever thread launches
// which size first.
class SmemLimit {
 public:
  cudaError_t raise(const void* kernel) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const bool kept = dev >= 0 && dev < kDevices;
    if (kept && done_[dev].load(std::memory_order_acquire)) return cudaSuccess;
    std::lock_guard<std::mutex> lock(mu_);
    if (kept && done_[dev].load(std::memory_order_relaxed)) return cudaSuccess;
    int most = 0;
    e = cudaDeviceGetAttribute(&most, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
    if (e != cudaSuccess) return e;
    cudaFuncAttributes f;
    e = cudaFuncGetAttributes(&f, kernel);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most - static_cast<int>(f.sharedSizeBytes));
    if (e == cudaSuccess && kept) done_[dev].store(true, std::memory_order_release);
    return e;
  }

 private:
  static constexpr int kDevices = 64;
  std::mutex mu_;
  std::atomic<bool> done_[kDevices] = {};
};

}  // namespace gf
