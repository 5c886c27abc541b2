// A step that each device needs once before its first use (function attributes,
// addresses of device symbols).
#pragma once

#include <cuda_runtime.h>

#include <atomic>
#include <mutex>

namespace dlm {

constexpr int kMaxDeviceOnce = 64;

// Success is remembered; after a failure (memory that was short while a module was
// loaded) the next call tries again.
class DeviceOnce {
 public:
  template <typename F>
  cudaError_t get(F&& f) {
    int dev = 0;
    if (cudaError_t e = cudaGetDevice(&dev); e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDeviceOnce) return cudaErrorInvalidDevice;
    if (done_[dev].load(std::memory_order_acquire)) return cudaSuccess;
    std::lock_guard<std::mutex> lock(one_);
    if (done_[dev].load(std::memory_order_relaxed)) return cudaSuccess;
    const cudaError_t e = f();
    if (e == cudaSuccess) done_[dev].store(true, std::memory_order_release);
    return e;
  }

 private:
  std::atomic<bool> done_[kMaxDeviceOnce] = {};
  std::mutex one_;
};

}  // namespace dlm
