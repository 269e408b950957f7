// device_once.h -- setup that belongs to a device, done once on each.
//
// A kernel's attributes (its dynamic shared memory above 48 KB, its carveout)
// are set for the current device only, so a process that calls the library on
// several devices sets them on each.  A device on which that failed is asked
// again by the next call, and says nothing about the others.
#pragma once

#include <cuda_runtime.h>

#include <atomic>
#include <mutex>

namespace gqa {

class DeviceOnce {
 public:
  // Runs setup() (a cudaError_t) unless it has succeeded on the current device.
  template <typename Setup>
  cudaError_t run(Setup setup) {
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kDevices) return setup();  // (more than are kept: each time)
    if (done_[dev].load(std::memory_order_acquire)) return cudaSuccess;
    std::lock_guard<std::mutex> lock(mu_);
    if (done_[dev].load(std::memory_order_relaxed)) return cudaSuccess;
    const cudaError_t r = setup();
    if (r == cudaSuccess) done_[dev].store(true, std::memory_order_release);
    return r;
  }

 private:
  static constexpr int kDevices = 64;
  std::mutex mu_;
  std::atomic<bool> done_[kDevices] = {};
};

}  // namespace gqa
