// device_once.h -- setup that belongs to a device, done once on each, and numbers
// that a device is asked for, once each.
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

// N numbers (of 0 or more) that depend on the device and on what the owner of the object
// asks: one object a kernel.  What could not be answered counts as 0 and is asked again.
template <int N>
class DeviceAnswers {
 public:
  // ask(int&) -> cudaError_t, unless number i of the current device is known.
  template <typename Ask>
  int get(int i, Ask ask) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    const bool kept = dev >= 0 && dev < kDevices;
    if (kept)
      if (const int known = known_[dev][i].load(std::memory_order_relaxed); known > 0) return known - 1;
    int n = 0;
    if (ask(n) != cudaSuccess) return 0;
    if (kept) known_[dev][i].store(n + 1, std::memory_order_relaxed);
    return n;
  }

 private:
  static constexpr int kDevices = 64;
  std::atomic<int> known_[kDevices][N] = {};  // the number + 1; 0: not known yet
};

}  // namespace gqa
