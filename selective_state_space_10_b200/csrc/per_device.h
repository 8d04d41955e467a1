// per_device.h -- what the host asks the runtime about a kernel and keeps: for each kernel and device by itself.
#pragma once

#include <cuda_runtime_api.h>

#include <atomic>

namespace ssd {

// A number that is not negative, for each device.  Threads that ask at the same time both ask the runtime.
class PerDevice {
 public:
  // value: what ask(value), a cudaError_t, set it to on this device; an answer that failed is not kept.
  template <typename Ask>
  cudaError_t get(int &value, Ask ask) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const bool kept = dev >= 0 && dev < kDevices;
    if (kept) {
      const int v = held_[dev].load(std::memory_order_relaxed);
      if (v != 0) {
        value = v - 1;
        return cudaSuccess;
      }
    }
    e = ask(value);
    if (e == cudaSuccess && kept) held_[dev].store(value + 1, std::memory_order_relaxed);
    return e;
  }

 private:
  static constexpr int kDevices = 64;
  std::atomic<int> held_[kDevices] = {};  // the number + 1; 0: not asked yet
};

// How many clusters of `size` (below kSizes) CTAs of this kernel a device holds.
template <auto *kernel, int kSizes>
PerDevice &clusters_held(int size) {
  static PerDevice held[kSizes];
  return held[size];
}

}  // namespace ssd
