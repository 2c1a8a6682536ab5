// What holds for one device and not for the process: cudaFuncSetAttribute and occupancies are the current device's.
// Declared before: the CUDA runtime's (tests/device_host.cpp puts its own in their place).
#pragma once
#include <atomic>

namespace moe {

constexpr int kDevices = 64;  // devices that are remembered; past them nothing is, and everything is set each time

// A number per device, 0 until it is stored.
class PerDevice {
 public:
  // The current device's, or null past kDevices.
  cudaError_t here(std::atomic<int>** at) {
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    *at = e == cudaSuccess && dev >= 0 && dev < kDevices ? &of_[dev] : nullptr;
    return e;
  }

 private:
  std::atomic<int> of_[kDevices] = {};
};

// A kernel's opt-in to `bytes` of dynamic shared memory, on each device before its first launch there.
class SmemOptIn {
 public:
  template <class Kernel>
  cudaError_t operator()(Kernel* kernel, int bytes) {
    std::atomic<int>* set;
    cudaError_t e = on_.here(&set);
    if (e != cudaSuccess || (set && set->load(std::memory_order_relaxed))) return e;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && set) set->store(1, std::memory_order_relaxed);
    return e;
  }

 private:
  PerDevice on_;
};

}  // namespace moe
