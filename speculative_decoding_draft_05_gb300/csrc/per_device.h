// per_device.h -- what is found out once: once for each device.  A function's attributes
// (its shared memory, its carveout) hold for the device that was current when they were
// set, and devices may differ in their sizes.
#pragma once

#include <cuda_runtime.h>

#include <atomic>

namespace dspark {

constexpr int kMaxDevices = 64;  // past that number a result is not kept

// set(), which returns a cudaError_t, once for each device that is current here, and again
// where it failed.  (By F, a lambda's own type: each place, in each instance of a template,
// has results of its own.  Two threads may both call it; what it sets is the same.)
template <typename F>
cudaError_t once_per_device(F set) {
  static std::atomic<bool> done[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const bool kept = dev >= 0 && dev < kMaxDevices;
  if (kept && done[dev].load(std::memory_order_acquire)) return cudaSuccess;
  e = set();
  if (e == cudaSuccess && kept) done[dev].store(true, std::memory_order_release);
  return e;
}

// An attribute of the current device; 1 where it cannot be had, or is less.
template <cudaDeviceAttr A>
int device_attribute() {
  static std::atomic<int> known[kMaxDevices];
  int dev = 0, v = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 1;
  const bool kept = dev >= 0 && dev < kMaxDevices;
  if (kept && (v = known[dev].load(std::memory_order_relaxed)) > 0) return v;
  if (cudaDeviceGetAttribute(&v, A, dev) != cudaSuccess || v <= 0) return 1;
  if (kept) known[dev].store(v, std::memory_order_relaxed);
  return v;
}

inline int device_sms() { return device_attribute<cudaDevAttrMultiProcessorCount>(); }

// Dynamic shared memory above 48 KB.
template <typename K>
cudaError_t allow_smem(K kernel, int bytes) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

}  // namespace dspark
