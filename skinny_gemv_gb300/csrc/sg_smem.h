// Dynamic shared memory past 48 KB has to be allowed per kernel and per device: the
// attribute belongs to the function as loaded on the current device.
#pragma once

#include <cuda_runtime_api.h>

#include <atomic>
#include <cstdint>

namespace sg {

// One bit per device (the library takes devices 0 to 63).
using DeviceBits = std::atomic<uint64_t>;

// Allows `kernel` `bytes` of dynamic shared memory on the current device, unless `done`
// says that it has been.
inline cudaError_t allow_dynamic_smem(const void* kernel, int bytes, DeviceBits* done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = uint64_t(1) << (dev & 63);
  if (done->load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done->fetch_or(bit, std::memory_order_release);
  return e;
}

}  // namespace sg
