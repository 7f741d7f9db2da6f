// The opt-in to more than 48 KB of dynamic shared memory: a kernel needs it once on every device.
#pragma once
#include <atomic>
#include <cuda_runtime.h>

namespace tt {

// `done` is the kernel's own word (static, zero at first): bit d says that device d has it.
inline cudaError_t smem_opt_in(const void* kernel, int bytes, std::atomic<unsigned long long>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

}  // namespace tt
