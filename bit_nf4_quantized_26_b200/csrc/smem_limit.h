// smem_limit.h — raising a kernel's limit of dynamic shared memory (host code
// of the runtime API only).
#pragma once

#include <cuda_runtime_api.h>

#include <cstdint>

namespace qnf4 {

// Raises `kernel`'s limit once per device: a kernel's attributes belong to the
// device that is current when they are set.  `done` holds a bit per device and
// is the kernel's own; threads that race set the same value twice.
inline cudaError_t allow_smem(const void* kernel, uint32_t bytes, uint64_t& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = uint64_t(1) << (dev & 63);
  if (__atomic_load_n(&done, __ATOMIC_RELAXED) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
  if (e == cudaSuccess) __atomic_fetch_or(&done, bit, __ATOMIC_RELAXED);
  return e;
}

template <typename... KArgs>
inline cudaError_t allow_smem(void (*kernel)(KArgs...), uint32_t bytes, uint64_t& done) {
  return allow_smem(reinterpret_cast<const void*>(kernel), bytes, done);
}

}  // namespace qnf4
