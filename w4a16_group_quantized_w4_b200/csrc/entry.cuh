// Host helpers of the entry points that live beside their kernels: the named profiler range,
// pointer checks and the device's SM count.
#pragma once

#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include <cmath>
#include <cstdint>

#include "../../include/w4a16.h"

// records the CUDA error behind a W4_ERR_CUDA for w4_last_cuda_error (api.cu)
w4_status w4_record_status(w4_status s);

namespace w4 {

struct EntryRange {
  explicit EntryRange(const char* name) { nvtxRangePushA(name); }
  ~EntryRange() { nvtxRangePop(); }
  EntryRange(const EntryRange&) = delete;
  EntryRange& operator=(const EntryRange&) = delete;
};

inline bool aligned_to(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline w4_status launched() {
  return w4_record_status(cudaGetLastError() == cudaSuccess ? W4_OK : W4_ERR_CUDA);
}

inline int device_sm_count() {
  static int cached[64] = {0};
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 148;
  if (dev < 64 && cached[dev]) return cached[dev];
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) n = 148;
  if (dev < 64) cached[dev] = n;
  return n;
}

// Raises a kernel's limit of dynamic shared memory to `bytes`, once per device and value.
// `raised` is the kernel's own static table.
struct SmemRaised {
  int bytes[64] = {0};
};
template <typename F>
inline cudaError_t raise_smem(F* kernel, int bytes, SmemRaised& raised) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 64 && raised.bytes[dev] >= bytes) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev < 64) raised.bytes[dev] = bytes;
  return e;
}

}  // namespace w4
