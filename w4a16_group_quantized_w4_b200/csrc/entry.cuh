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

}  // namespace w4
