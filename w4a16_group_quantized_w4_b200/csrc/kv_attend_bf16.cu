// kv_cache_attend's kernels over a bf16 cache (see kv_attend.cuh).
#include "kv_attend.cuh"

w4_status w4::at::launch_bf16(const Args& a, int D, cudaStream_t s, int sms) {
  return launch_kind<W4_KV_BF16>(a, D, s, sms);
}
