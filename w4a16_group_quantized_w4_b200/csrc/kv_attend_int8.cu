// kv_cache_attend's kernels over a int8 cache (see kv_attend.cuh).
#include "kv_attend.cuh"

w4_status w4::at::launch_int8(const Args& a, int D, cudaStream_t s, int sms) {
  return launch_kind<W4_KV_INT8>(a, D, s, sms);
}
