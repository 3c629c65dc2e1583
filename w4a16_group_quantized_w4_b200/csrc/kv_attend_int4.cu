// kv_cache_attend's kernels over a int4 cache (see kv_attend.cuh).
#include "kv_attend.cuh"

w4_status w4::at::launch_int4(const Args& a, int D, cudaStream_t s, int sms) {
  return launch_kind<W4_KV_INT4>(a, D, s, sms);
}
