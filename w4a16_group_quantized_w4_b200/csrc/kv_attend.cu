// kv_cache_attend: attention of one new token per sequence over a paged key/value cache.
//
// First form: one block per (sequence, query head); each of four warps walks every fourth token with
// a running maximum and sum, and the four partial results are joined in shared memory.
#include "common.cuh"
#include "entry.cuh"

namespace w4 {
namespace at {

struct Args {
  const uint16_t* q;
  int64_t q_stride;
  const void *k, *v;
  const uint16_t *ks, *vs;
  const int32_t *table, *lens;
  int table_width, B, q_heads, kv_heads, page_size;
  int64_t pages;
  float scale, softcap;
  int window;
  uint16_t* out;
  float* lse;
  int32_t* dev_status;
};

template <int KIND, int D>
__device__ __forceinline__ float elem(const void* cache, const uint16_t* scales, int64_t row, int d) {
  if (KIND == W4_KV_BF16) return bf16_lo_to_f32(reinterpret_cast<const uint16_t*>(cache)[row * D + d]);
  const float s = bf16_lo_to_f32(scales[row * (D / 32) + (d >> 5)]);
  if (KIND == W4_KV_INT8) return static_cast<float>(reinterpret_cast<const int8_t*>(cache)[row * D + d]) * s;
  const uint32_t w = reinterpret_cast<const uint32_t*>(cache)[row * (D / 8) + (d >> 3)];
  return static_cast<float>(static_cast<int>((w >> (4 * (d & 7))) & 15u) - 8) * s;
}

template <int KIND, int D>
__global__ void __launch_bounds__(128) attend_kernel(Args a) {
  __shared__ float s_o[4][D], s_m[4], s_l[4];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = blockIdx.x / a.q_heads, hq = blockIdx.x % a.q_heads;
  const int hk = hq / (a.q_heads / a.kv_heads);
  int64_t len = a.lens[b];
  const int64_t most = static_cast<int64_t>(a.table_width) * a.page_size;
  if (len > most || len < 0) {
    if (threadIdx.x == 0) set_status(a.dev_status, W4_ERR_INVALID_ARG);
    len = len < 0 ? 0 : most;
  }
  const int64_t first = a.window > 0 && len > a.window ? len - a.window : 0;
  float qv[D / 32], o[D / 32];
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    qv[i] = bf16_lo_to_f32(a.q[b * a.q_stride + static_cast<int64_t>(hq) * D + i * 32 + lane]);
    o[i] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int64_t t = first + warp; t < len; t += 4) {
    const int page = a.table[static_cast<int64_t>(b) * a.table_width + t / a.page_size];
    if (page < 0 || page >= a.pages) { set_status(a.dev_status, W4_ERR_INVALID_ARG); continue; }
    const int64_t row = (static_cast<int64_t>(page) * a.kv_heads + hk) * a.page_size + t % a.page_size;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) s = fmaf(qv[i], elem<KIND, D>(a.k, a.ks, row, i * 32 + lane), s);
#pragma unroll
    for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    s *= a.scale;
    if (a.softcap > 0.f) s = a.softcap * tanhf(s / a.softcap);
    const float mn = fmaxf(m, s);
    const float alpha = __expf(m - mn), p = __expf(s - mn);
    m = mn;
    l = l * alpha + p;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) o[i] = fmaf(p, elem<KIND, D>(a.v, a.vs, row, i * 32 + lane), o[i] * alpha);
  }
#pragma unroll
  for (int i = 0; i < D / 32; ++i) s_o[warp][i * 32 + lane] = o[i];
  if (lane == 0) { s_m[warp] = m; s_l[warp] = l; }
  __syncthreads();
  float mm = -INFINITY, ll = 0.f;
  for (int w = 0; w < 4; ++w) mm = fmaxf(mm, s_m[w]);
  float f[4];
  for (int w = 0; w < 4; ++w) {
    f[w] = s_m[w] == -INFINITY ? 0.f : __expf(s_m[w] - mm);
    ll += f[w] * s_l[w];
  }
  for (int d = threadIdx.x; d < D; d += 128) {
    float x = 0.f;
    for (int w = 0; w < 4; ++w) x = fmaf(f[w], s_o[w][d], x);
    a.out[(static_cast<int64_t>(b) * a.q_heads + hq) * D + d] = f32_to_bf16_bits(ll > 0.f ? x / ll : 0.f);
  }
  if (a.lse && threadIdx.x == 0) a.lse[static_cast<int64_t>(b) * a.q_heads + hq] = ll > 0.f ? mm + logf(ll) : -INFINITY;
}

template <int KIND>
bool launch_kind(const Args& a, int D, cudaStream_t s) {
  const unsigned grid = static_cast<unsigned>(a.B) * a.q_heads;
  switch (D) {
    case 64: attend_kernel<KIND, 64><<<grid, 128, 0, s>>>(a); return true;
    case 128: attend_kernel<KIND, 128><<<grid, 128, 0, s>>>(a); return true;
    case 192: attend_kernel<KIND, 192><<<grid, 128, 0, s>>>(a); return true;
    case 256: attend_kernel<KIND, 256><<<grid, 128, 0, s>>>(a); return true;
    default: return false;
  }
}

}  // namespace at
}  // namespace w4

extern "C" w4_status kv_cache_attend(const uint16_t* q, int64_t q_stride, const void* k_cache, const void* v_cache,
                                     const uint16_t* k_scales, const uint16_t* v_scales, int32_t kind,
                                     const int32_t* page_table, int32_t table_width, const int32_t* seq_lens,
                                     int32_t B, int32_t q_heads, int32_t kv_heads, int32_t head_dim, int64_t pages,
                                     int32_t page_size, float scale, float softcap, int32_t window, uint16_t* out,
                                     float* lse, void* workspace, size_t workspace_bytes, int32_t* dev_status,
                                     void* stream) {
  using namespace w4;
  const EntryRange range("kv_cache_attend");
  if (kind != W4_KV_BF16 && kind != W4_KV_INT8 && kind != W4_KV_INT4) return W4_ERR_INVALID_ARG;
  if (B < 0 || q_heads < 1 || kv_heads < 1 || q_heads % kv_heads || head_dim < 1 || pages < 1 || page_size < 1 ||
      table_width < 1 || window < 0)
    return W4_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || !std::isfinite(softcap) || softcap < 0.f) return W4_ERR_INVALID_ARG;
  if (head_dim != 64 && head_dim != 128 && head_dim != 192 && head_dim != 256) return W4_ERR_UNSUPPORTED;
  if (q_heads > 65536 || static_cast<int64_t>(B) * q_heads > 0x7FFFFFFFLL || pages > 0x7FFFFFFFLL ||
      static_cast<int64_t>(table_width) * page_size > 0x7FFFFFFFLL)
    return W4_ERR_UNSUPPORTED;
  if (q_stride < static_cast<int64_t>(q_heads) * head_dim || q_stride % 8) return W4_ERR_INVALID_ARG;
  if (!k_cache || !v_cache || !aligned_to(k_cache, 16) || !aligned_to(v_cache, 16)) return W4_ERR_INVALID_ARG;
  if (kind != W4_KV_BF16 && (!k_scales || !v_scales || !aligned_to(k_scales, 16) || !aligned_to(v_scales, 16)))
    return W4_ERR_INVALID_ARG;
  if (B == 0) return W4_OK;
  if (!q || !page_table || !seq_lens || !out || !aligned_to(q, 16) || !aligned_to(out, 16) ||
      !aligned_to(page_table, 4) || !aligned_to(seq_lens, 4) || !aligned_to(lse, 4) || !aligned_to(workspace, 16))
    return W4_ERR_INVALID_ARG;
  if (workspace_bytes < w4_workspace_bytes(W4_OP_ATTEND, B, q_heads, head_dim, kv_heads, 0) ||
      (!workspace && w4_workspace_bytes(W4_OP_ATTEND, B, q_heads, head_dim, kv_heads, 0)))
    return W4_ERR_WORKSPACE;
  const at::Args a{q, q_stride, k_cache, v_cache, k_scales, v_scales, page_table, seq_lens, table_width, B, q_heads,
                   kv_heads, page_size, pages, scale, softcap, window, out, lse, dev_status};
  auto s = static_cast<cudaStream_t>(stream);
  if (kind == W4_KV_BF16) at::launch_kind<W4_KV_BF16>(a, head_dim, s);
  else if (kind == W4_KV_INT8) at::launch_kind<W4_KV_INT8>(a, head_dim, s);
  else at::launch_kind<W4_KV_INT4>(a, head_dim, s);
  return launched();
}

size_t w4_attend_workspace_bytes(int64_t, int64_t, int64_t, int64_t) { return 0; }
