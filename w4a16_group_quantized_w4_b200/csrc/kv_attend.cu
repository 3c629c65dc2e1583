// kv_cache_attend: argument checks, workspace and dispatch (kernels: kv_attend.cuh).
#include "kv_attend.cuh"

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
  if (!std::isfinite(scale) || !std::isfinite(softcap) || softcap < 0.f ||
      (softcap > 0.f && softcap < 1e-30f)) return W4_ERR_INVALID_ARG;
  if (head_dim != 64 && head_dim != 128 && head_dim != 192 && head_dim != 256) return W4_ERR_UNSUPPORTED;
  if (q_heads > 65536 || static_cast<int64_t>(B) * q_heads > 0x7FFFFFFFLL || pages > 0x7FFFFFFFLL ||
      static_cast<int64_t>(table_width) * page_size > at::kMostTokens ||
      static_cast<int64_t>(table_width) * page_size / at::kUnit * q_heads > 0x3FFFFFFFLL)
    return W4_ERR_UNSUPPORTED;
  // rows of the cache are counted in 32 bits (they would fill more than 128 GB)
  if (static_cast<uint64_t>(pages) * kv_heads > 0xFFFFFFFFull / page_size) return W4_ERR_UNSUPPORTED;
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
  // blocks write their heads while others still read theirs
  const uintptr_t q0 = reinterpret_cast<uintptr_t>(q), o0 = reinterpret_cast<uintptr_t>(out);
  const uint64_t row = static_cast<uint64_t>(q_heads) * head_dim * 2;
  if (o0 < q0 + static_cast<uint64_t>(B - 1) * q_stride * 2 + row && q0 < o0 + B * row) return W4_ERR_INVALID_ARG;
  at::Args a{};
  a.q = q;
  a.q_stride = q_stride;
  a.k = k_cache;
  a.v = v_cache;
  a.ks = k_scales;
  a.vs = v_scales;
  a.table = page_table;
  a.lens = seq_lens;
  a.table_width = table_width;
  a.B = B;
  a.q_heads = q_heads;
  a.kv_heads = kv_heads;
  a.page_size = page_size;
  a.pages = static_cast<int>(pages);
  a.scale = scale;
  a.softcap = softcap;
  a.window = window;
  a.out = out;
  a.lse = lse;
  a.recs = static_cast<at::Rec*>(workspace);
  a.parts = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + at::recs_bytes(device_sm_count()));
  a.dev_status = dev_status;
  a.G = q_heads / kv_heads;
  a.div_shift = 0;
  while ((1LL << a.div_shift) < page_size) ++a.div_shift;
  a.div_mul = static_cast<uint32_t>((((1ULL << a.div_shift) - page_size) << 32) / page_size + 1);
  auto s = static_cast<cudaStream_t>(stream);
  const int sms = device_sm_count();
  return w4_record_status(kind == W4_KV_BF16 ? at::launch_bf16(a, head_dim, s, sms)
                          : kind == W4_KV_INT8 ? at::launch_int8(a, head_dim, s, sms)
                                               : at::launch_int4(a, head_dim, s, sms));
}

// A record and two parts (of a block's first and last item) of 8 heads for every block of the largest grid.
size_t w4_attend_workspace_bytes(int64_t B, int64_t q_heads, int64_t head_dim, int64_t kv_heads) {
  if (B < 1 || q_heads < 1 || kv_heads < 1 || head_dim < 64 || head_dim > 256) return 0;
  const int sms = w4::device_sm_count();
  const int64_t blocks = static_cast<int64_t>(sms) * w4::at::kMostBlocks;
  return static_cast<size_t>(w4::at::recs_bytes(sms) + 2 * blocks * 8 * (head_dim + 2) * 4);
}
