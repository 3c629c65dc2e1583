// kv_cache_write, kv_cache_read: rows of a paged key/value cache, quantised as they are written and
// turned back into bf16 as they are read.
//
// A cache row is one token's head_dim values of one head.  Groups of 32 along head_dim share one bf16
// scale, as everywhere in this library:
//   int8: s = bf16(max|x| / 127), q = rint(x / s) in -127..127;   int4: s = bf16(max|x| / 7), q in -7..7.
// Both operands of the quotient have 8-bit significands, so it either is a half-integer or lies at least
// 2^-16 of its value away from one: a float32 quotient with a Newton step (exact where the quotient is
// representable, which half-integers are) gives the codes of exact arithmetic.
//
// Bound by memory.  A thread moves 8 elements of the key row and the 8 beside them of the value row, for
// kTokens tokens (independent 16-byte loads or stores); four neighbouring threads share a group, so its
// maximum takes two shuffles.  Measured (8192 tokens, 8 heads of 128): a division per element takes 23 us
// to write int8, the multiplication by 1 / s with its step FIGW; reading 32768 such rows takes FIGR us.
#include "common.cuh"
#include "entry.cuh"

namespace w4 {
namespace kv {

struct Shape {
  int64_t T, pages;
  int heads, dim, page_size, chunks;   // chunks = heads * dim / 8 per token
};

// Cache row index ((page * heads) * page_size + offset, for head 0) of a slot; -1 for none.
__device__ __forceinline__ int64_t slot_row(int64_t slot, const Shape& s, int32_t* dev_status) {
  if (slot < 0) return -1;
  if (slot >= s.pages * s.page_size) { set_status(dev_status, W4_ERR_INVALID_ARG); return -1; }
  int64_t page;
  int off;
  if ((slot >> 32) == 0) {
    page = static_cast<uint32_t>(slot) / static_cast<uint32_t>(s.page_size);
    off = static_cast<int>(static_cast<uint32_t>(slot) - static_cast<uint32_t>(page) * s.page_size);
  } else {
    page = slot / s.page_size;
    off = static_cast<int>(slot - page * s.page_size);
  }
  return page * s.heads * s.page_size + off;
}

constexpr int kTokens = 2;

// rint(x / s) + bias in the low bits of a float of 1.5 * 2^23 and more; s positive and normal, inv = 1 / s
__device__ __forceinline__ uint32_t quotient(float x, float s, float inv, float bias) {
  const float q = x * inv;
  return __float_as_uint(fmaf(fmaf(-q, s, x), inv, q) + (12582912.f + bias));
}
// the low bytes of four words
__device__ __forceinline__ uint32_t low_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// 8 bf16 of a group quartet -> codes (2 words int8, 1 word int4) and, in lane 0 of the four, the scale.
template <int KIND>
__device__ __forceinline__ uint32_t quantise8(const uint4& x, uint32_t (&o)[2]) {
  constexpr int kTop = KIND == W4_KV_INT8 ? 127 : 7;
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) m = max(m, max(w[j] & 0x7FFFu, (w[j] >> 16) & 0x7FFFu));
  const uint32_t quad = 0xFu << ((threadIdx.y * blockDim.x + threadIdx.x) & 28);
  m = max(m, __shfl_xor_sync(quad, m, 1));
  m = max(m, __shfl_xor_sync(quad, m, 2));
  o[0] = KIND == W4_KV_INT4 ? 0x88888888u : 0u;
  o[1] = 0u;
  if (m >= 0x7F80u) return 0x7FC0u;                       // NaN or infinity: codes 0, scale NaN
  const uint32_t sb = f32_to_bf16_bits(__fdiv_rn(bf16_lo_to_f32(m), static_cast<float>(kTop)));
  const float s = bf16_lo_to_f32(sb);
  if (s == 0.f) return 0u;
  uint32_t c[8];                                          // codes (int4: plus 8) in the low bits
  constexpr float kBias = KIND == W4_KV_INT4 ? 8.f : 0.f;
  if (s >= 0x1p-100f) {
    // Rounding max / top to bf16 takes off at most 2^-8 of a scale of 1: |x / s| <= top (1 + 2^-8) < top + 1/2,
    // so nothing has to be clamped.
    const float inv = __frcp_rn(s);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      c[2 * j] = quotient(bf16_lo_to_f32(w[j]), s, inv, kBias);
      c[2 * j + 1] = quotient(bf16_hi_to_f32(w[j]), s, inv, kBias);
    }
  } else {                                                // (a subnormal step can be far below max / top)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float x = j & 1 ? bf16_hi_to_f32(w[j >> 1]) : bf16_lo_to_f32(w[j >> 1]);
      c[j] = static_cast<uint32_t>(max(-kTop, min(kTop, __float2int_rn(__fdiv_rn(x, s)))) + static_cast<int>(kBias));
    }
  }
  if (KIND == W4_KV_INT8) {
    o[0] = low_bytes(c[0], c[1], c[2], c[3]);
    o[1] = low_bytes(c[4], c[5], c[6], c[7]);
  } else {
    o[0] = (low_bytes(c[0], c[2], c[4], c[6]) & 0x0F0F0F0Fu) | ((low_bytes(c[1], c[3], c[5], c[7]) & 0x0F0F0F0Fu) << 4);
  }
  return sb;
}

template <int KIND>
__device__ __forceinline__ void store_row8(const uint4& x, int64_t row, int dim, int d8, void* cache,
                                           uint16_t* scales) {
  if (KIND == W4_KV_BF16) {
    reinterpret_cast<uint4*>(cache)[row * (dim >> 3) + d8] = x;
    return;
  }
  uint32_t o[2];
  const uint32_t sb = quantise8<KIND>(x, o);
  if (KIND == W4_KV_INT8) reinterpret_cast<uint2*>(cache)[row * (dim >> 3) + d8] = make_uint2(o[0], o[1]);
  else reinterpret_cast<uint32_t*>(cache)[row * (dim >> 3) + d8] = o[0];
  if ((d8 & 3) == 0) scales[row * (dim >> 5) + (d8 >> 2)] = static_cast<uint16_t>(sb);
}

// blockDim = (chunks of a token handled at once, a multiple of 4; tokens), so a group's four threads are
// neighbours in one warp; what they branch on (the token, its slot) is the same for all four.
template <int KIND>
__global__ void __launch_bounds__(256)
write_kernel(const uint16_t* __restrict__ k, const uint16_t* __restrict__ v, int64_t k_stride, int64_t v_stride,
             const int64_t* __restrict__ slots, Shape s, void* k_cache, void* v_cache, uint16_t* k_scales,
             uint16_t* v_scales, int32_t* dev_status) {
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * blockDim.y * kTokens + threadIdx.y;
  int64_t row0[kTokens];
#pragma unroll
  for (int i = 0; i < kTokens; ++i) {
    const int64_t t = t0 + i * static_cast<int>(blockDim.y);
    row0[i] = t < s.T ? slot_row(__ldg(slots + t), s, dev_status) : -1;
  }
  const int per_head = s.dim >> 3;
  for (int c = threadIdx.x; c < s.chunks; c += blockDim.x) {
    const int head = c / per_head, d8 = c - head * per_head;
    uint4 kx[kTokens], vx[kTokens];
#pragma unroll
    for (int i = 0; i < kTokens; ++i) {
      if (row0[i] < 0) continue;
      const int64_t t = t0 + i * static_cast<int>(blockDim.y);
      kx[i] = __ldg(reinterpret_cast<const uint4*>(k + t * k_stride) + c);
      vx[i] = __ldg(reinterpret_cast<const uint4*>(v + t * v_stride) + c);
    }
#pragma unroll
    for (int i = 0; i < kTokens; ++i) {
      if (row0[i] < 0) continue;
      const int64_t row = row0[i] + static_cast<int64_t>(head) * s.page_size;
      store_row8<KIND>(kx[i], row, s.dim, d8, k_cache, k_scales);
      store_row8<KIND>(vx[i], row, s.dim, d8, v_cache, v_scales);
    }
  }
}

// 8 elements of a cache row as they are held
template <int KIND>
struct Raw {
  uint32_t w[KIND == W4_KV_BF16 ? 4 : KIND == W4_KV_INT8 ? 2 : 1];
  uint16_t scale;
};
template <int KIND>
__device__ __forceinline__ Raw<KIND> load_row8(int64_t row, int dim, int d8, const void* cache, const uint16_t* scales) {
  Raw<KIND> r;
  const int64_t at = row * (dim >> 3) + d8;
  if constexpr (KIND == W4_KV_BF16) {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(cache) + at);
    r.w[0] = v.x; r.w[1] = v.y; r.w[2] = v.z; r.w[3] = v.w;
  } else if constexpr (KIND == W4_KV_INT8) {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(cache) + at);
    r.w[0] = v.x; r.w[1] = v.y;
  } else {
    r.w[0] = __ldg(reinterpret_cast<const uint32_t*>(cache) + at);
  }
  if constexpr (KIND != W4_KV_BF16) r.scale = __ldg(scales + row * (dim >> 5) + (d8 >> 2));
  return r;
}

// Codes become floats through the low byte of 2^23 (0x4B0000uu is 2^23 + u), which costs a byte permute
// and a subtraction; code * scale is exact in float32 (at most 7 + 8 bits) and rounded once.
template <int KIND>
__device__ __forceinline__ uint4 values8(const Raw<KIND>& r) {
  if constexpr (KIND == W4_KV_BF16) {
    return make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
  } else {
    const float s = bf16_lo_to_f32(r.scale);
    constexpr float kBias = 8388608.f + (KIND == W4_KV_INT8 ? 128.f : 8.f);
    uint32_t u[2];                                        // bytes: elements 0..3, 4..7 (int8), even, odd (int4)
    if constexpr (KIND == W4_KV_INT8) {
      u[0] = r.w[0] ^ 0x80808080u;
      u[1] = r.w[1] ^ 0x80808080u;
    } else {
      u[0] = r.w[0] & 0x0F0F0F0Fu;
      u[1] = (r.w[0] >> 4) & 0x0F0F0F0Fu;
    }
    float f[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t word = KIND == W4_KV_INT8 ? u[j >> 2] : u[j & 1];
      const int byte = KIND == W4_KV_INT8 ? j & 3 : j >> 1;
      f[j] = (__uint_as_float(__byte_perm(word, 0x4B000000u, 0x7440 | byte)) - kBias) * s;
    }
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
  }
}

template <int KIND>
__global__ void __launch_bounds__(256)
read_kernel(const int64_t* __restrict__ slots, Shape s, const void* __restrict__ k_cache,
            const void* __restrict__ v_cache, const uint16_t* __restrict__ k_scales,
            const uint16_t* __restrict__ v_scales, uint16_t* __restrict__ k, uint16_t* __restrict__ v,
            int32_t* dev_status) {
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * blockDim.y * kTokens + threadIdx.y;
  int64_t row0[kTokens];
#pragma unroll
  for (int i = 0; i < kTokens; ++i) {
    const int64_t t = t0 + i * static_cast<int>(blockDim.y);
    row0[i] = t < s.T ? slot_row(__ldg(slots + t), s, dev_status) : -1;
  }
  const int per_head = s.dim >> 3;
  for (int c = threadIdx.x; c < s.chunks; c += blockDim.x) {
    const int head = c / per_head, d8 = c - head * per_head;
    Raw<KIND> kx[kTokens], vx[kTokens];
#pragma unroll
    for (int i = 0; i < kTokens; ++i) {
      if (row0[i] < 0) continue;
      const int64_t row = row0[i] + static_cast<int64_t>(head) * s.page_size;
      kx[i] = load_row8<KIND>(row, s.dim, d8, k_cache, k_scales);
      vx[i] = load_row8<KIND>(row, s.dim, d8, v_cache, v_scales);
    }
#pragma unroll
    for (int i = 0; i < kTokens; ++i) {
      const int64_t t = t0 + i * static_cast<int>(blockDim.y);
      if (t >= s.T) continue;
      const uint4 none = make_uint4(0, 0, 0, 0);
      reinterpret_cast<uint4*>(k)[t * s.chunks + c] = row0[i] < 0 ? none : values8<KIND>(kx[i]);
      reinterpret_cast<uint4*>(v)[t * s.chunks + c] = row0[i] < 0 ? none : values8<KIND>(vx[i]);
    }
  }
}

// Shared argument checks; fills the shape and the launch geometry.
w4_status check(int64_t T, int32_t kind, int32_t heads, int32_t dim, int64_t pages, int32_t page_size,
                const void* k_cache, const void* v_cache, const uint16_t* k_scales, const uint16_t* v_scales,
                Shape& s, dim3& block, unsigned& grid) {
  if (kind != W4_KV_BF16 && kind != W4_KV_INT8 && kind != W4_KV_INT4) return W4_ERR_INVALID_ARG;
  if (T < 0 || heads < 1 || dim < 32 || dim % 32 || pages < 1 || page_size < 1) return W4_ERR_INVALID_ARG;
  if (dim > 1024 || heads > 65536 || T > 0x7FFFFFFFLL || pages > 0x7FFFFFFFLL) return W4_ERR_UNSUPPORTED;
  if (!k_cache || !v_cache || !aligned_to(k_cache, 16) || !aligned_to(v_cache, 16)) return W4_ERR_INVALID_ARG;
  if (kind != W4_KV_BF16 && (!k_scales || !v_scales || !aligned_to(k_scales, 2) || !aligned_to(v_scales, 2)))
    return W4_ERR_INVALID_ARG;
  s = Shape{T, pages, heads, dim, page_size, heads * (dim / 8)};
  const int bx = s.chunks < 256 ? s.chunks : 256;          // a multiple of 4 either way
  const int by = 256 / bx;
  block = dim3(bx, by);
  grid = static_cast<unsigned>((T + by * kTokens - 1) / (by * kTokens));
  return W4_OK;
}

}  // namespace kv
}  // namespace w4

extern "C" {

w4_status kv_cache_write(const uint16_t* k, const uint16_t* v, int64_t k_stride, int64_t v_stride,
                         const int64_t* slots, int64_t T, int32_t kind, int32_t kv_heads, int32_t head_dim,
                         int64_t pages, int32_t page_size, void* k_cache, void* v_cache, uint16_t* k_scales,
                         uint16_t* v_scales, int32_t* dev_status, void* stream) {
  using namespace w4;
  const EntryRange range("kv_cache_write");
  kv::Shape s;
  dim3 block;
  unsigned grid;
  const w4_status st = kv::check(T, kind, kv_heads, head_dim, pages, page_size, k_cache, v_cache, k_scales, v_scales,
                                 s, block, grid);
  if (st != W4_OK) return st;
  const int64_t wide = static_cast<int64_t>(kv_heads) * head_dim;
  if (k_stride < wide || v_stride < wide || k_stride % 8 || v_stride % 8) return W4_ERR_INVALID_ARG;
  if (T == 0) return W4_OK;
  if (!k || !v || !slots || !aligned_to(k, 16) || !aligned_to(v, 16) || !aligned_to(slots, 8)) return W4_ERR_INVALID_ARG;
  auto str = static_cast<cudaStream_t>(stream);
  auto fn = kind == W4_KV_BF16 ? kv::write_kernel<W4_KV_BF16>
            : kind == W4_KV_INT8 ? kv::write_kernel<W4_KV_INT8> : kv::write_kernel<W4_KV_INT4>;
  fn<<<grid, block, 0, str>>>(k, v, k_stride, v_stride, slots, s, k_cache, v_cache, k_scales, v_scales, dev_status);
  return launched();
}

w4_status kv_cache_read(const int64_t* slots, int64_t T, int32_t kind, int32_t kv_heads, int32_t head_dim,
                        int64_t pages, int32_t page_size, const void* k_cache, const void* v_cache,
                        const uint16_t* k_scales, const uint16_t* v_scales, uint16_t* k, uint16_t* v,
                        int32_t* dev_status, void* stream) {
  using namespace w4;
  const EntryRange range("kv_cache_read");
  kv::Shape s;
  dim3 block;
  unsigned grid;
  const w4_status st = kv::check(T, kind, kv_heads, head_dim, pages, page_size, k_cache, v_cache, k_scales, v_scales,
                                 s, block, grid);
  if (st != W4_OK) return st;
  if (T == 0) return W4_OK;
  if (!k || !v || !slots || !aligned_to(k, 16) || !aligned_to(v, 16) || !aligned_to(slots, 8)) return W4_ERR_INVALID_ARG;
  auto str = static_cast<cudaStream_t>(stream);
  auto fn = kind == W4_KV_BF16 ? kv::read_kernel<W4_KV_BF16>
            : kind == W4_KV_INT8 ? kv::read_kernel<W4_KV_INT8> : kv::read_kernel<W4_KV_INT4>;
  fn<<<grid, block, 0, str>>>(slots, s, k_cache, v_cache, k_scales, v_scales, k, v, dev_status);
  return launched();
}

}  // extern "C"
