// kv_cache_write, kv_cache_read: rows of a paged key/value cache, quantised as they are written and
// turned back into bf16 as they are read.
//
// A cache row is one token's head_dim values of one head.  Groups of 32 along head_dim share one bf16
// scale, as everywhere in this library:
//   int8: s = bf16(max|x| / 127), q = rint(x / s) in -127..127;   int4: s = bf16(max|x| / 7), q in -7..7.
// The quotient is a correctly rounded float32 division.  Both operands have 8-bit significands, so
// x / s lies at least 2^-11 (values of 64 and more) or 2^-18 (below) away from any half-integer it
// does not equal; float32 resolves that, hence the codes are those of exact arithmetic.
//
// Bound by memory.  A thread moves 8 elements of the key row and the 8 beside them of the value row
// (two independent 16-byte loads or stores); four neighbouring threads share a group, so its
// maximum takes two shuffles.
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

// 8 bf16 of a group quartet -> codes (2 words int8, 1 word int4) and, in lane 0 of the four, the scale.
template <int KIND>
__device__ __forceinline__ uint32_t quantise8(const uint4& x, uint32_t (&o)[2]) {
  constexpr float kTop = KIND == W4_KV_INT8 ? 127.f : 7.f;
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
  const uint32_t sb = f32_to_bf16_bits(__fdiv_rn(bf16_lo_to_f32(m), kTop));
  const float s = bf16_lo_to_f32(sb);
  if (s == 0.f) return 0u;
  int c[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    c[2 * j] = __float2int_rn(fminf(fmaxf(__fdiv_rn(bf16_lo_to_f32(w[j]), s), -kTop), kTop));
    c[2 * j + 1] = __float2int_rn(fminf(fmaxf(__fdiv_rn(bf16_hi_to_f32(w[j]), s), -kTop), kTop));
  }
  o[0] = 0u;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (KIND == W4_KV_INT8) o[j >> 2] |= static_cast<uint32_t>(c[j] & 0xFF) << (8 * (j & 3));
    else o[0] |= static_cast<uint32_t>(c[j] + 8) << (4 * j);
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
  if (row < 0) return;
  if (KIND == W4_KV_INT8) reinterpret_cast<uint2*>(cache)[row * (dim >> 3) + d8] = make_uint2(o[0], o[1]);
  else reinterpret_cast<uint32_t*>(cache)[row * (dim >> 3) + d8] = o[0];
  if ((d8 & 3) == 0) scales[row * (dim >> 5) + (d8 >> 2)] = static_cast<uint16_t>(sb);
}

// blockDim = (chunks of a token handled at once, a multiple of 4; tokens), so a group's four
// threads are neighbours in one warp.
template <int KIND>
__global__ void __launch_bounds__(256)
write_kernel(const uint16_t* __restrict__ k, const uint16_t* __restrict__ v, int64_t k_stride, int64_t v_stride,
             const int64_t* __restrict__ slots, Shape s, void* k_cache, void* v_cache, uint16_t* k_scales,
             uint16_t* v_scales, int32_t* dev_status) {
  const int64_t t = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
  if (t >= s.T) return;                                   // uniform over a group's four threads
  const int64_t row0 = slot_row(__ldg(slots + t), s, dev_status);
  if (row0 < 0) return;
  const int per_head = s.dim >> 3;
  for (int c = threadIdx.x; c < s.chunks; c += blockDim.x) {
    const int head = c / per_head, d8 = c - head * per_head;
    const uint4 kx = __ldg(reinterpret_cast<const uint4*>(k + t * k_stride) + c);
    const uint4 vx = __ldg(reinterpret_cast<const uint4*>(v + t * v_stride) + c);
    const int64_t row = row0 + static_cast<int64_t>(head) * s.page_size;
    store_row8<KIND>(kx, row, s.dim, d8, k_cache, k_scales);
    store_row8<KIND>(vx, row, s.dim, d8, v_cache, v_scales);
  }
}

template <int KIND>
__device__ __forceinline__ uint4 load_row8(int64_t row, int dim, int d8, const void* cache, const uint16_t* scales) {
  const int64_t at = row * (dim >> 3) + d8;
  if (KIND == W4_KV_BF16) return __ldg(reinterpret_cast<const uint4*>(cache) + at);
  const float s = bf16_lo_to_f32(__ldg(scales + row * (dim >> 5) + (d8 >> 2)));
  float f[8];
  if (KIND == W4_KV_INT8) {
    const uint2 w = __ldg(reinterpret_cast<const uint2*>(cache) + at);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      f[j] = static_cast<float>(static_cast<int32_t>((j < 4 ? w.x : w.y) << (24 - 8 * (j & 3))) >> 24) * s;
  } else {
    const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(cache) + at);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = static_cast<float>(static_cast<int32_t>((w >> (4 * j)) & 15u) - 8) * s;
  }
  // code * scale is exact in float32 (at most 7 + 8 bits), then rounded once
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}

template <int KIND>
__global__ void __launch_bounds__(256)
read_kernel(const int64_t* __restrict__ slots, Shape s, const void* __restrict__ k_cache,
            const void* __restrict__ v_cache, const uint16_t* __restrict__ k_scales,
            const uint16_t* __restrict__ v_scales, uint16_t* __restrict__ k, uint16_t* __restrict__ v,
            int32_t* dev_status) {
  const int64_t t = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
  if (t >= s.T) return;
  const int64_t row0 = slot_row(__ldg(slots + t), s, dev_status);
  const int per_head = s.dim >> 3;
  for (int c = threadIdx.x; c < s.chunks; c += blockDim.x) {
    const int head = c / per_head, d8 = c - head * per_head;
    uint4 kx = make_uint4(0, 0, 0, 0), vx = kx;
    if (row0 >= 0) {
      const int64_t row = row0 + static_cast<int64_t>(head) * s.page_size;
      kx = load_row8<KIND>(row, s.dim, d8, k_cache, k_scales);
      vx = load_row8<KIND>(row, s.dim, d8, v_cache, v_scales);
    }
    reinterpret_cast<uint4*>(k)[t * s.chunks + c] = kx;
    reinterpret_cast<uint4*>(v)[t * s.chunks + c] = vx;
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
  grid = static_cast<unsigned>((T + by - 1) / by);
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
