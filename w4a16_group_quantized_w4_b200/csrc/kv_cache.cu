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
// Bound by memory, if the instructions are few.  A writing thread takes 16 elements of the key row and the 16
// beside them of the value row; two neighbouring lanes share a group, so its maximum takes one shuffle.
// Measured for 8192 tokens of 8 heads of 128 to int8: 23.4 us with a division per element, 19.2 us with a
// reciprocal and a Newton step, 15.1 us with packed maxima, whole-warp shuffles and divisions of indexes by
// multiplication, 12.4 us with 16 elements a thread instead of 8, 12.1 us (4.3 TB/s; 5.2 for 32768 tokens) with
// quotients in pairs.  A reading
// thread takes 8 of each, twice, so that a warp's stores fill whole lines: 32768 int8 tokens take 36 us (5.6
// TB/s), 45 us with 16 elements a thread.
#include "common.cuh"
#include "entry.cuh"

namespace w4 {
namespace kv {

// n / d for n < 2^31: (umulhi(n, mul) + n) >> shift
struct Divider {
  uint32_t d, mul;
  int shift;
};
inline Divider divider(uint32_t d) {
  Divider v{d, 0, 0};
  while ((1ull << v.shift) < d) ++v.shift;
  v.mul = static_cast<uint32_t>((((1ull << v.shift) - d) << 32) / d + 1);
  return v;
}
__device__ __forceinline__ uint32_t divide(uint32_t n, const Divider& v) { return (__umulhi(n, v.mul) + n) >> v.shift; }

struct Shape {
  int64_t slots;                       // pages * page_size
  uint32_t total;                      // chunks of 16 (writing) or 8 elements in this launch, below 2^31
  int heads, dim;
  Divider chunks, per_head, page_size; // chunks a token, chunks a head, tokens a page
};

// One thread's chunk: its token, and its place in the cache.
struct Chunk {
  uint32_t t, c;                       // token, chunk within it
  int64_t row;                         // cache row (all heads of all pages counted); -1 for none
  int part;                            // chunk within the row
};
__device__ __forceinline__ Chunk chunk_of(uint32_t i, const Shape& s, const int64_t* slots, int32_t* dev_status) {
  Chunk k;
  k.t = divide(i, s.chunks);
  k.c = i - k.t * s.chunks.d;
  const uint32_t head = divide(k.c, s.per_head);
  k.part = static_cast<int>(k.c - head * s.per_head.d);
  const int64_t slot = __ldg(slots + k.t);
  k.row = -1;
  if (slot < 0) return k;
  if (slot >= s.slots) {
    set_status(dev_status, W4_ERR_INVALID_ARG);
    return k;
  }
  int64_t page;
  uint32_t off;
  if (slot <= 0x7FFFFFFF) {
    const uint32_t p = divide(static_cast<uint32_t>(slot), s.page_size);
    off = static_cast<uint32_t>(slot) - p * s.page_size.d;
    page = p;
  } else {
    page = slot / s.page_size.d;
    off = static_cast<uint32_t>(slot - page * s.page_size.d);
  }
  k.row = (page * s.heads + head) * s.page_size.d + off;
  return k;
}

constexpr int kThreads = 256;

// rint(x / s) + bias of two elements in the low bits of floats of 1.5 * 2^23 and more; s positive and normal, inv
// near 1 / s.  As packed float32 pairs: the negative of s and the bias come as pairs too.
__device__ __forceinline__ uint64_t twice(float v) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %1};" : "=l"(d) : "f"(v));
  return d;
}
__device__ __forceinline__ void quotients(uint32_t x2, uint64_t minus_s, uint64_t inv, uint64_t bias, uint32_t& lo, uint32_t& hi) {
  uint64_t x, q, e;
  asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(bf16_lo_to_f32(x2)), "f"(bf16_hi_to_f32(x2)));
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(q) : "l"(x), "l"(inv));
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(e) : "l"(q), "l"(minus_s), "l"(x));
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(q) : "l"(e), "l"(inv));
  asm("add.rn.f32x2 %0, %0, %1;" : "+l"(q) : "l"(bias));
  asm("mov.b64 {%0, %1}, %2;" : "=r"(lo), "=r"(hi) : "l"(q));
}
// the low bytes of four words
__device__ __forceinline__ uint32_t low_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// 16 bf16 of half a group -> codes (4 words int8, 2 words int4); returns the scale's bits.  Whole warps only.
template <int KIND>
__device__ __forceinline__ uint32_t quantise16(const uint32_t (&w)[8], uint32_t (&o)[4]) {
  constexpr int kTop = KIND == W4_KV_INT8 ? 127 : 7;
  uint32_t pair = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) pair = __vmaxu2(pair, w[j] & 0x7FFF7FFFu);
  pair = __vmaxu2(pair, __shfl_xor_sync(0xffffffffu, pair, 1));
  const uint32_t m = max(pair & 0xFFFFu, pair >> 16);
#pragma unroll
  for (int j = 0; j < 4; ++j) o[j] = KIND == W4_KV_INT4 ? 0x88888888u : 0u;
  if (m >= 0x7F80u) return 0x7FC0u;                       // NaN or infinity: codes 0, scale NaN
  // max / top keeps at least 2^-16 of itself from a bf16 midpoint, so a product rounds as the quotient does
  const uint32_t sb = f32_to_bf16_bits(bf16_lo_to_f32(m) * (1.f / kTop));
  const float s = bf16_lo_to_f32(sb);
  if (s == 0.f) return 0u;
  uint32_t c[16];                                         // codes (int4: plus 8) in the low bits
  constexpr float kBias = KIND == W4_KV_INT4 ? 8.f : 0.f;
  if (s >= 0x1p-100f && s <= 0x1p100f) {
    // Rounding max / top to bf16 takes off at most 2^-8 of a scale of 1: |x / s| <= top (1 + 2^-8) < top + 1/2,
    // so nothing has to be clamped.
    float inv;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
    const uint64_t minus_s2 = twice(-s), inv2 = twice(inv), bias2 = twice(12582912.f + kBias);
#pragma unroll
    for (int j = 0; j < 8; ++j) quotients(w[j], minus_s2, inv2, bias2, c[2 * j], c[2 * j + 1]);
  } else {                                                // (a subnormal step can be far below max / top)
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const float v = j & 1 ? bf16_hi_to_f32(w[j >> 1]) : bf16_lo_to_f32(w[j >> 1]);
      c[j] = static_cast<uint32_t>(max(-kTop, min(kTop, __float2int_rn(__fdiv_rn(v, s)))) + static_cast<int>(kBias));
    }
  }
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    if (KIND == W4_KV_INT8) {
      o[h] = low_bytes(c[4 * h], c[4 * h + 1], c[4 * h + 2], c[4 * h + 3]);
    } else if (h < 2) {
      const uint32_t* q = c + 8 * h;
      o[h] = (low_bytes(q[0], q[2], q[4], q[6]) & 0x0F0F0F0Fu) | ((low_bytes(q[1], q[3], q[5], q[7]) & 0x0F0F0F0Fu) << 4);
    }
  }
  return sb;
}

// all lanes of the warp take part; those without a row store nothing
template <int KIND>
__device__ __forceinline__ void store_row16(const uint32_t (&w)[8], const Chunk& k, int dim, void* cache, uint16_t* scales) {
  const int64_t at = k.row * (dim >> 4) + k.part;
  if constexpr (KIND == W4_KV_BF16) {
    if (k.row < 0) return;
    uint4* dst = reinterpret_cast<uint4*>(cache) + 2 * at;
    dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
    dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
  } else {
    uint32_t o[4];
    const uint32_t sb = quantise16<KIND>(w, o);
    if (k.row < 0) return;
    if (KIND == W4_KV_INT8) reinterpret_cast<uint4*>(cache)[at] = make_uint4(o[0], o[1], o[2], o[3]);
    else reinterpret_cast<uint2*>(cache)[at] = make_uint2(o[0], o[1]);
    if ((k.part & 1) == 0) scales[at >> 1] = static_cast<uint16_t>(sb);
  }
}

__device__ __forceinline__ void load16(uint32_t (&w)[8], const uint4* p) {
  const uint4 a = __ldg(p), b = __ldg(p + 1);
  w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
  w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
}

template <int KIND>
__global__ void __launch_bounds__(kThreads)
write_kernel(const uint16_t* __restrict__ k, const uint16_t* __restrict__ v, int64_t k_stride, int64_t v_stride,
             const int64_t* __restrict__ slots, Shape s, void* k_cache, void* v_cache, uint16_t* k_scales,
             uint16_t* v_scales, int32_t* dev_status) {
  const uint32_t i = blockIdx.x * kThreads + threadIdx.x;
  Chunk at = chunk_of(min(i, s.total - 1), s, slots, dev_status);   // (total is even: a group stays whole)
  if (i >= s.total) at.row = -1;
  uint32_t kx[8], vx[8];
  load16(kx, reinterpret_cast<const uint4*>(k + at.t * k_stride) + 2 * at.c);
  load16(vx, reinterpret_cast<const uint4*>(v + at.t * v_stride) + 2 * at.c);
  store_row16<KIND>(kx, at, s.dim, k_cache, k_scales);
  store_row16<KIND>(vx, at, s.dim, v_cache, v_scales);
}

constexpr int kTokens = 2;             // chunks of 8 elements a reading thread works on at once

// 8 elements of a cache row as they are held
template <int KIND>
struct Raw {
  uint32_t w[KIND == W4_KV_BF16 ? 4 : KIND == W4_KV_INT8 ? 2 : 1];
  uint16_t scale;
};
template <int KIND>
__device__ __forceinline__ Raw<KIND> load_row8(const Chunk& k, int dim, const void* cache, const uint16_t* scales) {
  Raw<KIND> r;
  const int64_t at = max(k.row, static_cast<int64_t>(0)) * (dim >> 3) + k.part;   // (row 0 for none: not used)
  if constexpr (KIND == W4_KV_BF16) {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(cache) + at);
    r.w[0] = v.x; r.w[1] = v.y; r.w[2] = v.z; r.w[3] = v.w;
  } else if constexpr (KIND == W4_KV_INT8) {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(cache) + at);
    r.w[0] = v.x; r.w[1] = v.y;
  } else {
    r.w[0] = __ldg(reinterpret_cast<const uint32_t*>(cache) + at);
  }
  if constexpr (KIND != W4_KV_BF16) r.scale = __ldg(scales + (at >> 2));
  return r;
}

// A code's bits u = q + bias in the second byte of 2^15 (0x4700uu00) are the float 2^15 + u.  Less 2^15 + bias it is
// q, and q * scale has 16 significant bits at most: both steps are exact whatever the scale (one fused step with
// (2^15 + bias) * scale as addend would overflow from scales of 2^113 on), and bf16 rounds once.
template <int KIND>
__device__ __forceinline__ uint4 values8(const Raw<KIND>& r) {
  if constexpr (KIND == W4_KV_BF16) {
    return make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
  } else {
    const uint64_t s2 = twice(bf16_lo_to_f32(r.scale)), off2 = twice(-(32768.f + (KIND == W4_KV_INT8 ? 128.f : 8.f)));
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
    for (int j = 0; j < 8; j += 2) {
      uint32_t b[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t word = KIND == W4_KV_INT8 ? u[j >> 2] : u[i];
        const int byte = KIND == W4_KV_INT8 ? (j + i) & 3 : j >> 1;
        b[i] = __byte_perm(word, 0x47000000u, 0x7404 | byte << 4);
      }
      uint64_t x;
      asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "r"(b[0]), "r"(b[1]));
      asm("add.rn.f32x2 %0, %0, %1;" : "+l"(x) : "l"(off2));
      asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(x) : "l"(s2));
      asm("mov.b64 {%0, %1}, %2;" : "=f"(f[j]), "=f"(f[j + 1]) : "l"(x));
    }
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
  }
}

template <int KIND>
__global__ void __launch_bounds__(kThreads)
read_kernel(const int64_t* __restrict__ slots, Shape s, const void* __restrict__ k_cache,
            const void* __restrict__ v_cache, const uint16_t* __restrict__ k_scales,
            const uint16_t* __restrict__ v_scales, uint16_t* __restrict__ k, uint16_t* __restrict__ v,
            int32_t* dev_status) {
  const uint32_t i0 = blockIdx.x * (kThreads * kTokens) + threadIdx.x;
  Chunk at[kTokens];
  Raw<KIND> kx[kTokens], vx[kTokens];
#pragma unroll
  for (int i = 0; i < kTokens; ++i) {
    at[i] = chunk_of(min(i0 + i * kThreads, s.total - 1), s, slots, dev_status);
    kx[i] = load_row8<KIND>(at[i], s.dim, k_cache, k_scales);
    vx[i] = load_row8<KIND>(at[i], s.dim, v_cache, v_scales);
  }
#pragma unroll
  for (int i = 0; i < kTokens; ++i) {
    const uint32_t n = i0 + i * kThreads;
    if (n >= s.total) return;
    const uint4 none = make_uint4(0, 0, 0, 0);
    reinterpret_cast<uint4*>(k)[n] = at[i].row < 0 ? none : values8<KIND>(kx[i]);
    reinterpret_cast<uint4*>(v)[n] = at[i].row < 0 ? none : values8<KIND>(vx[i]);
  }
}

// Shared argument checks; fills the shape (but its total) for chunks of `wide` elements.
w4_status check(int64_t T, int32_t kind, int32_t heads, int32_t dim, int64_t pages, int32_t page_size,
                const void* k_cache, const void* v_cache, const uint16_t* k_scales, const uint16_t* v_scales,
                int wide, Shape& s) {
  if (kind != W4_KV_BF16 && kind != W4_KV_INT8 && kind != W4_KV_INT4) return W4_ERR_INVALID_ARG;
  if (T < 0 || heads < 1 || dim < 32 || dim % 32 || pages < 1 || page_size < 1) return W4_ERR_INVALID_ARG;
  if (dim > 1024 || heads > 65536 || T > 0x7FFFFFFFLL || pages > 0x7FFFFFFFLL) return W4_ERR_UNSUPPORTED;
  if (!k_cache || !v_cache || !aligned_to(k_cache, 16) || !aligned_to(v_cache, 16)) return W4_ERR_INVALID_ARG;
  if (kind != W4_KV_BF16 && (!k_scales || !v_scales || !aligned_to(k_scales, 2) || !aligned_to(v_scales, 2)))
    return W4_ERR_INVALID_ARG;
  s.slots = pages * page_size;
  s.heads = heads;
  s.dim = dim;
  s.chunks = divider(heads * (dim / wide));
  s.per_head = divider(dim / wide);
  s.page_size = divider(page_size);
  return W4_OK;
}

// Tokens a launch takes: their chunks are counted in 31 bits, less the last block's overhang.
inline int64_t tokens_at_once(const Shape& s) { return 0x7FFFF000LL / s.chunks.d; }
inline unsigned blocks_for(uint32_t total, int per_thread) {
  return (total + kThreads * per_thread - 1) / (kThreads * per_thread);
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
  const w4_status st = kv::check(T, kind, kv_heads, head_dim, pages, page_size, k_cache, v_cache, k_scales, v_scales, 16, s);
  if (st != W4_OK) return st;
  const int64_t wide = static_cast<int64_t>(kv_heads) * head_dim;
  if (k_stride < wide || v_stride < wide || k_stride % 8 || v_stride % 8) return W4_ERR_INVALID_ARG;
  if (T == 0) return W4_OK;
  if (!k || !v || !slots || !aligned_to(k, 16) || !aligned_to(v, 16) || !aligned_to(slots, 8)) return W4_ERR_INVALID_ARG;
  auto fn = kind == W4_KV_BF16 ? kv::write_kernel<W4_KV_BF16>
            : kind == W4_KV_INT8 ? kv::write_kernel<W4_KV_INT8> : kv::write_kernel<W4_KV_INT4>;
  const int64_t most = kv::tokens_at_once(s);
  for (int64_t t = 0; t < T; t += most) {
    s.total = static_cast<uint32_t>((T - t < most ? T - t : most) * s.chunks.d);
    fn<<<kv::blocks_for(s.total, 1), kv::kThreads, 0, static_cast<cudaStream_t>(stream)>>>(
        k + t * k_stride, v + t * v_stride, k_stride, v_stride, slots + t, s, k_cache, v_cache, k_scales, v_scales,
        dev_status);
  }
  return launched();
}

w4_status kv_cache_read(const int64_t* slots, int64_t T, int32_t kind, int32_t kv_heads, int32_t head_dim,
                        int64_t pages, int32_t page_size, const void* k_cache, const void* v_cache,
                        const uint16_t* k_scales, const uint16_t* v_scales, uint16_t* k, uint16_t* v,
                        int32_t* dev_status, void* stream) {
  using namespace w4;
  const EntryRange range("kv_cache_read");
  kv::Shape s;
  const w4_status st = kv::check(T, kind, kv_heads, head_dim, pages, page_size, k_cache, v_cache, k_scales, v_scales, 8, s);
  if (st != W4_OK) return st;
  if (T == 0) return W4_OK;
  if (!k || !v || !slots || !aligned_to(k, 16) || !aligned_to(v, 16) || !aligned_to(slots, 8)) return W4_ERR_INVALID_ARG;
  auto fn = kind == W4_KV_BF16 ? kv::read_kernel<W4_KV_BF16>
            : kind == W4_KV_INT8 ? kv::read_kernel<W4_KV_INT8> : kv::read_kernel<W4_KV_INT4>;
  const int64_t most = kv::tokens_at_once(s), wide = static_cast<int64_t>(kv_heads) * head_dim;
  for (int64_t t = 0; t < T; t += most) {
    s.total = static_cast<uint32_t>((T - t < most ? T - t : most) * s.chunks.d);
    fn<<<kv::blocks_for(s.total, kv::kTokens), kv::kThreads, 0, static_cast<cudaStream_t>(stream)>>>(
        slots + t, s, k_cache, v_cache, k_scales, v_scales, k + t * wide, v + t * wide, dev_status);
  }
  return launched();
}

}  // extern "C"
