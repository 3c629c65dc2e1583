// w4_rms_add, w4_rms_add_q8: residual addition and root-mean-square norm of token rows, in bf16 or
// as 8-bit codes with one float32 scale per row.
//
// Per row, h = bf16(x + residual) is stored and normalised:
//   y_i = (h_i * w_i) * (1 / sqrt(mean(h^2) + eps)).
// h_i * w_i is exact in float32 (two 8-bit significands), and multiplication by one positive
// number keeps the order, so max|y| = max|h w| * (1 / rms): both row statistics come out of one
// pass over registers and one reduction, and every input byte is read once.  The 8-bit form takes
// s = max|y| / 127 and q_i = rint(y_i / s) = rint(h_i w_i * (127 / max|h w|)): one fused multiply and add
// of 1.5 * 2^23, which leaves the rounded integer in the low bits.
//
// Bound by memory: x, residual and h at 2 bytes an element, y at 2 or 1.  A row is held in the
// registers of 1 to 32 warps, CPT 16-byte chunks a thread; short rows share a block, so that a
// block has at least 3 warps.  Instructions come next, so elements go through in pairs.  8192 rows of 2816 with
// residual and weight: bf16 31.1 us (5.9 TB/s, 0.91 of a copy's rate), 8-bit 31.5 us (35 with a division an element,
// 36.5 with single elements and the weights read twice); 64 rows 2.8 us, latency.
#include "common.cuh"
#include "entry.cuh"

namespace w4 {
namespace ra {

// Packed forms, two elements an instruction: bf16(x + residual) rounded once, float32 pairs.
__device__ __forceinline__ uint32_t add_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint64_t pair_of(uint32_t bf16x2) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(bf16_lo_to_f32(bf16x2)), "f"(bf16_hi_to_f32(bf16x2)));
  return v;
}
__device__ __forceinline__ void halves(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t twice(float v) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %1};" : "=l"(d) : "f"(v));
  return d;
}
// the larger magnitude; NaN if either is
__device__ __forceinline__ float max_abs(float m, float v) {
  asm("max.NaN.f32 %0, %0, %1;" : "+f"(m) : "f"(fabsf(v)));
  return m;
}

// A row whose mean square and eps are too small for float32 (only with an eps that small), from its stored h on: by a
// power of two that brings its largest element, or the root of eps where that is larger, to about 1.  Every warp of
// the row goes over the whole of it and writes its threads' part.  Not inlined: it is hardly ever taken, and with
// rescaled registers in the kernel itself 8192 rows of 512 took 6.2 us, not 5.6.
template <bool Q8>
__device__ __noinline__ void tiny_row(const uint4* h, const uint4* weight, int nv, int H, float eps, int tid, int tpr,
                                      uint4* y, uint2* q, float* q_scale) {
  const int lane = tid & 31;
  const uint4 ones = make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);
  uint32_t most = 0;
  for (int i = lane; i < nv; i += 32) {
    const uint4 v = h[i];
    most = __vmaxu2(__vmaxu2(most, v.x & 0x7FFF7FFFu), __vmaxu2(v.y & 0x7FFF7FFFu, __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu)));
  }
  most = __reduce_max_sync(0xffffffffu, max(most & 0xFFFFu, most >> 16));
  const uint32_t root = __float_as_uint(sqrtf(eps)) >> 23;                // exponents, plus 127
  const float up = __uint_as_float((254u - max(max(most >> 7, 1u), root)) << 23);
  float sum = 0.f, largest = 0.f;                                          // of |h w|, scaled
  for (int i = lane; i < nv; i += 32) {
    const uint4 v = h[i], wv = weight ? __ldg(weight + i) : ones;
    const uint32_t x[4] = {v.x, v.y, v.z, v.w}, w[4] = {wv.x, wv.y, wv.z, wv.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float lo = bf16_lo_to_f32(x[j]) * up, hi = bf16_hi_to_f32(x[j]) * up;
      sum = fmaf(hi, hi, fmaf(lo, lo, sum));
      largest = max_abs(max_abs(largest, lo * bf16_lo_to_f32(w[j])), hi * bf16_hi_to_f32(w[j]));
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  const float amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(largest)));
  // (a row of zeros gives zeros, with eps = 0 too)
  const float inv = most ? 1.f / sqrtf(sum / static_cast<float>(H) + eps * up * up) : 0.f;
  const bool finite = amax < __int_as_float(0x7F800000);
  const float s = finite ? amax * inv / 127.f : __int_as_float(0x7FC00000);
  if (Q8 && tid == 0) *q_scale = s;
  for (int i = tid; i < nv; i += tpr) {
    const uint4 v = h[i], wv = weight ? __ldg(weight + i) : ones;
    const uint32_t x[4] = {v.x, v.y, v.z, v.w}, w[4] = {wv.x, wv.y, wv.z, wv.w};
    uint32_t o[4] = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float lo = bf16_lo_to_f32(x[j]) * up * bf16_lo_to_f32(w[j]) * inv, hi = bf16_hi_to_f32(x[j]) * up * bf16_hi_to_f32(w[j]) * inv;
      if constexpr (!Q8) o[j] = pack_bf16x2(lo, hi);
      else if (finite && s > 0.f)
        o[j >> 1] |= (static_cast<uint32_t>(max(-127, min(127, __float2int_rn(__fdiv_rn(lo, s))))) & 0xFF |
                      (static_cast<uint32_t>(max(-127, min(127, __float2int_rn(__fdiv_rn(hi, s))))) & 0xFF) << 8) << (16 * (j & 1));
    }
    if constexpr (Q8) q[i] = make_uint2(o[0], o[1]);
    else y[i] = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

// wpr warps per row, blockDim.x / (32 wpr) rows per block.
template <int CPT, bool Q8>
__global__ void __launch_bounds__(1024)
rms_add_kernel(const uint16_t* __restrict__ x, const uint16_t* residual, const uint16_t* __restrict__ weight,
               int64_t T, int H, float eps, int wpr, uint16_t* h_out, uint16_t* __restrict__ y,
               int8_t* __restrict__ q, float* __restrict__ q_scale) {
  __shared__ float s_sum[32];
  __shared__ uint32_t s_max[32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row_in_block = warp / wpr;
  const int rpb = (blockDim.x >> 5) / wpr;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * rpb + row_in_block;
  const int tid = threadIdx.x - row_in_block * wpr * 32;   // thread within the row
  const int tpr = wpr * 32;
  const int nv = H >> 3;                                   // 16-byte chunks
  const bool live = row < T;
  const uint4* xr = reinterpret_cast<const uint4*>(x + row * H);
  const uint4* rr = residual ? reinterpret_cast<const uint4*>(residual + row * H) : nullptr;

  uint4 hv[CPT], rv[CPT];
#pragma unroll
  for (int c = 0; c < CPT; ++c) {
    const int i = c * tpr + tid;
    const bool ok = live && i < nv;
    hv[c] = ok ? __ldg(xr + i) : make_uint4(0, 0, 0, 0);
    // plain load: h_out may be residual itself
    if (residual) rv[c] = ok ? rr[i] : make_uint4(0, 0, 0, 0);
  }
  uint64_t sum2 = 0;                                       // (0.f, 0.f)
  float largest = 0.f;                                     // of |h w|
  uint64_t hw2[Q8 ? CPT : 1][4];                           // h w
#pragma unroll
  for (int c = 0; c < CPT; ++c) {
    const int i = c * tpr + tid;
    if (!(live && i < nv)) continue;
    uint32_t* hw = reinterpret_cast<uint32_t*>(&hv[c]);
    if (residual) {
      const uint32_t* rw = reinterpret_cast<const uint32_t*>(&rv[c]);
#pragma unroll
      for (int j = 0; j < 4; ++j) hw[j] = add_bf16x2(hw[j], rw[j]);
      reinterpret_cast<uint4*>(h_out + row * H)[i] = hv[c];
    }
    uint4 wv = make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);
    if (Q8 && weight) wv = __ldg(reinterpret_cast<const uint4*>(weight) + i);
    const uint32_t* ww = reinterpret_cast<const uint32_t*>(&wv);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint64_t h2 = pair_of(hw[j]);
      sum2 = fma2(h2, h2, sum2);
      if constexpr (Q8) {
        hw2[c][j] = mul2(h2, pair_of(ww[j]));
        float lo, hi;
        halves(hw2[c][j], lo, hi);
        largest = max_abs(max_abs(largest, lo), hi);
      }
    }
  }
  float sum, sum_hi;
  halves(sum2, sum, sum_hi);
  sum += sum_hi;
  uint32_t amax = __float_as_uint(largest);                // as a bit pattern: NaN > inf > finite
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (Q8) amax = __reduce_max_sync(0xffffffffu, amax);
  if (wpr > 1) {
    if (lane == 0) { s_sum[warp] = sum; s_max[warp] = amax; }
    __syncthreads();
    sum = 0.f;
    amax = 0;
    for (int w = 0; w < wpr; ++w) {
      sum += s_sum[row_in_block * wpr + w];
      if (Q8) amax = max(amax, s_max[row_in_block * wpr + w]);
    }
  }
  if (!live) return;
  const float mean = sum / static_cast<float>(H) + eps;
  if (mean < 0x1p-90f) {                                   // squares may have fallen below float32's range
    __syncwarp();                                          // (several warps a row: the barrier above)
    tiny_row<Q8>(residual ? reinterpret_cast<const uint4*>(h_out + row * H) : xr, reinterpret_cast<const uint4*>(weight),
                 nv, H, eps, tid, tpr, reinterpret_cast<uint4*>(y + row * H), reinterpret_cast<uint2*>(q + row * H),
                 q_scale + row);
    return;
  }
  const float inv = 1.0f / sqrtf(mean);
  float s = 0.f;
  bool finite = true;
  if (Q8) {
    // a row holding NaN or infinity: scale NaN, codes 0, so that it stands for NaN throughout
    finite = amax < 0x7F800000u && sum < __int_as_float(0x7F800000);
    s = finite ? __uint_as_float(amax) * inv / 127.f : __int_as_float(0x7FC00000);
    if (tid == 0) q_scale[row] = s;
  }
  const float up = Q8 ? 127.f / __uint_as_float(amax) : 0.f;
#pragma unroll
  for (int c = 0; c < CPT; ++c) {
    const int i = c * tpr + tid;
    if (i >= nv) break;
    float v[8];
    if constexpr (Q8) {
      uint32_t code[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float lo, hi;
        halves(fma2(hw2[c][j], twice(up), twice(12582912.f)), lo, hi);
        code[2 * j] = __float_as_uint(lo);
        code[2 * j + 1] = __float_as_uint(hi);
        halves(hw2[c][j], v[2 * j], v[2 * j + 1]);
      }
      uint2 o = make_uint2(__byte_perm(__byte_perm(code[0], code[1], 0x0040), __byte_perm(code[2], code[3], 0x0040), 0x5410),
                           __byte_perm(__byte_perm(code[4], code[5], 0x0040), __byte_perm(code[6], code[7], 0x0040), 0x5410));
      if (!(finite && s >= 0x1p-126f && __uint_as_float(amax) >= 0x1p-120f)) {
        // no scale to speak of; a subnormal one, which need not be close to max / 127; or 127 / max past float32
        o = make_uint2(0, 0);
        if (finite && s > 0.f) {
          uint32_t b[2] = {0, 0};
          for (int j = 0; j < 8; ++j)
            b[j >> 2] |= static_cast<uint32_t>(max(-127, min(127, __float2int_rn(__fdiv_rn(v[j] * inv, s)))) & 0xFF) << (8 * (j & 3));
          o = make_uint2(b[0], b[1]);
        }
      }
      reinterpret_cast<uint2*>(q + row * H)[i] = o;
    } else {
      uint4 wv = make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);
      if (weight) wv = __ldg(reinterpret_cast<const uint4*>(weight) + i);
      const uint32_t* ww = reinterpret_cast<const uint32_t*>(&wv);
      const uint32_t* hw = reinterpret_cast<const uint32_t*>(&hv[c]);
#pragma unroll
      for (int j = 0; j < 4; ++j) halves(mul2(mul2(pair_of(hw[j]), pair_of(ww[j])), twice(inv)), v[2 * j], v[2 * j + 1]);
      reinterpret_cast<uint4*>(y + row * H)[i] = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                            pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
    }
  }
}

template <int CPT, bool Q8>
void launch_cpt(const uint16_t* x, const uint16_t* residual, const uint16_t* weight, int64_t T, int H, float eps,
                uint16_t* h, uint16_t* y, int8_t* q, float* qs, cudaStream_t stream) {
  const int nv = H / 8;
  const int wpr = (nv + 32 * CPT - 1) / (32 * CPT);        // at most 32: the caller picked CPT
  const int rpb = wpr >= 4 ? 1 : 4 / wpr;
  const int64_t grid = (T + rpb - 1) / rpb;
  rms_add_kernel<CPT, Q8><<<static_cast<unsigned>(grid), 32 * wpr * rpb, 0, stream>>>(x, residual, weight, T, H, eps,
                                                                                     wpr, h, y, q, qs);
}

constexpr int kMaxH = 8 * 4 * 1024;                        // CPT 4, 1024 threads

template <bool Q8>
w4_status run(const uint16_t* x, const uint16_t* residual, const uint16_t* weight, int64_t T, int32_t H, float eps,
              uint16_t* h, uint16_t* y, int8_t* q, float* qs, void* stream) {
  if (T < 0 || H < 8 || H % 8 || !(eps >= 0.f) || eps > 1e30f) return W4_ERR_INVALID_ARG;
  if (H > kMaxH || T > 0x7FFFFFFFLL) return W4_ERR_UNSUPPORTED;
  if (T == 0) return W4_OK;
  if (!x || (residual && !h) || (Q8 ? (!q || !qs) : !y)) return W4_ERR_INVALID_ARG;
  if (!aligned_to(x, 16) || !aligned_to(residual, 16) || !aligned_to(weight, 16) || !aligned_to(h, 16) ||
      !aligned_to(y, 16) || !aligned_to(q, 8) || !aligned_to(qs, 4))
    return W4_ERR_INVALID_ARG;
  auto s = static_cast<cudaStream_t>(stream);
  const int nv = H / 8;
  // few rows: one chunk a thread for the shortest chain; many rows: more bytes in flight a thread
  const int64_t few = 2 * device_sm_count();
  if (nv <= 1024 && T <= few) launch_cpt<1, Q8>(x, residual, weight, T, H, eps, h, y, q, qs, s);
  else if (nv <= 2048) launch_cpt<2, Q8>(x, residual, weight, T, H, eps, h, y, q, qs, s);
  else launch_cpt<4, Q8>(x, residual, weight, T, H, eps, h, y, q, qs, s);
  return launched();
}

}  // namespace ra
}  // namespace w4

extern "C" {

w4_status w4_rms_add(const uint16_t* x, const uint16_t* residual, const uint16_t* weight, int64_t T, int32_t H,
                     float eps, uint16_t* h, uint16_t* y, void* stream) {
  const w4::EntryRange range("w4_rms_add");
  return w4::ra::run<false>(x, residual, weight, T, H, eps, h, y, nullptr, nullptr, stream);
}

w4_status w4_rms_add_q8(const uint16_t* x, const uint16_t* residual, const uint16_t* weight, int64_t T, int32_t H,
                        float eps, uint16_t* h, int8_t* q, float* q_scale, void* stream) {
  const w4::EntryRange range("w4_rms_add_q8");
  return w4::ra::run<true>(x, residual, weight, T, H, eps, h, nullptr, q, q_scale, stream);
}

}  // extern "C"
