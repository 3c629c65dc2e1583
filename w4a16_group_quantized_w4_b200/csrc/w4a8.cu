// w4a8_linear: y = xs * (xq (s q)^T), 8-bit activation rows times 4-bit group-32 weights.
//
// Inside a group of 32 the products of int8 activations and int4 codes are summed exactly in
// integers; a group's sum times its bf16 scale is accumulated in float32, and the row's scale is
// applied once at the end.
//
// First form: one warp per output, a lane per group (four dp4a pairs of a 16-byte code load and
// two 16-byte activation loads).
#include "common.cuh"
#include "entry.cuh"

namespace w4 {
namespace a8 {

__global__ void __launch_bounds__(256)
linear_kernel(const int8_t* __restrict__ xq, const float* __restrict__ xs, const uint32_t* __restrict__ codes,
              const uint16_t* __restrict__ scales, uint16_t* __restrict__ y, int64_t M, int64_t N, int64_t K) {
  const int lane = threadIdx.x & 31;
  const int64_t out = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (out >= M * N) return;
  const int64_t m = out / N, n = out - m * N;
  const int64_t groups = K >> 5;
  float acc = 0.f;
  for (int64_t g = lane; g < groups; g += 32) {
    const uint4 w = __ldg(reinterpret_cast<const uint4*>(codes + n * (K >> 3)) + g);
    const uint4* xr = reinterpret_cast<const uint4*>(xq + m * K) + 2 * g;
    const uint4 x0 = __ldg(xr), x1 = __ldg(xr + 1);
    const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
    const uint32_t xx[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
    int sum = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      // elements 0,2,4,6 and 1,3,5,7 of the word, times 16 as signed bytes
      const int even = static_cast<int>(((ww[j] ^ 0x88888888u) << 4) & 0xF0F0F0F0u);
      const int odd = static_cast<int>((ww[j] ^ 0x88888888u) & 0xF0F0F0F0u);
      sum = __dp4a(even, static_cast<int>(__byte_perm(xx[2 * j], xx[2 * j + 1], 0x6420)), sum);
      sum = __dp4a(odd, static_cast<int>(__byte_perm(xx[2 * j], xx[2 * j + 1], 0x7531)), sum);
    }
    acc = fmaf(static_cast<float>(sum), bf16_lo_to_f32(__ldg(scales + n * groups + g)), acc);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
  if (lane == 0) y[out] = f32_to_bf16_bits(acc * 0.0625f * __ldg(xs + m));
}

}  // namespace a8
}  // namespace w4

extern "C" w4_status w4a8_linear(const int8_t* xq, const float* xs, const uint32_t* codes, const uint16_t* scales,
                                 uint16_t* y, int64_t M, int64_t N, int64_t K, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  using namespace w4;
  const EntryRange range("w4a8_linear");
  if (M < 0 || N < 1 || K < 32 || K % 32 || N > (1LL << 30) || K > (1LL << 30)) return W4_ERR_INVALID_ARG;
  if (!codes || !scales || !aligned_to(codes, 16) || !aligned_to(scales, 2)) return W4_ERR_INVALID_ARG;
  if (M > 0 && (!xq || !xs || !y)) return W4_ERR_INVALID_ARG;
  if (!aligned_to(xq, 16) || !aligned_to(xs, 4) || !aligned_to(y, 16) || !aligned_to(workspace, 16))
    return W4_ERR_INVALID_ARG;
  if (M > (1LL << 40) / N) return W4_ERR_UNSUPPORTED;
  if (M == 0) return W4_OK;
  if (workspace_bytes < w4_workspace_bytes(W4_OP_LINEAR_8, M, N, K, 1, 1) ||
      (!workspace && w4_workspace_bytes(W4_OP_LINEAR_8, M, N, K, 1, 1)))
    return W4_ERR_WORKSPACE;
  const int64_t blocks = (M * N + 7) / 8;
  if (blocks > 0x7FFFFFFFLL) return W4_ERR_UNSUPPORTED;
  a8::linear_kernel<<<static_cast<unsigned>(blocks), 256, 0, static_cast<cudaStream_t>(stream)>>>(xq, xs, codes,
                                                                                               scales, y, M, N, K);
  return launched();
}

size_t w4_linear8_workspace_bytes(int64_t, int64_t, int64_t) { return 0; }
