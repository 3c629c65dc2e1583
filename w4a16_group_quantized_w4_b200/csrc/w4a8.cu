// w4a8_linear: y = xs * (xq (s q)^T), 8-bit activation rows times 4-bit group-32 weights.
//
// Inside a group of 32 the products of int8 activations and int4 codes are summed exactly in integers by
// one m16n8k32 product (16 weight rows, 8 tokens); a group's sum times its bf16 scale is accumulated in
// float32, and the row's scale is applied once at the end.
//   * A code word of layout L1 holds 8 consecutive elements.  Flipping the top bit of its nibbles makes
//     them two's complement; masked in place (odd elements) or shifted up by 4 (even ones) they are bytes
//     16 q, so a word becomes two operand registers in three operations, and no offset has to be taken
//     back.  The activation side is put in the same order, even elements and odd ones.
//   * The product starts from 0x4B400000, the bits of 1.5 * 2^23: |16 * sum| <= 2^19, so the integer
//     result read as a float32 is that number plus the sum, exactly, and one subtraction converts it.
//
// Three ways.  Few rows (M <= 32, and the rows fit in shared memory): bound by the weights' bytes, which
// each warp streams through its own ring of stages (TMA tiles) with no block-wide wait; the rows lie in
// shared memory as ready operands.  More rows: tiles of 128 weight rows by 16 to 64 tokens, 256 k a stage.
// Many rows of shapes that fit it: the tensor-memory kernel of tm_gemm.cu on fp16 rows, to which 8-bit rows
// convert exactly; there a sum runs over products of 24 bits, exact each, in float32 throughout.  It begins on the
// codes while the conversion runs (512 x 2816 x 2816 24.0 us, 25.4 one after the other).
#include <cuda.h>
#include <cudaTypedefs.h>

#include "entry.cuh"
#include "tcgen05.cuh"

// from tm_gemm.cu
bool w4_tm_supported(int N, int K, int epi);
w4_status w4_launch_tm_prepared(const uint32_t* codes, const uint16_t* scales, const int32_t* offsets, int E,
                                int64_t rows, int N, int K, int epi, uint16_t* out, void* ws, int32_t* dev_status,
                                cudaStream_t stream, int sm_count, int early_block, int stall);

namespace w4 {
namespace a8 {

constexpr uint32_t kMagic = 0x4B400000u;
constexpr float kMagicF = 12582912.f;

// 16 * q of the odd (even: after a shift by 4) elements of a code word
__device__ __forceinline__ uint32_t codes_hi(uint32_t w) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0x28;" : "=r"(r) : "r"(w), "r"(0x80808080u), "r"(0xF0F0F0F0u));   // (a ^ b) & c
  return r;
}

__device__ __forceinline__ void mma_s8(uint32_t (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
  asm("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "r"(kMagic));
}

// acc (two neighbouring tokens) += s * (sums - magic), as packed float32 pairs
__device__ __forceinline__ void add_scaled(uint64_t& acc, uint32_t d0, uint32_t d1, uint64_t ss) {
  uint64_t v, m;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "r"(d0), "r"(d1));
  asm("mov.b64 %0, {%1, %1};" : "=l"(m) : "f"(-kMagicF));
  asm("add.rn.f32x2 %0, %0, %1;" : "+l"(v) : "l"(m));
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(v), "l"(ss));
}
__device__ __forceinline__ uint64_t twice(float s) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %1};" : "=l"(v) : "f"(s));
  return v;
}
__device__ __forceinline__ void halves(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}

struct Args {
  const int8_t* x;
  const float* xs;
  const uint32_t* codes;
  const uint16_t* scales;
  uint16_t* y;
  int64_t M, N;
  int K, KG;                       // KG = K / 32 groups
  int eights, more;                // few rows: a block's runs of 8 weight rows; the first `more` have one more
  float* parts;                    // [splits][M][N], when K is split over blocks
  int32_t* dev_status;             // W4_ERR_TIMEOUT where a wait ran out; the sums behind it are NaN
  uint64_t wait_ns;                // limit of every bounded wait
  int stall;                       // fault injection for tests: a ring's copies from this stage on are left out
};

// ------------------------------------------------------------------------------------ few rows
constexpr int kUnitRows = 16, kUnitGroups = 8;           // a stage: 16 weight rows by 256 k
constexpr int kCodeBytes = kUnitRows * 16 * kUnitGroups;  // of a stage; its scales follow all stages' codes
constexpr int kScaleBytes = kUnitRows * 2 * kUnitGroups;
constexpr int kStageBytes = kCodeBytes + kScaleBytes;
// Stages of a warp's ring.  Two: 16 warps have 70 KB in flight, which is enough, and more of these boxes (16 rows
// of 128 bytes each) in flight make the memory slower: the copies alone took 6.9 us with 2 stages and 8.2
// with 6 for 14336 x 4096 codes, and the kernel at M 1 9.5 and 10.3 us.
constexpr int kMostStages = 2;

// What a warp works on, in order: its share of pass after pass (see few_kernel).
struct Walk {
  int W, warp, tiles, KT;
  int pass, tile, kt, left;        // pass, tile of the pass, its stage, stages left to this warp in the pass
  __device__ __forceinline__ int pass_tiles(int p) const { return min(W, tiles - p * W); }
  // goes to the first pass from `pass` on that leaves this warp anything
  __device__ __forceinline__ bool enter() {
    for (; pass * W < tiles; ++pass) {
      const int U = pass_tiles(pass) * KT, u = U < W ? min(warp, U) : U * warp / W;
      left = (U < W ? min(warp + 1, U) : U * (warp + 1) / W) - u;
      tile = u / KT;
      kt = u - tile * KT;
      if (left > 0) return true;
    }
    return false;
  }
  __device__ __forceinline__ bool next() {
    if (--left > 0) {
      if (++kt == KT) {
        kt = 0;
        ++tile;
      }
      return true;
    }
    ++pass;
    return enter();
  }
};

// W warps, NT blocks of 8 tokens.  SB: 16 where the scales come by TMA (their rows are 16-byte aligned), else
// the bytes of a scale load (4 or 2, by their alignment).
// A block owns a run of weight rows (multiples of 8) in passes of up to W tiles of 16; a pass's tiles times
// their stages form a line that the warps share evenly, and the parts that warps have of a tile are joined
// in shared memory, in order.  Every warp refills its own ring as it frees a stage: one feeding warp for all
// (a lane per ring) saved instructions but was slower, 14.4 us against 11.7 at M 16, 12.3 against 11.0 at M 1.
template <int W, int NT, int SB>
__global__ void __launch_bounds__(32 * W, 1)
few_kernel(const __grid_constant__ CUtensorMap codes16, const __grid_constant__ CUtensorMap codes8,
           const __grid_constant__ CUtensorMap scales16, const Args a, int S) {
  extern __shared__ __align__(16) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, t = lane & 3;
  const int KT = (a.KG + kUnitGroups - 1) / kUnitGroups;
  uint8_t* rings = smem + (-smem_u32(smem) & 1023u);    // [W][S] codes (the swizzle goes by 1024 bytes), then scales
  uint2* xf = reinterpret_cast<uint2*>(rings + W * S * kStageBytes);            // [NT][8 KT][32] operands
  // sums of the parts of a pass's tiles: the part that warp w has of a tile lies at w + tile, so a tile's
  // parts follow one another in the order of their stages
  float* red = reinterpret_cast<float*>(xf + static_cast<size_t>(NT) * KT * kUnitGroups * 32);   // [2 W][8 NT][16]
  __shared__ int s_first[W], s_last[W];                                        // a tile's first and last warp
  __shared__ uint64_t s_full[W][kMostStages];

  const int c = blockIdx.x;
  const int64_t row_begin = (static_cast<int64_t>(c) * a.eights + min(c, a.more)) * 8;
  const int64_t row_end = min(a.N, row_begin + (a.eights + (c < a.more ? 1 : 0)) * 8);
  const int tiles = static_cast<int>((row_end - row_begin + kUnitRows - 1) / kUnitRows);
  if (lane < kMostStages) mbar_init(&s_full[warp][lane], 1);
  if (threadIdx.x == 0) {
    prefetch_tmap(&codes16);
    prefetch_tmap(&codes8);
    if (SB == 16) prefetch_tmap(&scales16);
  }
  fence_barrier_init();
  __syncwarp();

  // Copies p's stage into place st of the ring of warp p.warp.  Boxes of 16 rows by 128 bytes of codes (8 rows
  // where the block has no more; a box is zero past the matrix), and 16 rows of scales; rows that are not
  // this block's feed sums that are not written.
  auto fetch = [&](const Walk& p, int st) {
    const int64_t row0 = row_begin + (p.pass * W + p.tile) * kUnitRows;
    const bool both = row_end - row0 > 8;
    uint64_t* bar = &s_full[p.warp][st];
    mbar_arrive_expect_tx(bar, (both ? kCodeBytes : kCodeBytes / 2) + (SB == 16 ? kScaleBytes : 0));
    tma_load_2d(rings + (p.warp * S + st) * kCodeBytes, both ? &codes16 : &codes8, p.kt * 4 * kUnitGroups,
                static_cast<int>(row0), bar);
    if constexpr (SB == 16)
      tma_load_2d(rings + W * S * kCodeBytes + (p.warp * S + st) * kScaleBytes, &scales16, p.kt * kUnitGroups,
                  static_cast<int>(row0), bar);
  };

  // The rows become operands while the first stages are on their way: lane (r, t) of token block b, group g
  // holds the even and the odd ones of elements 32 g + 8 t .. + 7 of token 8 b + r.  A lane turns 16 bytes of
  // a row into the operands of two neighbouring lanes.  The first batch of loads goes out before the ring's.
  constexpr int kBatch = 8 / NT;                       // 8 loads in flight a lane
  uint4 v[NT][kBatch];
  auto load_x = [&](int p0) {
#pragma unroll
    for (int b = 0; b < NT; ++b) {
      const int64_t m = b * 8 + r;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int g = 2 * (p0 + i * W) + (t >> 1);
        v[b][i] = m < a.M && g < a.KG ? __ldg(reinterpret_cast<const uint4*>(a.x + m * a.K + g * 32) + (t & 1))
                                      : make_uint4(0, 0, 0, 0);
      }
    }
  };
  load_x(warp);
  Walk at{W, warp, tiles, KT, 0, 0, 0, 0};
  bool have = at.enter();
  Walk ahead = at;                                     // the next stage to fetch
  bool more = have;
  int issued = 0, used = 0;                            // stages of this warp's ring
  for (int i = 0; i < S && more; ++i) {
    if (lane == 0 && issued < a.stall) fetch(ahead, i);
    ++issued;
    more = ahead.next();
  }
  for (int p0 = warp; p0 < KT * (kUnitGroups / 2); p0 += W * kBatch) {
    if (p0 != warp) load_x(p0);
#pragma unroll
    for (int b = 0; b < NT; ++b)
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int g = 2 * (p0 + i * W) + (t >> 1);
        if (g < KT * kUnitGroups)
          *reinterpret_cast<uint4*>(xf + (b * KT * kUnitGroups + g) * 32 + r * 4 + 2 * (t & 1)) =
              make_uint4(__byte_perm(v[b][i].x, v[b][i].y, 0x6420), __byte_perm(v[b][i].x, v[b][i].y, 0x7531),
                         __byte_perm(v[b][i].z, v[b][i].w, 0x6420), __byte_perm(v[b][i].z, v[b][i].w, 0x7531));
      }
  }
  __syncthreads();

  // scales of this lane's rows r and r + 8, two groups a word; loaded a stage ahead where they do not come by TMA
  uint32_t next_sw[2][4];
  auto load_scales = [&](const Walk& p) {
    const int64_t row0 = row_begin + (p.pass * W + p.tile) * kUnitRows + r;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int g = p.kt * kUnitGroups + 2 * j;
        const int64_t row = row0 + 8 * h;
        const uint16_t* at_ = a.scales + row * a.KG + g;
        const bool on = row < row_end && g < a.KG;
        if constexpr (SB == 4) next_sw[h][j] = on ? __ldg(reinterpret_cast<const uint32_t*>(at_)) : 0u;
        else
          next_sw[h][j] = (on ? ldg_u16(at_) : 0u) | (on && g + 1 < a.KG ? static_cast<uint32_t>(ldg_u16(at_ + 1)) << 16 : 0u);
      }
  };
  if constexpr (SB != 16)
    if (have) load_scales(at);

  const uint32_t ring = smem_u32(rings) + warp * S * kCodeBytes;             // codes: 128-byte swizzled rows
  const uint32_t sring = smem_u32(rings) + W * S * kCodeBytes + warp * S * kScaleBytes;
  uint64_t acc[NT][2];
#pragma unroll
  for (int b = 0; b < NT; ++b) acc[b][0] = acc[b][1] = 0;
  int st = 0;
  uint32_t parity = 0;                                 // of the ring's current round
  bool alive = true;                                   // false once a bounded wait ran out: no more waits or copies
  int swz[kUnitGroups];                                // where this lane's word of group g lies in a swizzled row
#pragma unroll
  for (int g = 0; g < kUnitGroups; ++g) swz[g] = r * 128 + ((g ^ r) << 4) + t * 4;
  const uint32_t xbase = smem_u32(xf) + lane * 8;
  for (int pass = 0; pass * W < tiles; ++pass) {
    while (have && at.pass == pass) {
      // the run of stages that this warp has of a tile
      const int tile = at.tile, k0 = at.kt, run = min(at.left, KT - k0);
      uint32_t xk = xbase + k0 * (kUnitGroups * 256);
      for (int u = 0; u < run; ++u, xk += kUnitGroups * 256) {
        if (alive && !mbar_wait_ring(&s_full[warp][st], parity, a.wait_ns)) {
          alive = false;
          set_status(a.dev_status, W4_ERR_TIMEOUT);
          // A stage that has not arrived is not asked for again, and what is on its way lands before the end.
          if (lane == 0)
            for (int i = used; i < min(issued, a.stall); ++i) mbar_wait_ring(&s_full[warp][i % S], (i / S) & 1);
        }
        const uint32_t base = ring + st * kCodeBytes;
        uint32_t sw[2][4];
        if constexpr (SB == 16) {
          const uint4 s0 = lds128(sring + st * kScaleBytes + r * 16), s1 = lds128(sring + st * kScaleBytes + (r + 8) * 16);
          sw[0][0] = s0.x; sw[0][1] = s0.y; sw[0][2] = s0.z; sw[0][3] = s0.w;
          sw[1][0] = s1.x; sw[1][1] = s1.y; sw[1][2] = s1.z; sw[1][3] = s1.w;
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) sw[j >> 2][j & 3] = next_sw[j >> 2][j & 3];
          at.kt = k0 + u + 1;                          // (the next stage's scales, if the run has one)
          if (u + 1 < run) load_scales(at);
        }
#pragma unroll
        for (int g = 0; g < kUnitGroups; ++g) {
          const uint32_t w0 = lds32(base + swz[g]), w1 = lds32(base + swz[g] + kCodeBytes / 2);
          const uint32_t a0 = codes_hi(w0 << 4), a1 = codes_hi(w1 << 4), a2 = codes_hi(w0), a3 = codes_hi(w1);
          const uint64_t q0 = twice(g & 1 ? bf16_hi_to_f32(sw[0][g / 2]) : bf16_lo_to_f32(sw[0][g / 2]));
          const uint64_t q1 = twice(g & 1 ? bf16_hi_to_f32(sw[1][g / 2]) : bf16_lo_to_f32(sw[1][g / 2]));
#pragma unroll
          for (int b = 0; b < NT; ++b) {
            const uint2 x = lds64(xk + (b * KT * kUnitGroups + g) * 256);
            uint32_t d[4];
            mma_s8(d, a0, a1, a2, a3, x.x, x.y);
            add_scaled(acc[b][0], d[0], d[1], q0);
            add_scaled(acc[b][1], d[2], d[3], q1);
          }
        }
        __syncwarp();                                  // the stage has been read
        ++used;
        if (more) {
          if (lane == 0 && alive && issued < a.stall) fetch(ahead, st);
          ++issued;
          more = ahead.next();
        }
        if (++st == S) {
          st = 0;
          parity ^= 1;
        }
      }
      float* o = red + (warp + tile) * (8 * NT * 16);            // [token][row]
#pragma unroll
      for (int b = 0; b < NT; ++b)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float lo, hi;
          halves(acc[b][h], lo, hi);
          if (!alive) lo = hi = __int_as_float(0x7FC00000);
          o[(8 * b + 2 * t) * 16 + r + 8 * h] = lo;
          o[(8 * b + 2 * t + 1) * 16 + r + 8 * h] = hi;
          acc[b][h] = 0;
        }
      if (lane == 0 && k0 == 0) s_first[tile] = warp;
      if (lane == 0 && k0 + run == KT) s_last[tile] = warp;
      at.kt = k0 + run - 1;
      at.left -= run - 1;
      have = at.next();
      if constexpr (SB != 16)
        if (have) load_scales(at);
    }
    __syncthreads();
    // a thread sums 4 rows of a token over the tile's parts, in order
    const int pt = at.pass_tiles(pass);
    for (int i = threadIdx.x; i < pt * 32 * NT; i += 32 * W) {
      const int quad = i & 3, m = (i >> 2) % (8 * NT), tile = (i >> 2) / (8 * NT);
      const int64_t n = row_begin + (pass * W + tile) * kUnitRows + quad * 4;
      if (m >= a.M || n >= row_end) continue;
      const float4* part = reinterpret_cast<const float4*>(red) + ((s_first[tile] + tile) * 8 * NT + m) * 4 + quad;
      float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int w = s_first[tile]; w <= s_last[tile]; ++w, part += 8 * NT * 4) {
        sum.x += part->x;
        sum.y += part->y;
        sum.z += part->z;
        sum.w += part->w;
      }
      const float f = 0.0625f * __ldg(a.xs + m);
      const uint2 o = make_uint2(pack_bf16x2(sum.x * f, sum.y * f), pack_bf16x2(sum.z * f, sum.w * f));
      uint16_t* y = a.y + m * a.N + n;
      if (a.N % 4 == 0) {
        *reinterpret_cast<uint2*>(y) = o;
      } else {
        const uint16_t h[4] = {static_cast<uint16_t>(o.x), static_cast<uint16_t>(o.x >> 16), static_cast<uint16_t>(o.y),
                               static_cast<uint16_t>(o.y >> 16)};
        for (int q = 0; q < 4; ++q)
          if (n + q < row_end) y[q] = h[q];
      }
    }
    __syncthreads();
  }
}

// ----------------------------------------------------------------------------------- more rows
// Tiles of 128 weight rows by BM tokens, 256 k a stage, everything by TMA into 128-byte swizzled rows.
// A warp holds MT x NT products (32 weight rows by 32 tokens at BM = 64); the blocks of 8 tokens are read
// in the order 0, 2, 4, 6, 1, 3, 5, 7, which keeps the 8-byte reads of half a warp free of bank conflicts
// under the swizzle.  Bound by instructions: about ten a product, of which four are the float32 pairs.
constexpr int kBN = 128, kGS = 8;                        // weight rows of a tile, groups a stage

template <int BM>
struct Many {
  static constexpr int WR = BM >= 64 ? 4 : 8, WC = 8 / WR;         // warps over rows, over tokens
  static constexpr int MT = kBN / 16 / WR, NT = BM / 8 / WC;       // 16-row and 8-token blocks of a warp
  static constexpr int S = 3;
  static constexpr int kX = kBN * 16 * kGS, kScales = kX + 2 * BM * 128, kStage = kScales + kBN * 2 * kGS;
  static constexpr int kOut = BM * (kBN + 4) * 4;
  static constexpr int kSmem = (S * kStage > kOut ? S * kStage : kOut) + 1024;
};

// blockIdx.x: token tile (fastest, so that a weight tile is shared in L2), y: row tile, z: part of K.
template <int BM, int SB>
__global__ void __launch_bounds__(256, 2)
many_kernel(const __grid_constant__ CUtensorMap codes_map, const __grid_constant__ CUtensorMap scales_map,
            const __grid_constant__ CUtensorMap x_map, const Args a) {
  using C = Many<BM>;
  extern __shared__ __align__(16) uint8_t smem_[];
  uint8_t* smem = smem_ + (-smem_u32(smem_) & 1023u);
  __shared__ uint64_t s_bar[C::S];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, t = lane & 3;
  const int wr = warp % C::WR, wc = warp / C::WR;
  const int64_t m0 = static_cast<int64_t>(blockIdx.x) * BM, n0 = static_cast<int64_t>(blockIdx.y) * kBN;
  const int KT = (a.KG + kGS - 1) / kGS;
  const int k0 = static_cast<int>(static_cast<int64_t>(KT) * blockIdx.z / gridDim.z);
  const int k1 = static_cast<int>(static_cast<int64_t>(KT) * (blockIdx.z + 1) / gridDim.z);
  const uint32_t s0 = smem_u32(smem);
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::S; ++i) mbar_init(s_bar + i, 1);
    fence_barrier_init();
  }
  __syncthreads();

  bool alive = true;                                       // false once a bounded wait ran out: no more waits or copies
  auto fetch = [&](int kt, int st) {
    uint8_t* base = smem + st * C::kStage;
    if (threadIdx.x == 0 && alive && kt - k0 < a.stall) {
      mbar_arrive_expect_tx(s_bar + st, SB == 16 ? C::kStage : C::kScales);
      tma_load_2d(base, &codes_map, kt * 4 * kGS, static_cast<int>(n0), s_bar + st);
      tma_load_2d(base + C::kX, &x_map, kt * 256, static_cast<int>(m0), s_bar + st);
      tma_load_2d(base + C::kX + BM * 128, &x_map, kt * 256 + 128, static_cast<int>(m0), s_bar + st);
      if constexpr (SB == 16) tma_load_2d(base + C::kScales, &scales_map, kt * kGS, static_cast<int>(n0), s_bar + st);
    }
    if constexpr (SB != 16) {                            // (visible with the block's next barrier)
#pragma unroll
      for (int i = 0; i < kBN * kGS / 256; ++i) {
        const int c = i * 256 + threadIdx.x, row = c / kGS, g = kt * kGS + c % kGS;
        const uint16_t v = n0 + row < a.N && g < a.KG ? ldg_u16(a.scales + (n0 + row) * a.KG + g) : 0;
        *reinterpret_cast<uint16_t*>(base + C::kScales + c * 2) = v;
      }
    }
  };

  uint64_t acc[C::MT][C::NT][2];
#pragma unroll
  for (int i = 0; i < C::MT; ++i)
#pragma unroll
    for (int j = 0; j < C::NT; ++j) acc[i][j][0] = acc[i][j][1] = 0;

  for (int i = 0; i < C::S - 1; ++i)
    if (k0 + i < k1) fetch(k0 + i, i);
  const int tok = 2 * (r & 3) + (r >> 2);                  // the token of this lane's operand, of 8
  const uint32_t wb = s0 + (wr * C::MT * 16 + r) * 128 + t * 4;
  const uint32_t xb = s0 + C::kX + (wc * C::NT * 8 + tok) * 128 + (t & 1) * 8;
  int st = 0;
  uint32_t parity = 0;
  for (int kt = k0; kt < k1; ++kt) {
    if (alive && !mbar_wait_ring(s_bar + st, parity, a.wait_ns)) {
      alive = false;
      set_status(a.dev_status, W4_ERR_TIMEOUT);
      // A stage that has not arrived is not asked for again, and what is on its way lands before the end.
      if (threadIdx.x == 0)
        for (int i = kt - k0; i < min(min(kt + C::S - 1, k1) - k0, a.stall); ++i) mbar_wait_ring(s_bar + i % C::S, (i / C::S) & 1);
    }
    __syncthreads();
    if (kt + C::S - 1 < k1) fetch(kt + C::S - 1, st == 0 ? C::S - 1 : st - 1);
    const uint32_t off = st * C::kStage;
    uint4 sw[C::MT][2];
#pragma unroll
    for (int i = 0; i < C::MT; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) sw[i][h] = lds128(s0 + off + C::kScales + (wr * C::MT * 16 + i * 16 + h * 8 + r) * 16);
#pragma unroll
    for (int g = 0; g < kGS; ++g) {
      uint32_t xe[C::NT], xo[C::NT];
      const uint32_t xg = xb + off + (g / 4) * (BM * 128) + (((2 * (g % 4) + (t >> 1)) ^ tok) << 4);
      const uint32_t wg = wb + off + ((g ^ r) << 4);
#pragma unroll
      for (int j = 0; j < C::NT; ++j) {
        const uint2 x = lds64(xg + j * 1024);
        xe[j] = __byte_perm(x.x, x.y, 0x6420);
        xo[j] = __byte_perm(x.x, x.y, 0x7531);
      }
#pragma unroll
      for (int i = 0; i < C::MT; ++i) {
        const uint32_t w0 = lds32(wg + i * 2048), w1 = lds32(wg + i * 2048 + 1024);
        const uint32_t a0 = codes_hi(w0 << 4), a1 = codes_hi(w1 << 4), a2 = codes_hi(w0), a3 = codes_hi(w1);
        const uint32_t p0 = reinterpret_cast<const uint32_t*>(&sw[i][0])[g / 2], p1 = reinterpret_cast<const uint32_t*>(&sw[i][1])[g / 2];
        const uint64_t q0 = twice(g & 1 ? bf16_hi_to_f32(p0) : bf16_lo_to_f32(p0));
        const uint64_t q1 = twice(g & 1 ? bf16_hi_to_f32(p1) : bf16_lo_to_f32(p1));
#pragma unroll
        for (int j = 0; j < C::NT; ++j) {
          uint32_t d[4];
          mma_s8(d, a0, a1, a2, a3, xe[j], xo[j]);
          add_scaled(acc[i][j][0], d[0], d[1], q0);
          add_scaled(acc[i][j][1], d[2], d[3], q1);
        }
      }
    }
    if (++st == C::S) {
      st = 0;
      parity ^= 1;
    }
  }
  __syncthreads();
  float* o = reinterpret_cast<float*>(smem);               // [token][kBN + 4]
#pragma unroll
  for (int i = 0; i < C::MT; ++i)
#pragma unroll
    for (int j = 0; j < C::NT; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float lo, hi;
        halves(acc[i][j][h], lo, hi);
        if (!alive) lo = hi = __int_as_float(0x7FC00000);
        // columns 2 t and 2 t + 1 of the product are these tokens
        const int m = wc * C::NT * 8 + j * 8, n = wr * C::MT * 16 + i * 16 + h * 8 + r;
        o[(m + 4 * (t & 1) + (t >> 1)) * (kBN + 4) + n] = lo;
        o[(m + 4 * (t & 1) + 2 + (t >> 1)) * (kBN + 4) + n] = hi;
      }
  __syncthreads();
  for (int i = threadIdx.x; i < BM * kBN; i += 256) {
    const int m = i / kBN, n = i % kBN;
    if (m0 + m >= a.M || n0 + n >= a.N) continue;
    const float v = o[m * (kBN + 4) + n];
    if (gridDim.z > 1) a.parts[(blockIdx.z * a.M + m0 + m) * a.N + n0 + n] = v;
    else a.y[(m0 + m) * a.N + n0 + n] = f32_to_bf16_bits(v * 0.0625f * __ldg(a.xs + m0 + m));
  }
}

// sums the parts of a split K in order
__global__ void __launch_bounds__(256) parts_kernel(const Args a, int splits) {
  pdl_wait();
  const int64_t total = a.M * a.N;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < total; i += static_cast<int64_t>(gridDim.x) * 256) {
    float v = 0.f;
    for (int z = 0; z < splits; ++z) v += a.parts[z * total + i];
    a.y[i] = f32_to_bf16_bits(v * 0.0625f * __ldg(a.xs + i / a.N));
  }
}

// ----------------------------------------------------------------------------------- dispatch
constexpr int kSmemMost = 232448 - 2048 - 1024;   // less the static arrays and the ring's alignment

// How the few-rows kernel is run: W warps, NT token blocks, S stages; S = 0 where the rows leave no room.
// 16 warps hide the latency of a warp's chain of products better (M 16, N 14336, K 4096: 17.9 us against
// 19.8 us with 8 when it was chosen), where their rings fit.
struct Few {
  int W, NT, S, smem;
};
Few few_plan(int64_t M, int64_t KG) {
  Few f{16, M <= 8 ? 1 : M <= 16 ? 2 : 4, 0, 0};
  if (M > 32) return f;
  const int64_t x = f.NT * ((KG + kUnitGroups - 1) / kUnitGroups) * kUnitGroups * 256;
  for (f.W = 16; f.W >= 8; f.W -= 8) {
    const int64_t red = f.W * 2 * 8 * f.NT * 16 * 4, S = (kSmemMost - x - red) / (f.W * kStageBytes);
    if (S < 2) continue;
    f.S = S > kMostStages ? kMostStages : static_cast<int>(S);
    f.smem = static_cast<int>(x + red + f.W * f.S * kStageBytes);
    return f;
  }
  return f;
}

int many_tile(int64_t M) { return M <= 16 ? 16 : M <= 32 ? 32 : 64; }

int64_t many_tiles(int64_t M, int64_t N) {
  const int BM = many_tile(M);
  return (M + BM - 1) / BM * ((N + kBN - 1) / kBN);
}

// Parts of K: enough to give every SM two blocks, each at least 1024 k long
int many_splits(int64_t M, int64_t N, int64_t KG, int sms) {
  const int64_t want = 2 * sms / many_tiles(M, N), most = KG / 32;
  const int64_t s = want < most ? want : most;
  return s < 2 ? 1 : s > 16 ? 16 : static_cast<int>(s);
}

// The tensor-memory kernel's token block (0: the kernel above is the faster one, or the only one).  That one works
// in tiles of 128 weight rows by `block` tokens, one an SM at a time, at about 5.4 ns a k of a tile for blocks of
// 192 and 6.6 for 256, behind 7.5 us for the conversion, the beginning and the end.  Measured with 192 and 256: 509 x
// 8192 x 2816 39.5 and 27.3 us (192 tiles or 128, for 148 SMs), 2048 x 8192 x 4096 125 and 119, 512 x 2816 x 2816
// 23.3 and 25.4, 128 x 14336 x 4096 30.4 and 32.5.  The kernel above takes about 7.6 ns a k of a tile of 128 by 64
// where an SM has one, 11 where it has two, on 4 us, and for a split K 2 us and the parts' bytes more: 64 x 14336 x
// 4096 34 us (29 with the other), 33 x 28672 x 4096 49 (52), 64 x 4096 x 4096 13 (27).
int tm_block(int64_t M, int64_t N, int64_t K, int sms) {
  if (M > 0x7FFFFFFF - 256 || !w4_tm_supported(static_cast<int>(N), static_cast<int>(K), W4_EPI_NONE)) return 0;
  auto waves = [&](int64_t tiles, int64_t at_once) { return static_cast<double>((tiles + at_once - 1) / at_once); };
  const double w192 = waves(N / 128 * ((M + 191) / 192), sms) * 5.4e-9, w256 = waves(N / 128 * ((M + 255) / 256), sms) * 6.6e-9;
  const double tm = 7.5e-6 + K * (w192 < w256 ? w192 : w256);
  const int splits = many_splits(M, N, K / 32, sms);
  const int64_t blocks = many_tiles(M, N) * splits;
  double many = 4e-6 + (blocks <= sms ? 7.6e-9 : waves(blocks, 2 * sms) * 11e-9) * K / splits;
  if (splits > 1) many += 2e-6 + splits * M * N * 8 / 6.5e12;
  return many <= tm ? 0 : w192 < w256 ? 192 : 256;
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  if (!fn) {
    cudaDriverEntryPointQueryResult q;
    void* p = nullptr;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }
  return fn;
}

// [rows, wide] elements of `size` bytes as boxes of `box` elements by `high` rows
bool encode(CUtensorMap* m, const void* p, CUtensorMapDataType type, int size, int64_t rows, int64_t wide, int box,
            int high, CUtensorMapSwizzle swizzle) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(wide), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(wide) * size};
  cuuint32_t boxes[2] = {static_cast<cuuint32_t>(box), static_cast<cuuint32_t>(high)}, estr[2] = {1, 1};
  return fn(m, type, 2, const_cast<void*>(p), dims, strides, boxes, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
            CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int W, int NT>
w4_status launch_few(const Args& a, const Few& f, int SB, int sms, cudaStream_t s) {
  auto kernel = SB == 16 ? few_kernel<W, NT, 16> : SB >= 4 ? few_kernel<W, NT, 4> : few_kernel<W, NT, 2>;
  static SmemRaised raised[3];
  if (raise_smem(kernel, kSmemMost + 1024, raised[SB == 16 ? 0 : SB >= 4 ? 1 : 2]) != cudaSuccess) return W4_ERR_CUDA;
  CUtensorMap codes16, codes8, scales;
  for (int high : {16, 8})
    if (!encode(high == 16 ? &codes16 : &codes8, a.codes, CU_TENSOR_MAP_DATA_TYPE_UINT32, 4, a.N, a.K / 8,
                4 * kUnitGroups, high, CU_TENSOR_MAP_SWIZZLE_128B))
      return W4_ERR_CUDA;
  if (SB != 16) scales = codes16;                      // (not used)
  else if (!encode(&scales, a.scales, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, a.N, a.KG, kUnitGroups, 16,
                   CU_TENSOR_MAP_SWIZZLE_NONE))
    return W4_ERR_CUDA;
  const int64_t R8 = (a.N + 7) / 8;
  const int grid = static_cast<int>(R8 < sms ? R8 : sms);
  Args b = a;
  b.eights = static_cast<int>(R8 / grid);
  b.more = static_cast<int>(R8 % grid);
  kernel<<<grid, 32 * W, f.smem + 1024, s>>>(codes16, codes8, scales, b, f.S);
  return cudaGetLastError() == cudaSuccess ? W4_OK : W4_ERR_CUDA;
}

template <int W>
w4_status launch_few(const Args& a, const Few& f, int SB, int sms, cudaStream_t s) {
  return f.NT == 1 ? launch_few<W, 1>(a, f, SB, sms, s)
         : f.NT == 2 ? launch_few<W, 2>(a, f, SB, sms, s) : launch_few<W, 4>(a, f, SB, sms, s);
}

template <int BM>
w4_status launch_many(const Args& a, int splits, int SB, int sms, cudaStream_t s) {
  auto kernel = SB == 16 ? many_kernel<BM, 16> : many_kernel<BM, 2>;
  static SmemRaised raised[2];
  if (raise_smem(kernel, Many<BM>::kSmem, raised[SB == 16]) != cudaSuccess) return W4_ERR_CUDA;
  CUtensorMap codes, scales, x;
  if (!encode(&codes, a.codes, CU_TENSOR_MAP_DATA_TYPE_UINT32, 4, a.N, a.K / 8, 4 * kGS, kBN, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode(&x, a.x, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, a.M, a.K, 128, BM, CU_TENSOR_MAP_SWIZZLE_128B))
    return W4_ERR_CUDA;
  if (SB != 16) scales = codes;                        // (not used)
  else if (!encode(&scales, a.scales, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, a.N, a.KG, kGS, kBN, CU_TENSOR_MAP_SWIZZLE_NONE))
    return W4_ERR_CUDA;
  const int64_t tm = (a.M + BM - 1) / BM, tn = (a.N + kBN - 1) / kBN;
  const dim3 grid(static_cast<unsigned>(tm), static_cast<unsigned>(tn), splits);
  kernel<<<grid, 256, Many<BM>::kSmem, s>>>(codes, scales, x, a);
  if (cudaGetLastError() != cudaSuccess) return W4_ERR_CUDA;
  if (splits == 1) return W4_OK;
  const int64_t blocks = (a.M * a.N + 255) / 256;
  return launch_pdl(parts_kernel, dim3(static_cast<unsigned>(blocks < 4 * sms ? blocks : 4 * sms)), dim3(256), 0, s, a,
                    splits) == cudaSuccess ? W4_OK : W4_ERR_CUDA;
}

}  // namespace a8
}  // namespace w4

size_t w4_linear8_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  if (M < 1 || N < 1 || K < 32 || K % 32 || N > (1LL << 30) || K > (1LL << 30)) return 0;
  if (w4::a8::few_plan(M, K / 32).S) return 0;
  const int splits = w4::a8::many_splits(M, N, K / 32, w4::device_sm_count());
  const size_t parts = splits > 1 ? static_cast<size_t>(splits) * M * N * 4 : 0;
  if (!w4::a8::tm_block(M, N, K, w4::device_sm_count())) return parts;
  // (scales at an odd address keep the call from the tensor-memory kernel: room for either)
  const size_t rows = w4_tc_workspace_bytes(M, static_cast<int>(K), N);
  return rows > parts ? rows : parts;
}

static w4_status linear8(const int8_t* xq, const float* xs, const uint32_t* codes, const uint16_t* scales, uint16_t* y,
                         int64_t M, int64_t N, int64_t K, void* workspace, size_t workspace_bytes, int32_t* dev_status,
                         void* stream, uint64_t wait_ns, int stall) {
  using namespace w4;
  if (M < 0 || N < 1 || K < 32 || K % 32 || N > (1LL << 30) || K > (1LL << 30)) return W4_ERR_INVALID_ARG;
  if (!codes || !scales || !aligned_to(codes, 16) || !aligned_to(scales, 2)) return W4_ERR_INVALID_ARG;
  if (M > 0 && (!xq || !xs || !y)) return W4_ERR_INVALID_ARG;
  if (!aligned_to(xq, 16) || !aligned_to(xs, 4) || !aligned_to(y, 16) || !aligned_to(workspace, 16))
    return W4_ERR_INVALID_ARG;
  if (M > (1LL << 40) / N || M > 0x7FFFFFFFLL) return W4_ERR_UNSUPPORTED;
  if (M == 0) return W4_OK;
  const size_t need = w4_linear8_workspace_bytes(M, N, K);
  if (need && (!workspace || workspace_bytes < need)) return W4_ERR_WORKSPACE;
  a8::Args a{xq, xs, codes, scales, y, M, N, static_cast<int>(K), static_cast<int>(K / 32), 0, 0, static_cast<float*>(workspace),
             dev_status, wait_ns, stall};
  auto s = static_cast<cudaStream_t>(stream);
  const int sms = device_sm_count();
  // what a copy of consecutive scales may take at once: every row starts at a multiple of it
  const int SB = K % 256 == 0 && aligned_to(scales, 16) ? 16
                 : K % 128 == 0 && aligned_to(scales, 8) ? 8
                 : K % 64 == 0 && aligned_to(scales, 4) ? 4 : 2;
  const a8::Few f = a8::few_plan(M, K / 32);
  if (f.S)
    return w4_record_status(f.W == 16 ? a8::launch_few<16>(a, f, SB, sms, s) : a8::launch_few<8>(a, f, SB, sms, s));
  if (const int block = a8::tm_block(M, N, K, sms); block && aligned_to(scales, 4)) {
    w4_launch_a8_to_f16(xq, xs, M, static_cast<int>(K), scales, N, workspace, s);
    if (cudaGetLastError() != cudaSuccess) return w4_record_status(W4_ERR_CUDA);
    return w4_record_status(w4_launch_tm_prepared(codes, scales, nullptr, 1, M, static_cast<int>(N), static_cast<int>(K),
                                                  W4_EPI_NONE, y, workspace, dev_status, s, sms, block, stall));
  }
  if (N > 65535LL * a8::kBN) return W4_ERR_UNSUPPORTED;       // (a grid's y)
  const int splits = a8::many_splits(M, N, K / 32, sms);
  const int BM = a8::many_tile(M);
  return w4_record_status(BM == 16 ? a8::launch_many<16>(a, splits, SB, sms, s)
                          : BM == 32 ? a8::launch_many<32>(a, splits, SB, sms, s)
                                     : a8::launch_many<64>(a, splits, SB, sms, s));
}

extern "C" {

w4_status w4a8_linear(const int8_t* xq, const float* xs, const uint32_t* codes, const uint16_t* scales, uint16_t* y,
                      int64_t M, int64_t N, int64_t K, void* workspace, size_t workspace_bytes, void* stream) {
  const w4::EntryRange range("w4a8_linear");
  return linear8(xq, xs, codes, scales, y, M, N, K, workspace, workspace_bytes, nullptr, stream, w4::kWaitLimitNs, 0x7FFFFFFF);
}

w4_status w4a8_linear_s(const int8_t* xq, const float* xs, const uint32_t* codes, const uint16_t* scales, uint16_t* y,
                        int64_t M, int64_t N, int64_t K, void* workspace, size_t workspace_bytes, int32_t* dev_status,
                        void* stream) {
  const w4::EntryRange range("w4a8_linear_s");
  return linear8(xq, xs, codes, scales, y, M, N, K, workspace, workspace_bytes, dev_status, stream, w4::kWaitLimitNs, 0x7FFFFFFF);
}

// Fault injection for the tests of the bounded waits (not part of the C ABI in w4a16.h): w4a8_linear with every
// wait limited to wait_ns (the tensor-memory kernel's to kWaitLimitNs as always: a limit of the call's own cost 2%) and every ring's copies from stage stall_after on left out, so that the waits for them run
// out.  The kernels then report W4_ERR_TIMEOUT in dev_status and return; nothing faults or hangs.
w4_status w4_testing_linear8_stall(const int8_t* xq, const float* xs, const uint32_t* codes, const uint16_t* scales,
                                   uint16_t* y, int64_t M, int64_t N, int64_t K, void* workspace, size_t workspace_bytes,
                                   int32_t* dev_status, void* stream, uint64_t wait_ns, int32_t stall_after) {
  const w4::EntryRange range("w4_testing_linear8_stall");
  if (stall_after < 0) return W4_ERR_INVALID_ARG;
  return linear8(xq, xs, codes, scales, y, M, N, K, workspace, workspace_bytes, dev_status, stream, wait_ns, stall_after);
}

}  // extern "C"
