// The attention kernel of kv_cache_attend (instantiated per cache kind in kv_attend_*.cu).
//
//   out = sum_t p_t v_t / sum_t p_t,  p_t = 2^(z_t - m),  z_t = log2(e) * cap(scale * q . k_t)
//
// One pass over the cache with a running reference m per head.  Bound by the cache's bytes, each of
// which is needed once.  Every warp streams its own tokens, 16 at a time, through its own ring of
// stages in shared memory (cp.async, whole rows, so that many bytes are in flight without registers
// and without a block-wide wait) and reads tensor-core operands from there as whole words:
//   * Scores, S^T = K Q^T: tokens are the 16 rows of an m16n8k16 product, up to 8 query heads of one
//     key/value head its 8 columns.  The product does not care in which order the head dimension
//     is summed, so lane (r, t) = (lane / 4, lane % 4) takes the 8 consecutive elements 32 g + 8 t of
//     token rows r and r + 8.
//   * Outputs, O^T = V^T P^T: head-dimension elements are the 16 rows, tokens the 16 summed ones.  Lane
//     (r, t) takes VE consecutive elements at VE r of tokens 2t, 2t+1, 2t+8, 2t+9; byte permutes pair
//     the tokens up.
// Rows lie in shared memory at a pitch that keeps both reads free of bank conflicts.
//   * The weights p leave the first product with tokens along r and enter the second with tokens
//     along t: one 8x8 register transpose (movmatrix) per 8 tokens.
// Codes are widened to fp16 exactly (a bias is taken back later).  Key scales multiply the float32 sum of their group; value
// scales multiply the widened code in fp16, brought into range by a power of two per output row
// (one more rounding of 2^-11; scaling the weights instead would need a weight per group).  Weights are
// rounded to fp16 against quantised values; against bf16 values they enter as a bf16 pair (high and
// remainder, two products), because a single bf16 would cost as much as the output's own rounding.
//
// Work is cut over all lengths: sequences' (windowed) tokens in units of 64, times key/value heads
// times blocks of 8 query heads, form one line that the blocks of the grid share evenly.  A block that
// holds an item (sequence, heads) whole writes its output; parts go to the workspace and a second
// kernel joins them in order.
#pragma once

#include "common.cuh"
#include "entry.cuh"

namespace w4 {
namespace at {

constexpr int kUnit = 64;             // tokens a work unit
constexpr int kWarps = 4;
constexpr int64_t kMostTokens = 0x7FFFEFFF;   // a sequence's table: token numbers stay below 2^31 past its end
constexpr float kLowest = -3.0e38f;   // reference before any token: finite, so that masked scores give p = 0
constexpr float kSlack = 8.f;         // a reference is raised once a score passes it by 2^kSlack
constexpr float kLift = 6.f;          // weights for fp16 are taken times 2^kLift: at most 2^14

struct Rec {
  int b, item, last;                  // last: the last block that holds a part, -1 for nothing to join
};

struct Args {
  const uint16_t* q;
  int64_t q_stride;
  const void *k, *v;
  const uint16_t *ks, *vs;
  const int32_t *table, *lens;
  int table_width, B, q_heads, kv_heads, page_size;
  int pages;
  float scale, softcap;
  int window;
  uint16_t* out;
  float* lse;
  float* parts;                       // [2 * grid][heads * (D + 2)]: outputs, references, totals of an item's heads
  Rec* recs;                          // [grid]
  int32_t* dev_status;
  // derived
  int G, HB;                          // query heads per key/value head, items they make (8 or 16 heads each)
  uint32_t div_mul;                   // token / page_size = (umulhi(token, div_mul) + token) >> div_shift
  int div_shift;
};

__device__ __forceinline__ int page_of(const Args& a, int tok) {
  return static_cast<int>((__umulhi(static_cast<uint32_t>(tok), a.div_mul) + static_cast<uint32_t>(tok)) >> a.div_shift);
}

// A sequence's visible tokens [first, len), the n units that cover them, and the length of one of its
// items on the line: n and the cost of beginning it.
struct Span {
  int first, len, u0, n, line;
};
__device__ __forceinline__ Span span_of(const Args& a, int b, int cost, bool report) {
  Span s;
  int len = __ldg(a.lens + b);
  const int most = a.table_width * a.page_size;
  if (len < 0 || len > most) {
    if (report) set_status(a.dev_status, W4_ERR_INVALID_ARG);
    len = len < 0 ? 0 : most;
  }
  s.len = len;
  s.first = a.window > 0 && len > a.window ? len - a.window : 0;
  s.u0 = s.first / kUnit;
  s.n = len > 0 ? (len + kUnit - 1) / kUnit - s.u0 : 0;
  s.line = s.n ? s.n + cost : 0;
  return s;
}

constexpr int kMostBlocks = 4;        // of one SM, in kShapes
inline int64_t recs_bytes(int sms) { return (static_cast<int64_t>(sms) * kMostBlocks * sizeof(Rec) + 15) / 16 * 16; }

// 16-token tiles a stage, stages of a warp's ring and blocks per SM, by [whole][kind][head_dim / 64 - 1]: for
// long streams, and for items that a block takes whole (short ones: more blocks hide the way to their first
// bytes, and deep rings would not fill).  Swept: of int8, 128, 64 sequences to 8192 tokens, {1, 3, 3} takes 74 us,
// {1, 2, 4} 84, {2, 2, 2} 128 (four blocks of three stages do not fit an SM's shared memory); of int4, 128, 8 sequences
// of 32768, {2, 3, 3} takes 83 us, {1, 5, 3} 90, {2, 4, 2} 92; of int4, 256, 48 windows of 16384, {1, 3, 3}, {1, 2, 3} and
// {1, 4, 2} 57 to 58, {2, 2, 2} 61; bf16 wants the deepest rings that fit.
struct Shape {
  int tiles, stages, blocks;
};
constexpr Shape kShapes[2][3][4] = {{{{1, 3, 3}, {1, 5, 1}, {1, 4, 1}, {1, 3, 1}},
                                     {{2, 3, 3}, {1, 3, 3}, {1, 3, 2}, {1, 3, 2}},
                                     {{2, 3, 4}, {2, 3, 3}, {1, 3, 4}, {1, 3, 3}}},
                                    {{{1, 2, 4}, {1, 2, 3}, {1, 2, 2}, {1, 3, 1}},
                                     {{2, 2, 4}, {1, 2, 3}, {1, 2, 3}, {1, 2, 2}},
                                     {{2, 2, 4}, {2, 2, 3}, {1, 2, 4}, {1, 2, 3}}}};
// Items of 16 heads (more than 8 share a key/value head, head_dim up to 128): keys and values are read from
// shared memory and widened once for both eights (64 heads over 4, int8, 16384 tokens: 49 us against 58; bf16 56 against 93).
constexpr Shape kShapes2[3][2] = {{{1, 4, 2}, {1, 3, 2}}, {{2, 3, 2}, {1, 4, 2}}, {{2, 4, 2}, {2, 3, 2}}};

// total * c / grid for c <= grid <= kMostGrid
constexpr int kMostGrid = 1024;
__device__ __forceinline__ int64_t share(int64_t total, int c, int grid) {
  if (total < (1 << 21)) return static_cast<uint32_t>(total) * static_cast<uint32_t>(c) / static_cast<uint32_t>(grid);
  return total * c / grid;
}

template <int KIND, int D, int HT, bool WHOLE>
struct Cfg {
  static constexpr int KW = KIND == W4_KV_BF16 ? 4 : KIND == W4_KV_INT8 ? 2 : 1;   // words per 8 elements
  static constexpr int ROWW = D / 8 * KW;                                           // words per row
  static constexpr int NG = D / 32;                                                 // groups per row
  static constexpr int VE = KIND == W4_KV_BF16 ? 8
                            : KIND == W4_KV_INT8 ? (D % 128 == 0 ? 16 : 8)
                            : (D % 256 == 0 ? 32 : D % 128 == 0 ? 16 : 8);
  static constexpr int VW = VE / 8 * KW;
  static constexpr int NV = D / (8 * VE);
  static constexpr int CPR = ROWW / 4;                                              // 16-byte chunks per row
  static constexpr int LC = CPR & -CPR;                                             // lanes that copy a row together
  // pitches in chunks: a key read of 8 rows and a value read of 4 cover all banks once
  static constexpr int PK = KIND == W4_KV_BF16 ? CPR + 4 : KIND == W4_KV_INT8 ? CPR + 2 : CPR + 1;
  static constexpr int PV = CPR + 1;
  static constexpr int kTileBytes = 16 * 16 * (PK + PV) + (KIND == W4_KV_BF16 ? 0 : 16 * 4 * NG);
  static constexpr Shape kShape = HT == 2 ? kShapes2[KIND][D / 64 - 1] : kShapes[WHOLE][KIND][D / 64 - 1];
  static constexpr int kHeads = 8 * HT;                                             // query heads an item
  static constexpr int TT = kShape.tiles, S = kShape.stages, MINB = kShape.blocks;
  static_assert(MINB * HT <= kMostBlocks, "the workspace has room for kMostBlocks an SM (of 8 heads)");
  static constexpr int kStage = TT * kTileBytes;
  static constexpr int kJoin = kWarps * kHeads * (D + 4) * 4;
  static constexpr int kSmem = kWarps * S * kStage > kJoin ? kWarps * S * kStage : kJoin;
  static_assert(MINB * (kSmem + 2048) <= 233472, "MINB blocks, with a KB of their own and one reserved each, fit an SM");
  // What beginning an item costs a block (its query, its first loads, its join), in units of tokens: about the
  // time in which an SM's share of the memory bandwidth brings 150 KB, divided among the SM's blocks.
  static constexpr int kUnitBytes = 2 * kUnit * (4 * ROWW + (KIND == W4_KV_BF16 ? 0 : 2 * NG));
  static constexpr int COST = 150000 / MINB > kUnitBytes ? (150000 / MINB + kUnitBytes / 2) / kUnitBytes : 1;
};

template <int W>
__device__ __forceinline__ void lds_words(uint32_t (&o)[W], uint32_t at) {
  if constexpr (W == 4) {
    const uint4 v = lds128(at);
    o[0] = v.x; o[1] = v.y; o[2] = v.z; o[3] = v.w;
  } else if constexpr (W == 2) {
    const uint2 v = lds64(at);
    o[0] = v.x; o[1] = v.y;
  } else {
    o[0] = lds32(at);
  }
}
// NG bf16 scales of a row as words
template <int NG>
__device__ __forceinline__ void lds_scales(uint32_t (&o)[NG / 2], uint32_t at) {
  if constexpr (NG == 8 || NG == 4) lds_words<NG / 2>(o, at);
  else
#pragma unroll
    for (int i = 0; i < NG / 2; ++i) o[i] = lds32(at + 4 * i);
}
__device__ __forceinline__ uint32_t lds_u16(uint32_t at) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(at));
  return v;
}
template <int N>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src) {
  if constexpr (N == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ uint32_t h2_mul(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t h2_fma(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
// Codes as exact fp16 numbers with a bias.  The bits of a code go into the mantissa of a power of two or
// of a subnormal number; the bias leaves again in float32 (keys: by products of scales and sums of q) or in the
// fused multiply by the scale (values), where it must be exact in fp16 after that multiplication.
//
// Keys, int8: bytes offset by 128, the subnormal u 2^-24 with u = code + 128.  (On 1024 instead, a group's
// product would reach 2^31, and scales from 2^98 on would take it out of float32's range.)
template <int SEL>
__device__ __forceinline__ uint32_t key_bytes(uint32_t v) { return __byte_perm(v, 0u, SEL); }
// int4: a nibble at bits 0..3 of a half is the subnormal u 2^-24, at bits 4..7 u 2^-20, with u = code + 8:
// one AND each, and a single shift by 8 for the other two nibbles of the half.
__device__ __forceinline__ uint32_t nib0(uint32_t v) { return v & 0x000F000Fu; }
__device__ __forceinline__ uint32_t nib1(uint32_t v) { return v & 0x00F000F0u; }
// what a key product's bias is, per unit of the queries' sum
template <int KIND>
constexpr float kKeyBias = (KIND == W4_KV_INT8 ? 128.f : 8.f) / 16777216.f;
// Values, int8: bytes sign-extended to 16 bits, (b & 0x3FF) ^ 0x6600 = 1536 + code; 1536 = 3 * 512, so
// 1536 * scale has 10 significant bits at most and fma(x, s, -1536 s) is code * s rounded once.
template <int SEL>
__device__ __forceinline__ uint32_t value_bytes(uint32_t a, uint32_t b, uint32_t s, uint32_t bias) {
  uint32_t e, r;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(e) : "r"(a), "r"(b), "n"(SEL));   // (selector bit 3: the byte's sign)
  asm("lop3.b32 %0, %1, %2, %3, 0x6A;" : "=r"(r) : "r"(e), "r"(0x03FF03FFu), "r"(0x66006600u));
  return h2_fma(r, s, bias);
}
// int4: nibbles at bits 4..7 of their halves, fma(u 2^-20, 2^20 s, -8 s) (with half of them at bits 0..3 for fewer
// shifts, 56.9 us instead of 58.4 over 48 windows of 16384 tokens, values would be 32 times nearer to fp16's end).
// Value scales in fp16: the largest of an output row is brought to [2^kScaleTop, 2 * 2^kScaleTop), where
// 1536 times it (int8) and 2^20 times it (int4) are below fp16's largest number.  Scales or values that are
// subnormal there lose bits: a value is off by 2^-21 (int8) or 2^-20 (int4) of that largest scale at most.
template <int KIND>
constexpr int kScaleTop = KIND == W4_KV_INT8 ? 4 : -5;
__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ uint32_t pack_b2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(v));
  return d;
}
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// tanh(y ln 2 / 2) = 1 - 2 / (2^y + 1), off by 2^-21 of 1 at most
__device__ __forceinline__ float tanh_fast(float y) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(exp2_fast(y) + 1.f));
  return fmaf(-2.f, r, 1.f);
}
// Up to this cap the whole of tanh_fast's error is 2^-15 of a score at most.  A larger cap would make it as much
// larger while the scores may be as small as ever: those calls have kernels of their own (WIDE), which
// need not be fast.  (The choice inside the loop cost every call: one short sequence 6.2 us, not 5.6, or 16
// capped bf16 sequences of 8192 tokens 93 us, not 90.)
constexpr float kFastCap = 64.f;
// cap tanh(s / cap) within a few float32 roundings of itself; in = 2 / softcap for s and cap in log2 units.  Below half
// the cap by tanh's Taylor series (its terms fall by 0.1 there, the first left out is 2^-23 of the sum), as a factor
// of s, so that scores far below the cap keep all their bits.
__device__ __forceinline__ float cap_exactly(float s, float cap, float in) {
  const float y = s * in, x = y * 0.34657359028f, x2 = x * x;
  float p = fmaf(x2, 21844.f / 6081075.f, -1382.f / 155925.f);
  p = fmaf(p, x2, 62.f / 2835.f);
  p = fmaf(p, x2, -17.f / 315.f);
  p = fmaf(p, x2, 2.f / 15.f);
  p = fmaf(p, x2, -1.f / 3.f);
  return fabsf(x) < 0.5f ? fmaf(s * x2, p, s) : cap * tanh_fast(y);
}

// Float32 pairs, both elements in one instruction: (a, b) *= (c, d), += (c, d), += (c, d) f.  (Scores, weights and
// totals in pairs: 48 int4 windows of 16384 tokens 57.8 us, singly 58.7.)
__device__ __forceinline__ uint64_t pair_of(float a, float b) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b));
  return v;
}
__device__ __forceinline__ void unpair(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ void mul_pair(float& a, float& b, float c, float d) {
  uint64_t v = pair_of(a, b);
  asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(v) : "l"(pair_of(c, d)));
  unpair(v, a, b);
}
__device__ __forceinline__ void add_pair(float& a, float& b, float c, float d) {
  uint64_t v = pair_of(a, b);
  asm("add.rn.f32x2 %0, %0, %1;" : "+l"(v) : "l"(pair_of(c, d)));
  unpair(v, a, b);
}
__device__ __forceinline__ void fma_pair(float& a, float& b, float c, float d, float f) {
  uint64_t v = pair_of(a, b);
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(v) : "l"(pair_of(c, d)), "l"(pair_of(f, f)));
  unpair(v, a, b);
}

// D += A(16x8 bf16) * B(8x8 bf16)
__device__ __forceinline__ void mma_k8(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t b) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5}, {%6}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(b));
}

template <bool BF16>
__device__ __forceinline__ void mma_acc(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  if constexpr (BF16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// What sums of weighted values are multiplied by, l being the sum of the weights: at least 1, or 0 for no token.
// Every partial output (a warp's, a block's) is divided by its own weights' sum, so that no step leaves the range
// of the values themselves: sums of weights reach 2^14 times the tokens.
__device__ __forceinline__ float inverse_of(float l) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(l));
  return l == 0.f ? 0.f : y;
}
// the logarithm of a sum of weights taken relative to m, less the lift (NaN of a NaN sum: -infinity says no token)
__device__ __forceinline__ float log_sum(float m, float l, float lift) {
  return l == 0.f ? -INFINITY : (m - lift + log2f(l)) * 0.6931471805599453f;
}

template <int KIND, int D, int HT, bool U16, bool WHOLE, bool WIDE>
struct Worker {
  using C = Cfg<KIND, D, HT, WHOLE>;
  static constexpr bool kBf = KIND == W4_KV_BF16;
  static constexpr int kUnitTop = KIND == W4_KV_INT4 ? kScaleTop<KIND> + 20 : kScaleTop<KIND>;   // of the factor's scale
  static constexpr int TT = C::TT, NG = C::NG, NV = C::NV, VW = C::VW, VE = C::VE, KW = C::KW;
  static constexpr int kTileStep = 16 * kWarps;   // a warp's tiles alternate with the other warps'

  const Args& a;
  int lane, r, t;
  int b, hk;
  int lo, hi;                                     // visible tokens of this segment
  uint32_t ring;                                  // this warp's stages in shared memory
  uint32_t* marks;                                // per stage: bit 16 x + i, token i of tile x counts
  uint32_t qf[HT][D / 16][2];
  // Quantised: minus the keys' bias times the sum of q over groups 2t and 2t + 1, for head r, as three bf16 pairs
  // (their sum has 24 bits).  With a token's scales for the other operand, one more product a part gives what
  // the biases put into its score.
  uint32_t qb[HT][3];
  float zmul[HT][2];                              // score -> log2 units, heads 2t and 2t + 1
  float acc[HT][D / 16][4];
  float m[HT][2], l[HT][2];
  int vexp;                                       // quantised: exponent of this output row's unit

  __device__ __forceinline__ explicit Worker(const Args& args) : a(args) {
    lane = threadIdx.x & 31;
    r = lane >> 2;
    t = lane & 3;
  }

  __device__ __forceinline__ void load_q(int head0, int heads) {
#pragma unroll
    for (int e = 0; e < HT; ++e) load_q8(e, head0 + 8 * e, heads - 8 * e);
  }

  __device__ __forceinline__ void load_q8(int e, int head0, int heads) {
    const uint16_t* row = a.q + static_cast<int64_t>(b) * a.q_stride + static_cast<int64_t>(head0 + r) * D;
    uint32_t w[NG][4];
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      uint4 v = make_uint4(0, 0, 0, 0);
      if (r < heads) v = __ldg(reinterpret_cast<const uint4*>(row + 32 * g + 8 * t));
      w[g][0] = v.x; w[g][1] = v.y; w[g][2] = v.z; w[g][3] = v.w;
    }
    const float base = a.scale * 1.4426950408889634f;
    if constexpr (kBf) {
#pragma unroll
      for (int g = 0; g < NG; ++g) {
#pragma unroll
        for (int s = 0; s < 2; ++s) { qf[e][2 * g + s][0] = w[g][2 * s]; qf[e][2 * g + s][1] = w[g][2 * s + 1]; }
      }
      zmul[e][0] = zmul[e][1] = base;
    } else {
      // to fp16 with a power of two per head that brings the largest element to [2^14, 2^15)
      uint32_t mx = 0;
#pragma unroll
      for (int g = 0; g < NG; ++g)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t x = w[g][j] & 0x7FFFu, y = (w[g][j] >> 16) & 0x7FFFu;
          if (x < 0x7F80u) mx = max(mx, x);
          if (y < 0x7F80u) mx = max(mx, y);
        }
      mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const int f = mx ? min(14 + 127 - static_cast<int>(max(mx >> 7, 1u)), 126) : 0;   // -113 at least
      const float up = pow2f(f);
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        if constexpr (KIND == W4_KV_INT8) {
#pragma unroll
          for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int i = 0; i < 2; ++i)
              qf[e][2 * g + s][i] = pack_h2(bf16_lo_to_f32(w[g][2 * s + i]) * up, bf16_hi_to_f32(w[g][2 * s + i]) * up);
        } else {
          // pairs (0, 4), (1, 5), (2, 6), (3, 7), the nibbles' order; those read at bits 4..7 divided by 16
          uint32_t o[4];
          f16_pairs_l1(w[g], up, up * 0.0625f, o);
          qf[e][2 * g][0] = o[0]; qf[e][2 * g][1] = o[1]; qf[e][2 * g + 1][0] = o[2]; qf[e][2 * g + 1][1] = o[3];
        }
      }
      float bias[2] = {0.f, 0.f};
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&qf[e][2 * g + i / 2][i & 1]));
          sum += (KIND == W4_KV_INT4 && (i & 1) ? 16.f : 1.f) * (v.x + v.y);
        }
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        if (g / 2 == t) bias[g & 1] = -kKeyBias<KIND> * sum;
      }
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        qb[e][i] = pack_b2(bias[0], bias[1]);
        bias[0] -= bf16_lo_to_f32(qb[e][i]);
        bias[1] -= bf16_hi_to_f32(qb[e][i]);
      }
      const float down = base * pow2f(-f) * 16777216.f;      // (the keys' 2^-24 is taken back too)
      zmul[e][0] = __shfl_sync(0xffffffffu, down, 8 * t);
      zmul[e][1] = __shfl_sync(0xffffffffu, down, 8 * t + 4);
    }
  }

  __device__ __forceinline__ int page_entry(int tok) const {
    return __ldg(a.table + static_cast<int64_t>(b) * a.table_width + page_of(a, tok));
  }
  __device__ __forceinline__ bool page_ok(int page) const {
    if (static_cast<unsigned>(page) < static_cast<unsigned>(a.pages)) return true;
    set_status(a.dev_status, W4_ERR_INVALID_ARG);
    return false;
  }
  // cache row (all heads of all pages counted) of tok on its page
  __device__ __forceinline__ uint32_t row_on(int page, int tok) const {
    return (static_cast<uint32_t>(page) * a.kv_heads + hk) * a.page_size + (tok - page_of(a, tok) * a.page_size);
  }
  // The page entries of the TT tiles from tok on, loaded a step before they are needed.  Page sizes
  // that are no multiple of 16 need one per token: lane l takes token l % 16 of tile l / 16.
  struct Pages {
    int e[U16 ? TT : 1];
  };
  __device__ __forceinline__ int lane_tok(int tok) const { return tok + (lane >> 4) * kTileStep + (lane & 15); }
  __device__ __forceinline__ int inside(int tok) const { return min(max(tok, lo), hi - 1); }
  __device__ __forceinline__ void look_up(Pages& p, int tok) const {
    if constexpr (U16) {
#pragma unroll
      for (int x = 0; x < TT; ++x) p.e[x] = page_entry(inside(tok + x * kTileStep));
    } else {
      p.e[0] = page_entry(inside(lane_tok(tok)));
    }
  }

  // copies the TT tiles from tok on into stage st
  __device__ __forceinline__ void fetch(const Pages& p, int tok, int st) {
    const uint32_t base = ring + st * C::kStage;
    const auto* kc = static_cast<const uint8_t*>(a.k);
    const auto* vc = static_cast<const uint8_t*>(a.v);
    constexpr int kRowB = 4 * C::ROWW, LC = C::LC, RPI = 32 / LC;
    const int lrow = lane / LC, lcol = lane % LC;
    bool whole = U16 && tok >= lo && tok + (TT - 1) * kTileStep + 16 <= hi;
    if constexpr (U16) {
#pragma unroll
      for (int x = 0; x < TT; ++x) whole = whole && static_cast<unsigned>(p.e[x]) < static_cast<unsigned>(a.pages);
    }
    if (whole) {                                    // 16 rows that follow one another
      if (lane == 0) marks[st] = ~0u;
#pragma unroll
      for (int x = 0; x < TT; ++x) {
        const uint32_t row0 = row_on(p.e[U16 ? x : 0], tok + x * kTileStep);
        const uint32_t ks = base + x * C::kTileBytes, vs = ks + 256 * C::PK, ss = vs + 256 * C::PV;
        const uint64_t off = static_cast<uint64_t>(row0 + lrow) * kRowB + lcol * 16;
#pragma unroll
        for (int y = 0; y < 16 / RPI; ++y)
#pragma unroll
          for (int c = 0; c < C::CPR / LC; ++c) {
            copy_async<16>(ks + ((y * RPI + lrow) * C::PK + c * LC + lcol) * 16, kc + off + y * RPI * kRowB + c * LC * 16);
            copy_async<16>(vs + ((y * RPI + lrow) * C::PV + c * LC + lcol) * 16, vc + off + y * RPI * kRowB + c * LC * 16);
          }
        if constexpr (!kBf) {
          if (lane < 4 * NG) {
            const uint16_t* sc = lane < 2 * NG ? a.ks : a.vs;
            const int c = lane < 2 * NG ? lane : lane - 2 * NG;
            copy_async<16>(ss + lane * 16, sc + static_cast<uint64_t>(row0) * NG + c * 8);
          }
        }
      }
      return;
    }
    // token by token: lane l knows the row of token l % 16 of tile l / 16 (row 0, to be left out, for none)
    static_assert(TT <= 2, "a warp's lanes and a mark's bits hold two tiles");
    const int want = lane_tok(tok), at = inside(want);
    int page;
    if constexpr (U16) page = page_entry(at);
    else page = p.e[0];
    bool ok = want >= lo && want < hi;
    if (ok) ok = page_ok(page);
    const uint32_t row = ok ? row_on(page, at) : 0u;
    const uint32_t mark = __ballot_sync(0xffffffffu, ok);
    if (lane == 0) marks[st] = mark;
#pragma unroll
    for (int x = 0; x < TT; ++x) {
      const uint32_t ks = base + x * C::kTileBytes, vs = ks + 256 * C::PK, ss = vs + 256 * C::PV;
#pragma unroll
      for (int y = 0; y < 16 / RPI; ++y) {
        const uint32_t rr = __shfl_sync(0xffffffffu, row, x * 16 + y * RPI + lrow);
        const uint64_t off = static_cast<uint64_t>(rr) * kRowB + lcol * 16;
#pragma unroll
        for (int c = 0; c < C::CPR / LC; ++c) {
          copy_async<16>(ks + ((y * RPI + lrow) * C::PK + c * LC + lcol) * 16, kc + off + c * LC * 16);
          copy_async<16>(vs + ((y * RPI + lrow) * C::PV + c * LC + lcol) * 16, vc + off + c * LC * 16);
        }
      }
      if constexpr (!kBf) {
#pragma unroll
        for (int y = 0; y < NG / 2; ++y) {                // 4-byte words: 8 NG of the keys', then the values'
          const int w = 32 * y + lane, v = w >= 8 * NG, i = w - v * 8 * NG, tk = i / (NG / 2), col = i - tk * (NG / 2);
          const uint32_t rr = __shfl_sync(0xffffffffu, row, x * 16 + tk);
          copy_async<4>(ss + w * 4, (v ? a.vs : a.ks) + static_cast<uint64_t>(rr) * NG + 2 * col);
        }
      }
    }
  }

  __device__ __forceinline__ void scores(uint32_t base, float (&s)[HT][TT][4]) const {
#pragma unroll
    for (int x = 0; x < TT; ++x) {
      const uint32_t ks = base + x * C::kTileBytes + r * (C::PK * 16) + t * (4 * KW);
      const uint32_t ss = base + x * C::kTileBytes + 256 * (C::PK + C::PV) + r * (2 * NG);
      uint32_t ksc[2][kBf ? 1 : NG / 2];
#pragma unroll
      for (int e = 0; e < HT; ++e)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[e][x][i] = 0.f;
      if constexpr (!kBf) {
        lds_scales<NG>(ksc[0], ss);
        lds_scales<NG>(ksc[1], ss + 16 * NG);
        const uint32_t pair = 4 * min(t, NG / 2 - 1);      // (beyond the groups the other operand is 0)
        const uint32_t a0 = lds32(ss + pair), a1 = lds32(ss + 16 * NG + pair);
#pragma unroll
        for (int e = 0; e < HT; ++e)
#pragma unroll
          for (int i = 0; i < 3; ++i) mma_k8(s[e][x], a0, a1, qb[e][i]);
      }
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        uint32_t k0[KW], k1[KW];
        lds_words<KW>(k0, ks + 16 * g * KW);
        lds_words<KW>(k1, ks + 8 * 16 * C::PK + 16 * g * KW);
        uint32_t f[2][4];                                // the operands of the group's two products
        if constexpr (kBf) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            f[h][0] = k0[2 * h]; f[h][1] = k1[2 * h]; f[h][2] = k0[2 * h + 1]; f[h][3] = k1[2 * h + 1];
          }
        } else if constexpr (KIND == W4_KV_INT8) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t x0 = k0[h] ^ 0x80808080u, x1 = k1[h] ^ 0x80808080u;
            f[h][0] = key_bytes<0x4140>(x0); f[h][1] = key_bytes<0x4140>(x1);
            f[h][2] = key_bytes<0x4342>(x0); f[h][3] = key_bytes<0x4342>(x1);
          }
        } else {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t x0 = h ? k0[0] >> 8 : k0[0], x1 = h ? k1[0] >> 8 : k1[0];
            f[h][0] = nib0(x0); f[h][1] = nib0(x1); f[h][2] = nib1(x0); f[h][3] = nib1(x1);
          }
        }
#pragma unroll
        for (int e = 0; e < HT; ++e) {
          if constexpr (kBf) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
              mma_acc<true>(s[e][x], f[h][0], f[h][1], f[h][2], f[h][3], qf[e][2 * g + h][0], qf[e][2 * g + h][1]);
          } else {
            float c[4];
            mma_f16_16816(c, f[0], qf[e][2 * g][0], qf[e][2 * g][1], {0.f, 0.f, 0.f, 0.f});
            mma_acc<false>(c, f[1][0], f[1][1], f[1][2], f[1][3], qf[e][2 * g + 1][0], qf[e][2 * g + 1][1]);
            const uint32_t w0 = ksc[0][g / 2], w1 = ksc[1][g / 2];
            const float s0 = g & 1 ? bf16_hi_to_f32(w0) : bf16_lo_to_f32(w0);
            const float s1 = g & 1 ? bf16_hi_to_f32(w1) : bf16_lo_to_f32(w1);
            fma_pair(s[e][x][0], s[e][x][1], c[0], c[1], s0);
            fma_pair(s[e][x][2], s[e][x][3], c[2], c[3], s1);
          }
        }
      }
    }
  }

  // scores -> weights: masks, the running reference, p in place of s
  __device__ __forceinline__ void weights(uint32_t mask, int e, float (&s)[TT][4]) {
    float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int x = 0; x < TT; ++x)
#pragma unroll
      for (int i = 0; i < 4; i += 2) mul_pair(s[x][i], s[x][i + 1], zmul[e][0], zmul[e][1]);
    // cap(z) = softcap tanh(z / softcap), in log2 units on both sides
    if constexpr (WIDE) {
      const float cap = fminf(a.softcap * 1.4426950408889634f, 3.4028234e38f), in = 2.f / a.softcap;
#pragma unroll
      for (int x = 0; x < TT; ++x)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[x][i] = cap_exactly(s[x][i], cap, in);
    } else if (a.softcap > 0.f) {
      const float cap = a.softcap * 1.4426950408889634f, in = 2.f / a.softcap;
#pragma unroll
      for (int x = 0; x < TT; ++x)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[x][i] = cap * tanh_fast(s[x][i] * in);
    }
    if (mask != ~0u) {
#pragma unroll
      for (int x = 0; x < TT; ++x)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (!(mask >> (16 * x + r + 8 * (i / 2)) & 1u)) s[x][i] = -INFINITY;
    }
#pragma unroll
    for (int x = 0; x < TT; ++x)
#pragma unroll
      for (int i = 0; i < 4; ++i) mx[i & 1] = fmaxf(mx[i & 1], s[x][i]);
    if (__any_sync(0xffffffffu, mx[0] > m[e][0] + kSlack || mx[1] > m[e][1] + kSlack)) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) mx[c] = fmaxf(mx[c], __shfl_xor_sync(0xffffffffu, mx[c], o));
        const float mn = fmaxf(m[e][c], mx[c]);
        const float f = exp2_fast(m[e][c] - mn);
        m[e][c] = mn;
        l[e][c] *= f;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) { acc[e][i][c] *= f; acc[e][i][2 + c] *= f; }
      }
    }
    const float less[2] = {kBf ? -m[e][0] : kLift - m[e][0], kBf ? -m[e][1] : kLift - m[e][1]};
#pragma unroll
    for (int x = 0; x < TT; ++x)
#pragma unroll
      for (int i = 0; i < 4; i += 2) add_pair(s[x][i], s[x][i + 1], less[0], less[1]);
#pragma unroll
    for (int x = 0; x < TT; ++x)
#pragma unroll
      for (int i = 0; i < 4; ++i) s[x][i] = exp2_fast(s[x][i]);
#pragma unroll
    for (int x = 0; x < TT; ++x)
#pragma unroll
      for (int i = 0; i < 4; i += 2) add_pair(l[e][0], l[e][1], s[x][i], s[x][i + 1]);
  }

  // The tokens 2t, 2t + 1, 2t + 8, 2t + 9 of tile x in the j-th chunk of columns; zeros where one does not count.
  __device__ __forceinline__ void values(uint32_t base, uint32_t mask, int x, int j, uint32_t (&v)[4][VW]) const {
    const uint32_t at = base + x * C::kTileBytes + 256 * C::PK + t * (2 * C::PV * 16) + (8 * j + r) * (4 * VW);
#pragma unroll
    for (int i = 0; i < 4; ++i) lds_words<VW>(v[i], at + ((i & 1) + 8 * (i >> 1)) * (C::PV * 16));
    if (mask != ~0u) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (!(mask >> (16 * x + 2 * t + (i & 1) + 8 * (i >> 1)) & 1u)) {
#pragma unroll
          for (int w = 0; w < VW; ++w) v[i][w] = 0;
        }
    }
  }

  __device__ __forceinline__ void outputs(uint32_t base, uint32_t mask, const float (&s)[HT][TT][4]) {
    if constexpr (kBf) {
#pragma unroll
      for (int x = 0; x < TT; ++x) {
        uint32_t hi_[HT][2], lo_[HT][2];
#pragma unroll
        for (int e = 0; e < HT; ++e)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float *p = &s[e][x][2 * h];
            const uint32_t w = pack_b2(p[0], p[1]);
            lo_[e][h] = transpose8(pack_b2(p[0] - bf16_lo_to_f32(w), p[1] - bf16_hi_to_f32(w)));
            hi_[e][h] = transpose8(w);
          }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          uint32_t v[4][VW];
          values(base, mask, x, j, v);
#pragma unroll
          for (int i = 0; i < VW; ++i) {
            const uint32_t a0 = __byte_perm(v[0][i], v[1][i], 0x5410), a1 = __byte_perm(v[0][i], v[1][i], 0x7632);
            const uint32_t a2 = __byte_perm(v[2][i], v[3][i], 0x5410), a3 = __byte_perm(v[2][i], v[3][i], 0x7632);
#pragma unroll
            for (int e = 0; e < HT; ++e) {
              mma_acc<true>(acc[e][j * VE / 2 + i], a0, a1, a2, a3, hi_[e][0], hi_[e][1]);
              mma_acc<true>(acc[e][j * VE / 2 + i], a0, a1, a2, a3, lo_[e][0], lo_[e][1]);
            }
          }
        }
      }
    } else {
      uint32_t vsc[TT][NV][2];                           // bf16 pairs: tokens (2t, 2t+1), (2t+8, 2t+9)
#pragma unroll
      for (int x = 0; x < TT; ++x)
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          const uint32_t at = base + x * C::kTileBytes + 256 * (C::PK + C::PV) + 32 * NG + t * (4 * NG) + (j * 8 + r) * VE / 32 * 2;
          uint32_t sc[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            sc[i] = lds_u16(at + ((i & 1) + 8 * (i >> 1)) * (2 * NG));
            if (mask != ~0u && !(mask >> (16 * x + 2 * t + (i & 1) + 8 * (i >> 1)) & 1u)) sc[i] = 0;
          }
          vsc[x][j][0] = sc[0] | (sc[1] << 16);
          vsc[x][j][1] = sc[2] | (sc[3] << 16);
        }
      // the unit of this output row: the largest finite scale seen so far in it
      uint32_t pair = 0;
#pragma unroll
      for (int x = 0; x < TT; ++x)
#pragma unroll
        for (int j = 0; j < NV; ++j) pair = __vmaxu2(pair, __vmaxu2(vsc[x][j][0], vsc[x][j][1]));
      uint32_t e = max(pair & 0xFFFFu, pair >> 16);
      if (e >= 0x7F80u) {                                // a scale of NaN or infinity: the largest finite one
        e = 0;
#pragma unroll
        for (int x = 0; x < TT; ++x)
#pragma unroll
          for (int j = 0; j < 2 * NV; ++j) {
            const uint32_t w = vsc[x][j / 2][j & 1];
            if ((w & 0xFFFFu) < 0x7F80u) e = max(e, w & 0xFFFFu);
            if ((w >> 16) < 0x7F80u) e = max(e, w >> 16);
          }
      }
      if (__any_sync(0xffffffffu, static_cast<int>(e >> 7) > vexp)) {
        e = max(e, __shfl_xor_sync(0xffffffffu, e, 1));
        e = max(e, __shfl_xor_sync(0xffffffffu, e, 2)) >> 7;
        const int en = max(static_cast<int>(e), vexp);
        const float f = exp2_fast(static_cast<float>(vexp - en));
        vexp = en;
#pragma unroll
        for (int i = 0; i < HT * D / 16; ++i)
#pragma unroll
          for (int c = 0; c < 4; ++c) acc[i / (D / 16)][i % (D / 16)][c] *= f;
      }
      const float unit = pow2f(kUnitTop + 127 - vexp);
#pragma unroll
      for (int x = 0; x < TT; ++x) {
        uint32_t p[HT][2];
#pragma unroll
        for (int q = 0; q < HT; ++q) {
          p[q][0] = transpose8(pack_h2(s[q][x][0], s[q][x][1]));
          p[q][1] = transpose8(pack_h2(s[q][x][2], s[q][x][3]));
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          uint32_t sv[2], bias[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            sv[h] = pack_h2(bf16_lo_to_f32(vsc[x][j][h]) * unit, bf16_hi_to_f32(vsc[x][j][h]) * unit);
            // int8: -1536 s.  int4: sv is 2^20 s, the factor of bits 4..7; -8 s = -2^-17 sv
            bias[h] = h2_mul(sv[h], KIND == W4_KV_INT8 ? 0xE600E600u : 0x80808080u);
          }
          uint32_t v[4][VW];
          values(base, mask, x, j, v);
#pragma unroll
          for (int i = 0; i < VW; ++i) {
            if constexpr (KIND == W4_KV_INT8) {
              uint32_t el[2][4];                         // [token pair][element of the word]
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const uint32_t wa = v[2 * h][i], wb = v[2 * h + 1][i];
                el[h][0] = value_bytes<0xC480>(wa, wb, sv[h], bias[h]);
                el[h][1] = value_bytes<0xD591>(wa, wb, sv[h], bias[h]);
                el[h][2] = value_bytes<0xE6A2>(wa, wb, sv[h], bias[h]);
                el[h][3] = value_bytes<0xF7B3>(wa, wb, sv[h], bias[h]);
              }
#pragma unroll
              for (int q = 0; q < HT; ++q) mma_acc<false>(acc[q][j * VE / 2 + 2 * i], el[0][0], el[0][1], el[1][0], el[1][1], p[q][0], p[q][1]);
#pragma unroll
              for (int q = 0; q < HT; ++q) mma_acc<false>(acc[q][j * VE / 2 + 2 * i + 1], el[0][2], el[0][3], el[1][2], el[1][3], p[q][0], p[q][1]);
            } else {
#pragma unroll
              for (int half = 0; half < 2; ++half) {     // elements 0..3, 4..7 of the word
                uint32_t el[2][4];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  const uint32_t u = __byte_perm(v[2 * h][i], v[2 * h + 1][i], half ? 0x7632 : 0x5410);
                  el[h][0] = h2_fma(nib1(u << 4), sv[h], bias[h]);
                  el[h][1] = h2_fma(nib1(u), sv[h], bias[h]);
                  el[h][2] = h2_fma(nib1(u >> 4), sv[h], bias[h]);
                  el[h][3] = h2_fma(nib1(u >> 8), sv[h], bias[h]);
                }
  #pragma unroll
              for (int q = 0; q < HT; ++q) mma_acc<false>(acc[q][j * VE / 2 + 4 * i + 2 * half], el[0][0], el[0][1], el[1][0], el[1][1], p[q][0], p[q][1]);
  #pragma unroll
              for (int q = 0; q < HT; ++q) mma_acc<false>(acc[q][j * VE / 2 + 4 * i + 2 * half + 1], el[0][2], el[0][3], el[1][2], el[1][3], p[q][0], p[q][1]);
              }
            }
          }
        }
      }
    }
  }

  // tiles warp, warp + kWarps, ... from token t0 (a multiple of 16) on, TT of them at once
  __device__ __forceinline__ void walk(int t0, int warp, int head0, int heads) {
#pragma unroll
    for (int e = 0; e < HT; ++e) {
      m[e][0] = m[e][1] = kLowest;
      l[e][0] = l[e][1] = 0.f;
    }
    vexp = kUnitTop + 1;                             // (2^(kUnitTop + 127 - vexp) stays a float)
#pragma unroll
    for (int i = 0; i < HT * D / 16; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[i / (D / 16)][i % (D / 16)][c] = 0.f;
    int tok = t0 + warp * 16;
    if (tok >= hi) return;
    constexpr int kStep = TT * kTileStep;
    Pages p, first[C::S - 1];
#pragma unroll
    for (int st = 0; st < C::S - 1; ++st) look_up(first[st], tok + st * kStep);
    int ahead = tok;                                   // where the next stage begins
#pragma unroll
    for (int st = 0; st < C::S - 1; ++st) {
      if (ahead < hi) fetch(first[st], ahead, st);
      copy_commit();
      ahead += kStep;
    }
    look_up(p, ahead);
    load_q(head0, heads);                              // while the first stages are on their way
    int st = 0, into = C::S - 1;                       // the stage at hand, and the one consumed last
    while (true) {
      copy_wait<C::S - 2>();
      __syncwarp();
      if (ahead < hi) {
        fetch(p, ahead, into);
        look_up(p, ahead + kStep);
      }
      copy_commit();
      const uint32_t base = ring + st * C::kStage, mask = marks[st];
      float s[HT][TT][4];
      scores(base, s);
#pragma unroll
      for (int e = 0; e < HT; ++e) weights(mask, e, s[e]);
      outputs(base, mask, s);
      tok += kStep;
      if (tok >= hi) break;
      ahead += kStep;
      into = st;
      st = st + 1 == C::S ? 0 : st + 1;
    }
    copy_wait<0>();
  }
};

// WHOLE: block x takes item x as it is.  Otherwise the blocks share the line evenly.  WIDE: caps above kFastCap.
template <int KIND, int D, int HT, bool U16, bool WHOLE, bool WIDE>
__global__ void __launch_bounds__(32 * kWarps, Cfg<KIND, D, HT, WHOLE>::MINB) attend_kernel(const Args a) {
  using C = Cfg<KIND, D, HT, WHOLE>;
  constexpr int kHeads = C::kHeads;
  extern __shared__ __align__(16) uint8_t s_ring[];
  auto& s_o = *reinterpret_cast<float(*)[kWarps][kHeads][D + 4]>(s_ring);   // once the stages are done with
  __shared__ uint32_t s_marks[kWarps][C::S];
  __shared__ float s_m[kWarps][kHeads], s_l[kWarps][kHeads];
  __shared__ int s_scan[2];
  __shared__ int64_t s_sum[kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  const int per_seq = a.kv_heads * a.HB;
  int64_t at, end, total = 0;                            // this block's share of the line, the line's length
  int grid = 1;
  int b, item, at_line;                                  // where it begins: sequence, item of it, place within that
  Span sp;
  if constexpr (WHOLE) {
    b = blockIdx.x / per_seq;
    item = blockIdx.x - b * per_seq;
    sp = span_of(a, b, C::COST, item == 0);
    at = at_line = 0;
    end = sp.line;
    if (sp.n == 0) {
      const int head0 = item / a.HB * a.G + item % a.HB * kHeads, heads = min(kHeads, a.G - item % a.HB * kHeads);
      const int64_t row0 = static_cast<int64_t>(b) * a.q_heads + head0;
      uint32_t* row = reinterpret_cast<uint32_t*>(a.out + row0 * D);
      for (int x = threadIdx.x; x < heads * (D / 2); x += 32 * kWarps) row[x] = 0u;
      if (a.lse && threadIdx.x < heads) a.lse[row0 + threadIdx.x] = -INFINITY;
      return;
    }
  } else {
    pdl_trigger();                                       // (the joining blocks wait for this grid's end)
    // Every thread adds up its run of sequences; the one whose run holds
    // the share's first place looks it up in there.
    const int run = (a.B + 32 * kWarps - 1) / (32 * kWarps), b0 = threadIdx.x * run, b1 = min(b0 + run, a.B);
    int64_t mine = 0;
    for (int i = b0; i < b1; ++i) mine += span_of(a, i, C::COST, blockIdx.x == 0).line;
    int64_t upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += v;
    }
    if (lane == 31) s_sum[warp] = upto;
    __syncthreads();
    for (int k = 0; k < kWarps; ++k) {
      if (k < warp) upto += s_sum[k];
      total += s_sum[k];
    }
    total *= per_seq;
    // the rows of sequences without tokens
    for (int i = blockIdx.x; i < a.B; i += gridDim.x) {
      if (__ldg(a.lens + i) > 0) continue;
      uint32_t* row = reinterpret_cast<uint32_t*>(a.out + static_cast<int64_t>(i) * a.q_heads * D);
      for (int x = threadIdx.x; x < a.q_heads * (D / 2); x += 32 * kWarps) row[x] = 0u;
      if (a.lse)
        for (int x = threadIdx.x; x < a.q_heads; x += 32 * kWarps) a.lse[static_cast<int64_t>(i) * a.q_heads + x] = -INFINITY;
    }
    grid = static_cast<int>(total < gridDim.x ? total : gridDim.x);   // blocks with a share, at least a unit each
    if (static_cast<int>(blockIdx.x) >= grid) {
      if (threadIdx.x == 0) a.recs[blockIdx.x].last = -1;
      return;
    }
    at = share(total, blockIdx.x, grid);
    end = share(total, blockIdx.x + 1, grid);
    int64_t from = (upto - mine) * per_seq;
    if (at >= from && at < upto * per_seq) {
      int i = b0;
      for (;; ++i) {
        const int64_t n = static_cast<int64_t>(span_of(a, i, C::COST, false).line) * per_seq;
        if (at < from + n) break;
        from += n;
      }
      s_scan[0] = i;
      s_scan[1] = static_cast<int>(at - from);             // below 2^31: the tokens' limit
    }
    __syncthreads();
    b = s_scan[0];
    const int into = s_scan[1];
    sp = span_of(a, b, C::COST, false);
    item = into / sp.line;
    at_line = into - item * sp.line;
  }
  const Rec start{b, item, at_line};
  const int64_t start_at = at;
  const int start_n = sp.n;

  Worker<KIND, D, HT, U16, WHOLE, WIDE> w(a);
  w.ring = smem_u32(s_ring) + warp * (C::S * C::kStage);
  w.marks = s_marks[warp];
  while (true) {
    const int step = static_cast<int>(end - at < sp.line - at_line ? end - at : sp.line - at_line);
    const int u = max(at_line - C::COST, 0), take = max(at_line + step - C::COST, 0) - u;   // units of it
    const int hk = item / a.HB, hb = item - hk * a.HB;
    const int heads = min(kHeads, a.G - hb * kHeads);
    const int head0 = hk * a.G + hb * kHeads;
    w.b = b;
    w.hk = hk;
    const int t0 = (sp.u0 + u) * kUnit;
    w.lo = max(sp.first, t0);
    w.hi = min(sp.len, t0 + take * kUnit);
    if (take > 0) {
      w.walk(max(t0, w.lo & ~15), warp, head0, heads);

      // join the warps: head h's reference is the largest of theirs, their shares go by their weights
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 2 * HT; ++i) {
        const int e = i >> 1, c = i & 1;
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) w.l[e][c] += __shfl_xor_sync(0xffffffffu, w.l[e][c], o);
        if (w.r == 0) {
          s_m[warp][8 * e + 2 * w.t + c] = w.m[e][c];
          s_l[warp][8 * e + 2 * w.t + c] = w.l[e][c];
        }
      }
      // (2^kMore goes to the other factor: an exponent stays below 127)
      constexpr int kMore = KIND == W4_KV_INT4 ? 8 : 0;
      const float unit = KIND == W4_KV_BF16 ? 1.f : pow2f(w.vexp - 127 - kScaleTop<KIND> - kMore);
#pragma unroll
      for (int e = 0; e < HT; ++e) {
        const float inv0 = inverse_of(w.l[e][0]) * (1 << kMore), inv1 = inverse_of(w.l[e][1]) * (1 << kMore);
#pragma unroll
        for (int j = 0; j < C::NV; ++j)
#pragma unroll
          for (int i = 0; i < C::VE / 2; ++i) {
            const float* o = w.acc[e][j * C::VE / 2 + i];
            const int d = j * 8 * C::VE + w.r * C::VE + 2 * i;
            *reinterpret_cast<float2*>(&s_o[warp][8 * e + 2 * w.t][d]) = make_float2(o[0] * inv0 * unit, o[2] * inv0 * unit);
            *reinterpret_cast<float2*>(&s_o[warp][8 * e + 2 * w.t + 1][d]) = make_float2(o[1] * inv1 * unit, o[3] * inv1 * unit);
          }
      }
      __syncthreads();
      const bool whole = take == sp.n;
      // a block continues an item in its slot 0 and begins one in its slot 1
      float* part = a.parts + static_cast<int64_t>(2 * blockIdx.x + (u > 0 ? 0 : 1)) * kHeads * (D + 2);
      for (int x = threadIdx.x; x < heads * (D / 4); x += 32 * kWarps) {
        const int h = x / (D / 4), d = (x - h * (D / 4)) * 4;
        float mm = kLowest, ll = 0.f, part_l[kWarps];
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k = 0; k < kWarps; ++k) mm = fmaxf(mm, s_m[k][h]);
#pragma unroll
        for (int k = 0; k < kWarps; ++k) {
          part_l[k] = exp2_fast(s_m[k][h] - mm) * s_l[k][h];
          ll += part_l[k];
        }
        const float inv = inverse_of(ll);
#pragma unroll
        for (int k = 0; k < kWarps; ++k) {
          const float f = part_l[k] * inv;
          const float4 v = *reinterpret_cast<const float4*>(&s_o[k][h][d]);
          o.x = fmaf(f, v.x, o.x);
          o.y = fmaf(f, v.y, o.y);
          o.z = fmaf(f, v.z, o.z);
          o.w = fmaf(f, v.w, o.w);
        }
        if (whole) {
          const int64_t row = static_cast<int64_t>(b) * a.q_heads + head0 + h;
          *reinterpret_cast<uint2*>(a.out + row * D + d) = make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
          if (a.lse && d == 0)
            a.lse[row] = log_sum(mm, ll, KIND == W4_KV_BF16 ? 0.f : kLift);
        } else {
          *reinterpret_cast<float4*>(part + h * D + d) = o;
          if (d == 0) { part[kHeads * D + h] = mm; part[kHeads * D + kHeads + h] = ll; }
        }
      }
    }
    at += step;
    if (at >= end) break;
    at_line = 0;
    if (++item == per_seq) {
      item = 0;
      do { sp = span_of(a, ++b, C::COST, false); } while (sp.n == 0);
    }
    __syncthreads();
  }
  if (!WHOLE && threadIdx.x == 0) {
    // What the joining kernel needs of an item that this block continued and the one before began: the last
    // block of it.  (An item begins, for that, at its first unit.)
    Rec rec{start.b, start.item, -1};
    if (start.last > C::COST) {
      const int64_t unit0 = start_at - start.last + C::COST;
      if (unit0 >= share(total, blockIdx.x - 1, grid)) {
        const int64_t x = unit0 + start_n;               // last + 1 = the least c with total * c >= x * grid
        rec.last = static_cast<int>((x * grid - 1) / total);
      }
    }
    a.recs[blockIdx.x] = rec;
  }
}

// Joins the parts of split items, in order.  An item is cut where a block's share ends, so the second of
// its blocks (x) stands for it; y counts its heads.  Up to kMostGrid parts: first all references and totals,
// then the sums with many loads in flight (one after the other, 55 parts took 12 us).
template <int D, int HT>
__global__ void __launch_bounds__(128) join_kernel(const Args a, float lift) {
  __shared__ float s_f[kMostGrid], s_t[kMostGrid], s_o[4][D], s_m[4], s_l[4];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kHeads = 8 * HT, kPart = kHeads * (D + 2), V = D / 32, kBatch = 8;
  pdl_wait();
  const Rec rec = a.recs[blockIdx.x];
  const int hk = rec.item / a.HB, hb = rec.item - hk * a.HB, h = blockIdx.y;
  if (rec.last < 0 || hb * kHeads + h >= a.G) return;
  // the first part lies in slot 1 of its block, the others in slot 0 of theirs
  const int c0 = blockIdx.x - 1, n = rec.last - c0 + 1;
  auto part = [&](int i) { return a.parts + static_cast<int64_t>(2 * (c0 + i) + (i == 0 ? 1 : 0)) * kPart; };
  // the first batch of sums is on its way while the factors are found
  float v[kBatch][V];
  auto load = [&](int i0) {
#pragma unroll
    for (int x = 0; x < kBatch; ++x)
#pragma unroll
      for (int i = 0; i < V; ++i) v[x][i] = i0 + 4 * x < n ? part(i0 + 4 * x)[h * D + lane + 32 * i] : 0.f;
  };
  load(warp);
  float m = kLowest;
  for (int i = threadIdx.x; i < n; i += 128) {
    s_f[i] = part(i)[kHeads * D + h];
    s_t[i] = part(i)[kHeads * D + kHeads + h];
    m = fmaxf(m, s_f[i]);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (lane == 0) s_m[warp] = m;
  __syncthreads();
  m = fmaxf(fmaxf(s_m[0], s_m[1]), fmaxf(s_m[2], s_m[3]));
  float l = 0.f;
  for (int i = threadIdx.x; i < n; i += 128) {
    s_f[i] = exp2_fast(s_f[i] - m) * s_t[i];
    l += s_f[i];
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  if (lane == 0) s_l[warp] = l;
  __syncthreads();
  l = (s_l[0] + s_l[1]) + (s_l[2] + s_l[3]);
  const float inv = inverse_of(l);
  float o[V];
#pragma unroll
  for (int i = 0; i < V; ++i) o[i] = 0.f;
  for (int i0 = warp; i0 < n; i0 += 4 * kBatch) {
    if (i0 != warp) load(i0);
#pragma unroll
    for (int x = 0; x < kBatch; ++x)
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (i0 + 4 * x < n) o[i] = fmaf(v[x][i], s_f[i0 + 4 * x] * inv, o[i]);
  }
#pragma unroll
  for (int i = 0; i < V; ++i) s_o[warp][lane + 32 * i] = o[i];
  __syncthreads();
  const int64_t row = static_cast<int64_t>(rec.b) * a.q_heads + hk * a.G + hb * kHeads + h;
  for (int d = threadIdx.x; d < D; d += 128)
    a.out[row * D + d] = f32_to_bf16_bits((s_o[0][d] + s_o[1][d]) + (s_o[2][d] + s_o[3][d]));
  if (a.lse && threadIdx.x == 0) a.lse[row] = log_sum(m, l, lift);
}

// How the work is cut.  A block per item, with no scan in front and no join behind it:
//   * where no table reaches further than kShort units (64 tokens each; 8 heads of 128, bf16, one sequence: 4.2 us
//     against 4.9 for 128 tokens, even at 384, 9.0 against 7.6 at 512), a launch less in any case;
//   * to kLittle units, where the items fill the SMs (512 items of up to 500 tokens: 20.0 us against 25.8);
//   * to kMiddling units, where there are four items for every block the SMs hold (2048 items of 4000 int8
//     tokens: 376 us against 403).
// Otherwise as many blocks as the SMs hold, or one a unit if there are fewer, share the line.
constexpr int kShort = 6, kLittle = 8, kMiddling = 64;

template <int KIND, int D, int HT, bool WHOLE, bool WIDE>
w4_status launch_mode(const Args& a, int grid, cudaStream_t s) {
  // (a wide cap's kernel takes all page sizes token by token)
  const bool u16 = !WIDE && a.page_size % 16 == 0;
  auto kernel = u16 ? attend_kernel<KIND, D, HT, !WIDE, WHOLE, WIDE> : attend_kernel<KIND, D, HT, false, WHOLE, WIDE>;
  constexpr int kSmem = Cfg<KIND, D, HT, WHOLE>::kSmem;
  static SmemRaised raised[2];
  if (raise_smem(kernel, kSmem, raised[u16]) != cudaSuccess) return W4_ERR_CUDA;
  kernel<<<grid, 32 * kWarps, kSmem, s>>>(a);
  if (cudaGetLastError() != cudaSuccess) return W4_ERR_CUDA;
  if (WHOLE) return W4_OK;
  const float lift = KIND == W4_KV_BF16 ? 0.f : kLift;
  const dim3 joins(grid, a.G < 8 * HT ? a.G : 8 * HT);
  return launch_pdl(join_kernel<D, HT>, joins, dim3(128), 0, s, a, lift) == cudaSuccess ? W4_OK : W4_ERR_CUDA;
}

template <int KIND, int D, int HT>
w4_status launch_heads(Args a, cudaStream_t s, int sms) {
  a.HB = (a.G + 8 * HT - 1) / (8 * HT);
  const int64_t items = static_cast<int64_t>(a.B) * a.kv_heads * a.HB;
  const int64_t units = (static_cast<int64_t>(a.table_width) * a.page_size + kUnit - 1) / kUnit;
  int64_t most = static_cast<int64_t>(sms) * Cfg<KIND, D, HT, false>::MINB;
  const bool wide = a.softcap > kFastCap;
  if (!wide && (units <= kShort || (units <= kLittle && items >= most) || (units <= kMiddling && items >= 4 * most)))
    return launch_mode<KIND, D, HT, true, false>(a, static_cast<int>(items), s);
  most = most < kMostGrid ? most : kMostGrid;
  const int grid = static_cast<int>(items * units < most ? items * units : most);
  return wide ? launch_mode<KIND, D, HT, false, true>(a, grid, s) : launch_mode<KIND, D, HT, false, false>(a, grid, s);
}

template <int KIND, int D>
w4_status launch_dim(const Args& a, cudaStream_t s, int sms) {
  if constexpr (D <= 128)
    if (a.G > 8) return launch_heads<KIND, D, 2>(a, s, sms);
  return launch_heads<KIND, D, 1>(a, s, sms);
}

template <int KIND>
w4_status launch_kind(const Args& a, int D, cudaStream_t s, int sms) {
  switch (D) {
    case 64: return launch_dim<KIND, 64>(a, s, sms);
    case 128: return launch_dim<KIND, 128>(a, s, sms);
    case 192: return launch_dim<KIND, 192>(a, s, sms);
    default: return launch_dim<KIND, 256>(a, s, sms);
  }
}

w4_status launch_bf16(const Args& a, int D, cudaStream_t s, int sms);
w4_status launch_int8(const Args& a, int D, cudaStream_t s, int sms);
w4_status launch_int4(const Args& a, int D, cudaStream_t s, int sms);

}  // namespace at
}  // namespace w4
