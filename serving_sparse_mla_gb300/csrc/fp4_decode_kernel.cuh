// Paged sparse-MLA decode over a 4-bit cache: the attention of
// fwd_kernel.cuh's paged mode,
//
//   s_j = sm_scale * q . x_j,   LSE = ln sum_j exp(s_j),
//   out = sum_j exp(s_j - LSE) * x_j[0:512],
//
// whose rows x_j are dequantized as they are used.  A slot is 416 bytes:
// 256 bytes of e2m1 codes (code 2i in the low half of byte i), 32 e4m3 scales
// (scale k for codes 16 k .. 16 k + 15), 64 bf16 values (the rotated part);
// x = code * scale * kv_scale, then the 64 values.
//
// Up to 16 heads a block of 64 rows needs only ~4 MMAs per gathered 1152-byte
// row's worth of values, and the cost is turning codes into MMA operands.  So
// the raw slots are staged in shared memory and the codes are widened in
// registers, straight into the operand layout of the warp-level MMA
// (m16n8k16): no wide tile is written back to shared memory.  Both products
// take rows as M or K and heads as N, so 8 heads fill the MMA:
//
//   S^T [64 rows x heads]  = X [64 x 576] . Q^T      a lane widens 4 codes each
//                                                    of two rows per MMA
//   O^T [512 x heads]     += X^T [512 x 64] . P^T    a lane widens codes of
//                                                    4 rows at the same column,
//                                                    paired by two logic
//                                                    instructions per 8 codes
//
// e2m1 * e4m3 has at most 6 significant bits and lies in [2^-10, 2688], so
// code * scale is exact in f16.  Q's latent part is brought to f16 by a power of two
// per head, from its own largest value (bf16 has 8 significant bits: values down to
// 2^-17 of that are exact, smaller ones lose bits below 2^-25 of it; the score is off
// by at most 2^-25 max |q| sum |x|).  The latent score takes that power and kv_scale,
// then the rotated part is added, whose Q is as it came.  P is
// f16 with the running maximum's weight at 2^kF4PBits: 11 bits down to 2^-21 of that
// weight, steps of 2^-31 below, so that a list of n rows loses at most n 2^-32 of a
// value's size (2^18 rows: 6e-5, where bf16's rounding of the output is 2e-3); its
// sum is taken from the unrounded weights.  The rotated part stays bf16 (its own
// MMAs).  All sums are fp32.
//
// What bounds it: the order of its phases.  Scores, barrier and values of a block
// follow one another with 8 or 12 warps on an SM, and the schedulers issue in 37 to
// 48 % of the cycles while no pipe is full (16 heads: MMA 37 %, ALU 37 %, shared memory
// 49 % of their peaks).  Per 16 rows a warp issues about 1100 instructions (8 heads), of
// which 256 are conversions, 256 multiplications by the scale and 68 MMAs per 8 heads;
// leaving out the multiplications alone takes 12 % off, the gather of the slots 8 %,
// the conversions 1 %.  Above 32 heads each unit of 32 gathers and widens its token's list
// again.  Lists of 2048, GPU time: 96 tokens x 8 heads 33.5 us (the bf16 cache's decode
// 60), 512 x 16 169 (212), 128 x 64 146 (101: there the bf16 decode wins), one token x 8
// 8.8.
//
// A warp takes 16 rows of a block: it copies their slots (cp.async, its own
// part of the ring), scores them, writes P to shared memory, and after one
// barrier a block takes 512 / W columns of O^T over all of the block's rows.
// Work is dealt in one of two ways.  Few units: a cluster of CTAs takes a unit,
// each an equal part of its list, and merges through distributed shared memory.
// Many: as in the paged forward (block ranges, fwd_kernel.cuh), the units' lists
// laid end to end and cut into one equal range per CTA; a second kernel merges
// the pieces of cut units.  With as many CTAs as units the ranges are whole lists.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>

#include "fwd_kernel.cuh"
#include "norm_rope_kernel.cuh"

namespace smla {

constexpr int kF4TileBytes = 16 * kFp4Slot;   // one warp's 16 rows
constexpr int kF4MaxCluster = 16;
// P = 2^kF4PBits exp(s - maximum), and a score may pass the maximum by 2^8 before that
// moves: below 2^15, inside f16's range.
constexpr int kF4PBits = 7;
constexpr int kF4PartRow = kDv + 8;           // floats of one head's piece in shared memory (the 8 spread the banks)

struct Fp4Params {
  const __nv_bfloat16* q;      // [n_tok, h_q, 576]
  const uint8_t* cache;        // [num_blocks * page_size, 416]
  const int32_t* indices;      // [n_tok, topk]
  const int32_t* block_table;  // [batch, max_blocks]
  const int32_t* seqlens;      // [batch]
  __nv_bfloat16* out;          // [n_tok, h_q, 512]
  float* lse;                  // [n_tok, h_q]
  float* part_o;               // [2 ctas, part_rows, 512]
  float* part_lse;             // [2 ctas, part_rows]
  int n_tok, h_q, topk, s_next, page_size, max_blocks, num_blocks;
  int groups;                  // head groups of a token
  int nb;                      // blocks of a list (Fp4Shape::kRows entries each)
  int ctas, part_rows;
  int cluster;                 // CTAs of a unit's cluster (0: the units' blocks cut into ranges)
  float scale_log2;            // sm_scale * log2(e)
  float kv_scale;
};

// A CTA's shape: 8 NT heads; blocks are 16 rows for each of W
// warps, two blocks in the ring.  kPad spreads P's rows over the banks.
template <int NT_, int W_, int kPerSm_, int kPad_>
struct Fp4Shape {
  static constexpr int NT = NT_, W = W_, kPerSm = kPerSm_;
  static constexpr int kHeads = 8 * NT;
  static constexpr int kThreads = 32 * W;
  static constexpr int kRows = 16 * W;
  static constexpr int kStage = W * kF4TileBytes;
  static constexpr int kPRow = kRows + kPad_;            // f16 values of one head's P
  static constexpr int kQOff = 2 * kStage;
  static constexpr int kPOff = kQOff + 18 * NT * 512;    // Q: 16 latent + 2 rope fragments of 32 lanes x 16 bytes
  static constexpr int kRedOff = kPOff + 2 * kHeads * kPRow * 2;
  static constexpr int kMiscOff = kRedOff + W * kHeads * 4;
  static constexpr int kBytes = kMiscOff + kHeads * 4 + 2 * W * 4;
  // A cluster's pieces: O in the ring's place, its LSEs and the weights in Q's.
  static_assert(kHeads * kF4PartRow * 4 <= 2 * kStage && (1 + kF4MaxCluster) * kHeads * 4 <= 18 * NT * 512, "pieces");
  static_assert(W == 4 || W == 8, "64 / W columns of O^T per lane, in one scale group");
  static_assert((kBytes + 1024) * kPerSm <= 233472, "shared memory of an SM");
};
// 8 and 16 heads: three CTAs of four warps per SM; at 16 P's rows keep an 8-value
// pad (two-way bank conflicts on its few reads), which is what makes three fit.
// 32 heads: one CTA of eight warps, half of the sums per thread (82 us at 128
// lists of 2048 against 93 us for two CTAs of four warps, which spill).
using Fp4Shape8 = Fp4Shape<1, 4, 3, 16>;
using Fp4Shape16 = Fp4Shape<2, 4, 3, 8>;
using Fp4Shape32 = Fp4Shape<4, 8, 1, 16>;
// 8 and 16 heads of few units: eight warps work at a unit's few blocks at once.
using Fp4Shape8Few = Fp4Shape<1, 8, 1, 16>;
using Fp4Shape16Few = Fp4Shape<2, 8, 1, 16>;

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t v) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<unsigned short>(v)));
  return h;
}

// S^T of this warp's 16 rows; f: the heads' 2^e (f4_load_q).  The MMA's row g is row
// rho(g) = g with bits 0 and 1 swapped, so that the two rows a quarter of a
// warp reads together lie 832 bytes apart: their 16-byte reads fall into
// different banks (416-byte rows step by 8 of 32 banks).  Lane (g, c) owns
// codes 128 c .. 128 c + 127 of rows rho(g) and rho(g) + 8, the four 32-code
// chunks taken in an order rotated by c for the same reason; Q's fragments are
// laid out to match (f4_load_q).  Two chains of sums per head tile keep
// dependent MMAs apart.
template <int NT>
__device__ __forceinline__ void f4_scores(const uint8_t* tile, const uint4* qf, float (&acc)[NT][4], int lane,
                                          float kv_scale, const float (&f)[NT][2]) {
  const int g = lane >> 2, c = lane & 3;
  const int rho = (g & 4) | ((g & 1) << 1) | ((g >> 1) & 1);
  const uint8_t* row0 = tile + rho * kFp4Slot;
  const uint8_t* row1 = row0 + 8 * kFp4Slot;
  float alt[NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[n][i] = alt[n][i] = 0.f;
#pragma unroll
  for (int i0 = 0; i0 < 4; ++i0) {
    const int chunk = 4 * c + ((i0 + c) & 3);   // 32 codes: 16 bytes, two scales
    const uint4 w0 = *reinterpret_cast<const uint4*>(row0 + 16 * chunk);
    const uint4 w1 = *reinterpret_cast<const uint4*>(row1 + 16 * chunk);
    const uint32_t s0 = e4m3x2_f16x2(*reinterpret_cast<const unsigned short*>(row0 + kFp4ScaleAt + 2 * chunk));
    const uint32_t s1 = e4m3x2_f16x2(*reinterpret_cast<const unsigned short*>(row1 + kFp4ScaleAt + 2 * chunk));
    const uint32_t a0[4] = {w0.x, w0.y, w0.z, w0.w};
    const uint32_t a1[4] = {w1.x, w1.y, w1.z, w1.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t f0 = __byte_perm(s0, 0, j < 2 ? 0x1010 : 0x3232);
      const uint32_t f1 = __byte_perm(s1, 0, j < 2 ? 0x1010 : 0x3232);
      uint32_t h0[4], h1[4];
      e2m1x8_value(a0[j], h0);
      e2m1x8_value(a1[j], h1);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        h0[i] = mul_f16x2(h0[i], f0);
        h1[i] = mul_f16x2(h1[i], f1);
      }
      const uint32_t fa[4] = {h0[0], h1[0], h0[1], h1[1]};
      const uint32_t fb[4] = {h0[2], h1[2], h0[3], h1[3]};
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const uint4 b = qf[((i0 * 4 + j) * NT + n) * 32 + lane];
        mma_f16(acc[n], fa, b.x, b.y);
        mma_f16(alt[n], fb, b.z, b.w);
      }
    }
  }
  // the rotated part (bf16), after the latent part took kv_scale and 2^e (one after the
  // other: their product may leave fp32's range where the score does not)
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      acc[n][i] = (acc[n][i] + alt[n][i]) * kv_scale * f[n][i & 1];
      alt[n][i] = 0.f;
    }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int piece = 2 * c + ((k + (c >> 1)) & 1);
    const uint4 r0 = *reinterpret_cast<const uint4*>(row0 + kFp4RopeAt + 16 * piece);
    const uint4 r1 = *reinterpret_cast<const uint4*>(row1 + kFp4RopeAt + 16 * piece);
    const uint32_t fa[4] = {r0.x, r1.x, r0.y, r1.y};
    const uint32_t fb[4] = {r0.z, r1.z, r0.w, r1.w};
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const uint4 b = qf[((16 + k) * NT + n) * 32 + lane];
      mma_bf16(acc[n], fa, b.x, b.y);
      mma_bf16(alt[n], fb, b.z, b.w);
    }
  }
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[n][i] += alt[n][i];
}

// O^T: this warp's 512 / W columns over the block's rows.  The MMA's K slots
// 2c, 2c + 1, 2c + 8, 2c + 9 are rows c, c + 4, c + 8, c + 12 of a 16-row tile:
// the four lanes' reads of one row each then fall into different banks.  Lane
// (g, c) widens 64 / W neighbouring columns (all in one scale group): MMA tile
// 4 j + t takes columns 8 j + 2 t (its row g) and 8 j + 2 t + 1 (its row g + 8) of
// the lane's.  P of a head is stored in the order of the slots.  Masked rows are
// zeros and take part: without a branch a tile, the next one's reads and
// conversions start under this one's MMAs (a chunk of 512 tokens: 165 us, 172
// with the branch).
template <int NT, int W, int kPRow>
__device__ __forceinline__ void f4_values(const uint8_t* stage, const __half* pf, float (&o)[32 / W][NT][4], int warp,
                                          int lane) {
  constexpr int kWords = 8 / W;             // 8 codes each, per row
  const int g = lane >> 2, c = lane & 3;
  const uint8_t* base = stage + c * kFp4Slot;
  const int code_at = (256 / W) * warp + (32 / W) * g;
  const int scale_at = kFp4ScaleAt + (code_at >> 3);
#pragma unroll
  for (int kt = 0; kt < W; ++kt) {
    const uint8_t* r = base + kt * kF4TileBytes;
    uint32_t w[4][kWords], s[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (kWords == 2) {
        const uint2 v = *reinterpret_cast<const uint2*>(r + 4 * i * kFp4Slot + code_at);
        w[i][0] = v.x;
        w[i][1] = v.y;
      } else {
        w[i][0] = *reinterpret_cast<const uint32_t*>(r + 4 * i * kFp4Slot + code_at);
      }
      s[i] = r[4 * i * kFp4Slot + scale_at];
    }
    uint2 b[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) b[n] = *reinterpret_cast<const uint2*>(pf + (8 * n + g) * kPRow + 16 * kt + 4 * c);
    const uint32_t f0 = e4m3x2_f16x2(s[0] | (s[1] << 8)), f1 = e4m3x2_f16x2(s[2] | (s[3] << 8));
#pragma unroll
    for (int j = 0; j < kWords; ++j) {
      // byte t: the codes of column 2t (even) or 2t + 1 (odd) of two rows
      uint32_t e0[4], o0[4], e1[4], o1[4];
      e2m1x8_value((w[0][j] & 0x0f0f0f0fu) | ((w[1][j] << 4) & 0xf0f0f0f0u), e0);
      e2m1x8_value(((w[0][j] >> 4) & 0x0f0f0f0fu) | (w[1][j] & 0xf0f0f0f0u), o0);
      e2m1x8_value((w[2][j] & 0x0f0f0f0fu) | ((w[3][j] << 4) & 0xf0f0f0f0u), e1);
      e2m1x8_value(((w[2][j] >> 4) & 0x0f0f0f0fu) | (w[3][j] & 0xf0f0f0f0u), o1);
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const uint32_t a[4] = {mul_f16x2(e0[t], f0), mul_f16x2(o0[t], f0), mul_f16x2(e1[t], f1), mul_f16x2(o1[t], f1)};
#pragma unroll
        for (int n = 0; n < NT; ++n) mma_f16(o[4 * j + t][n], a, b[n].x, b[n].y);
      }
    }
  }
}

// Q of a unit: a warp brings every W-th head's latent part to f16 by 2^-e (the exponent
// of its largest value), leaves the rotated part in bf16 and stores both as MMA
// fragments; qscale[h] = 2^e.  Heads past h_q are zero.
template <int NT, int W>
__device__ __forceinline__ void f4_load_q(const Fp4Params& p, int unit, uint8_t* qbytes, float* qscale, int warp,
                                          int lane) {
  const int tok = unit / p.groups, h0 = (unit % p.groups) * (8 * NT);
#pragma unroll 2
  for (int hl = warp; hl < 8 * NT; hl += W) {
    const int h = h0 + hl, n = hl >> 3, g = hl & 7;
    const bool live = h < p.h_q;
    const uint4* src = reinterpret_cast<const uint4*>(p.q + (static_cast<size_t>(tok) * p.h_q + (live ? h : 0)) * kRowW);
    uint4 v[3];
    v[0] = __ldg(src + lane);
    v[1] = __ldg(src + 32 + lane);
    v[2] = __ldg(src + 64 + (lane & 7));
    float x[3][8];
    float top = 0.f;
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      unpack8(v[k], x[k]);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (!live) x[k][i] = 0.f;
        if (k < 2) top = fmaxf(top, fabsf(x[k][i]));
      }
    }
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
    int e = static_cast<int>(__float_as_uint(top) >> 23) - 127;
    e = top > 0.f && top <= 3.402823466e38f ? min(max(e, -126), 126) : 0;
    const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
    if (lane == 0) qscale[hl] = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
    // values 8 x .. 8 x + 7 (x = lane or 32 + lane) are word j of chunk i of
    // owner c; the owner's iteration i0 has (i0 + c) % 4 = i
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int at = 32 * k + lane;
      const int c = at >> 4, i = (at >> 2) & 3, j = at & 3, i0 = (i - c) & 3;
      uint32_t h2[4];
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const __half2 t = __floats2half2_rn(x[k][2 * y] * down, x[k][2 * y + 1] * down);
        h2[y] = *reinterpret_cast<const uint32_t*>(&t);
      }
      *reinterpret_cast<uint4*>(qbytes + (((i0 * 4 + j) * NT + n) * 32 + 4 * g + c) * 16) =
          make_uint4(h2[0], h2[1], h2[2], h2[3]);
    }
    if (lane < 8) {   // rotated part: piece `lane` belongs to owner c = lane / 2, half kh with (kh + c / 2) % 2 = lane % 2
      const int c = lane >> 1, kh = (lane + (c >> 1)) & 1;
      *reinterpret_cast<uint4*>(qbytes + (((16 + kh) * NT + n) * 32 + 4 * g + c) * 16) = pack8(x[2]);
    }
  }
}

// The pieces of the cut units merged: LSE = ln sum exp(LSE_s), out = sum
// exp(LSE_s - LSE) O_s, in piece order (at most 64 pieces).  A warp takes half of a
// head row: lanes form the pieces' weights, then every lane adds 8 of the 256
// columns, the pieces' reads independent of one another.  Launched as a
// dependent of the decode, so that it is set up while that runs; it reads only
// after the decode has completed.
__global__ void __launch_bounds__(256) fp4_merge_kernel(const __grid_constant__ Fp4Params p, int heads_per_unit) {
  const int lane = static_cast<int>(lane_id());
  const long long item = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const long long row = item >> 1;   // (token, head)
  const int half = static_cast<int>(item & 1);
  const long long total = static_cast<long long>(p.n_tok) * p.groups * p.nb;
  int pieces = 1, c_first = 0, h = 0;
  long long ub = 0;
  if (row < static_cast<long long>(p.n_tok) * p.h_q) {
    const int tok = static_cast<int>(row / p.h_q), hq = static_cast<int>(row - static_cast<long long>(tok) * p.h_q);
    const long long unit = static_cast<long long>(tok) * p.groups + hq / heads_per_unit;
    h = hq % heads_per_unit;
    ub = unit * p.nb;
    c_first = range_cta(ub, total, p.ctas);
    pieces = range_cta(ub + p.nb - 1, total, p.ctas) - c_first + 1;
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (pieces == 1) return;   // one CTA ran the whole unit
  int slot[2];
  float w[2];
  float m = -INFINITY;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    slot[k] = 0;
    w[k] = -INFINITY;
    const int i = lane + 32 * k;
    if (i < pieces) {
      const int cta = c_first + i;
      slot[k] = 2 * cta + (range_start(cta, total, p.ctas) < ub ? 1 : 0);
      w[k] = __ldcg(p.part_lse + static_cast<size_t>(slot[k]) * p.part_rows + h);
    }
    m = fmaxf(m, w[k]);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
#pragma unroll
  for (int k = 0; k < 2; ++k) w[k] = w[k] == -INFINITY ? 0.f : expf(w[k] - m);
  const float l = warp_sum(w[0] + w[1]);
  if (half == 0 && lane == 0) p.lse[row] = l == 0.f ? -INFINITY : m + logf(l);
  const float inv = l == 0.f ? 0.f : 1.f / l;
  float4 a0 = make_float4(0.f, 0.f, 0.f, 0.f), a1 = a0;
#pragma unroll 8
  for (int i = 0; i < pieces; ++i) {
    const int sl = __shfl_sync(0xffffffffu, i < 32 ? slot[0] : slot[1], i & 31);
    const float wi = __shfl_sync(0xffffffffu, i < 32 ? w[0] : w[1], i & 31) * inv;
    const float4* src = reinterpret_cast<const float4*>(p.part_o + (static_cast<size_t>(sl) * p.part_rows + h) * kDv + 256 * half) + lane;
    const float4 v0 = __ldcg(src), v1 = __ldcg(src + 32);
    a0.x += wi * v0.x;
    a0.y += wi * v0.y;
    a0.z += wi * v0.z;
    a0.w += wi * v0.w;
    a1.x += wi * v1.x;
    a1.y += wi * v1.y;
    a1.z += wi * v1.z;
    a1.w += wi * v1.w;
  }
  uint2* o = reinterpret_cast<uint2*>(p.out + row * kDv + 256 * half) + lane;
  o[0] = make_uint2(pack_bf16x2(a0.x, a0.y), pack_bf16x2(a0.z, a0.w));
  o[32] = make_uint2(pack_bf16x2(a1.x, a1.y), pack_bf16x2(a1.z, a1.w));
}

// CTA `rank` of this cluster: its shared address of what is at `local` here.
__device__ __forceinline__ uint32_t cluster_addr(uint32_t local, int rank) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(local), "r"(rank));
  return a;
}
__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ float ld_cluster_f(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The merge of a unit whose pieces are in the shared memory of its cluster's CTAs:
// every CTA forms all pieces' weights, a lane a piece, then adds its share of the
// columns, whose first reads are under way meanwhile (a remote read takes about
// a microsecond).  part: [heads][kF4PartRow] here and at the same place in every
// CTA, lse: [heads], weight: [cluster][heads].
template <class L>
__device__ __forceinline__ void f4_cluster_merge(const Fp4Params& p, int unit, int rank, const float* part, const float* lse,
                                                 float* weight) {
  const int tid = static_cast<int>(threadIdx.x), warp = tid >> 5, lane = tid & 31;
  const int tok = unit / p.groups, h0 = (unit % p.groups) * L::kHeads;
  const int heads = min(L::kHeads, p.h_q - h0);
  const int n = heads * (kDv / 4);   // float4 of the unit's output
  const int hi = (rank + 1) * n / p.cluster;
  int i = rank * n / p.cluster + tid;
  // 8 heads: all pieces' reads of a float4 at once.  More heads: two at a time (a
  // larger batch cost the decode loop registers: 512 tokens x 16 heads 171 us
  // against 167), each CTA from its own piece on, so that they do not all read the
  // same CTA's (one token, 32 heads: 17.1 and 18.3 us; 8 heads: 10.9 and 10.5).
  constexpr int kBatch = L::NT == 1 ? kF4MaxCluster : 2;
  auto piece = [&](int s) { return L::NT == 1 ? s : (rank + s) & (p.cluster - 1); };
  float4 v[kBatch];
  auto read = [&](int s0) {
    const uint32_t at = smem_u32(part + (i / (kDv / 4)) * kF4PartRow + 4 * (i % (kDv / 4)));
#pragma unroll
    for (int s = 0; s < kBatch; ++s)
      if (s0 + s < p.cluster) v[s] = ld_cluster_f4(cluster_addr(at, piece(s0 + s)));
  };
  if (i < hi) read(0);
  constexpr int kMine = L::kHeads / L::W;
  float x[kMine];
#pragma unroll
  for (int k = 0; k < kMine; ++k)
    x[k] = lane < p.cluster ? ld_cluster_f(cluster_addr(smem_u32(lse + warp + k * L::W), lane)) : -INFINITY;
#pragma unroll
  for (int k = 0; k < kMine; ++k) {
    const int h = warp + k * L::W;
    float m = x[k];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float e = x[k] == -INFINITY ? 0.f : expf(x[k] - m);
    const float sum = warp_sum(e);
    if (lane < p.cluster) weight[lane * L::kHeads + h] = sum == 0.f ? 0.f : e / sum;
    if (rank == 0 && lane == 0 && h < heads)
      p.lse[static_cast<size_t>(tok) * p.h_q + h0 + h] = sum == 0.f ? -INFINITY : m + logf(sum);
  }
  __syncthreads();
  while (i < hi) {
    const int h = i / (kDv / 4), c4 = i % (kDv / 4);
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int s0 = 0; s0 < kF4MaxCluster; s0 += kBatch) {
      if (s0 > 0) {
        if (s0 >= p.cluster) break;
        read(s0);
      }
#pragma unroll
      for (int s = 0; s < kBatch; ++s) {
        if (s0 + s < p.cluster) {
          const float w = weight[piece(s0 + s) * L::kHeads + h];
          a.x += w * v[s].x;
          a.y += w * v[s].y;
          a.z += w * v[s].z;
          a.w += w * v[s].w;
        }
      }
    }
    *reinterpret_cast<uint2*>(p.out + (static_cast<size_t>(tok) * p.h_q + h0 + h) * kDv + 4 * c4) =
        make_uint2(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w));
    i += L::kThreads;
    if (i < hi) read(0);
  }
}

template <class L>
__global__ void __launch_bounds__(L::kThreads, L::kPerSm) fp4_decode_kernel(const __grid_constant__ Fp4Params p) {
  constexpr int NT = L::NT, W = L::W;
  extern __shared__ __align__(128) uint8_t f4_smem[];
  uint8_t* qbytes = f4_smem + L::kQOff;
  __half* pf = reinterpret_cast<__half*>(f4_smem + L::kPOff);         // [2][heads][kPRow]
  float* red = reinterpret_cast<float*>(f4_smem + L::kRedOff);        // [W][heads]
  float* qscale = reinterpret_cast<float*>(f4_smem + L::kMiscOff);    // [heads]
  uint32_t* livew = reinterpret_cast<uint32_t*>(qscale + L::kHeads);  // [2][W] validity of a warp's rows
  const int tid = static_cast<int>(threadIdx.x), warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, c = lane & 3;
  asm volatile("griddepcontrol.launch_dependents;");   // the merge may be set up (it waits for this grid's end)

  int n_blocks, unit0, j0, rank = 0;
  if (p.cluster == 0) {
    const long long total = static_cast<long long>(p.n_tok) * p.groups * p.nb;
    // this CTA's first block, over all units' lists laid end to end
    const long long x0 = range_start(static_cast<int>(blockIdx.x), total, p.ctas);
    n_blocks = static_cast<int>(range_start(static_cast<int>(blockIdx.x) + 1, total, p.ctas) - x0);
    unit0 = static_cast<int>(x0 / p.nb);
    j0 = static_cast<int>(x0 % p.nb);
  } else {
    unit0 = static_cast<int>(blockIdx.x) / p.cluster;
    rank = static_cast<int>(blockIdx.x) % p.cluster;
    j0 = rank * p.nb / p.cluster;
    n_blocks = (rank + 1) * p.nb / p.cluster - j0;
  }

  // The gather of this warp's rows goes by pairs of blocks: lane 16 k + r
  // follows row r of block 2 i + k from its list entry (read two pairs ahead)
  // over its page-table entry (one pair ahead) to its slot, so that no step
  // waits for the one before it.
  int eu = unit0, ej = j0 + (lane >> 4), eb = lane >> 4;   // unit, block of the list and block of the CTA
  if (ej >= p.nb) {
    ej -= p.nb;
    ++eu;
  }
  int req_n = 0, len_n = 0, idx_n = -1, idx_p = -1, page_p = -1, slot_n = -1;
  auto read_entry = [&]() {
    idx_n = -1;
    if (eb < n_blocks) {
      const int tok = eu / p.groups;
      req_n = tok / p.s_next;
      len_n = __ldg(p.seqlens + req_n);
      const int e = ej * L::kRows + 16 * warp + (lane & 15);
      if (e < p.topk) idx_n = __ldg(p.indices + static_cast<size_t>(tok) * p.topk + e);
    }
    eb += 2;
    ej += 2;
    while (ej >= p.nb) {   // lists of one block: two units on
      ej -= p.nb;
      ++eu;
    }
  };
  auto look_up = [&]() {
    idx_p = idx_n;
    page_p = -1;
    if (idx_n >= 0 && idx_n < len_n) {
      const int pg = idx_n / p.page_size;
      if (pg < p.max_blocks) page_p = __ldg(p.block_table + static_cast<size_t>(req_n) * p.max_blocks + pg);
    }
  };
  auto resolve = [&]() {
    slot_n = page_p >= 0 && page_p < p.num_blocks ? page_p * p.page_size + idx_p % p.page_size : -1;
  };
  // Copies of this warp's 16 rows of a block (row r's slot is held by lane
  // 16 half + r), eight lanes a row; masked rows are zeros and are not read.
  // Returns the rows' validity.  Past the CTA's last block (live false) nothing
  // is written: a cluster's piece may be there.
  auto copy = [&](int slots, int half, int st, bool live) -> uint32_t {
    const uint32_t valid = (__ballot_sync(0xffffffffu, slots >= 0) >> (16 * half)) & 0xffffu;
    if (live) {
      const uint32_t dst = smem_u32(f4_smem + st * L::kStage + warp * kF4TileBytes);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int r = 4 * q + (lane >> 3), ch = lane & 7;
        const int sl = __shfl_sync(0xffffffffu, slots, 16 * half + r);
        const uint8_t* src = p.cache + static_cast<size_t>(sl < 0 ? 0 : sl) * kFp4Slot + 16 * ch;
        const uint32_t bytes = sl < 0 ? 0u : 16u, d = dst + r * kFp4Slot + 16 * ch;
        cp_async_16(d, src, bytes);
        cp_async_16(d + 128, src + 128, bytes);
        cp_async_16(d + 256, src + 256, bytes);
        if (ch < 2) cp_async_16(d + 384, src + 384, bytes);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    return valid;
  };
  auto prefetch_q = [&](int u) {   // a unit's Q on its way into L2
    const int tok = u / p.groups, h0 = (u % p.groups) * L::kHeads;
    const char* q0 = reinterpret_cast<const char*>(p.q + (static_cast<size_t>(tok) * p.h_q + h0) * kRowW);
    const int bytes = min(L::kHeads, p.h_q - h0) * 2 * kRowW;
    for (int x = 128 * tid; x < bytes; x += 128 * L::kThreads) prefetch_line_l2(q0 + x);
  };
  int slots_a, slots_b;   // the current pair's slots, the next pair's
  prefetch_q(unit0);
  read_entry();
  look_up();
  f4_load_q<NT, W>(p, unit0, qbytes, qscale, warp, lane);   // while the first page-table entries are on their way
  read_entry();
  resolve();
  slots_a = slot_n;
  look_up();
  read_entry();
  uint32_t rows = copy(slots_a, 0, 0, true);   // validity of this warp's rows in block b
  resolve();
  slots_b = slot_n;
  look_up();
  read_entry();

  float o[32 / W][NT][4];
  float m[NT][2], l[NT][2], f[NT][2];   // heads 8 n + 2 c + k: maximum (of the CTA) less kF4PBits, this lane's share of the sum, 2^e
  int unit = unit0, j = j0;
#pragma unroll 1
  for (int b = 0; b < n_blocks; ++b) {
    if (b == 0 || j == 0) {   // a new unit
      if (b > 0) {
        __syncthreads();   // the last unit's Q has been read
        f4_load_q<NT, W>(p, unit, qbytes, qscale, warp, lane);
      }
      __syncthreads();
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          m[n][k] = -INFINITY;
          l[n][k] = 0.f;
          f[n][k] = qscale[8 * n + 2 * c + k];
        }
#pragma unroll
      for (int t = 0; t < 32 / W; ++t)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[t][n][i] = 0.f;
    }
    uint32_t* lw = livew + (b & 1) * W;
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    if (lane == 0) lw[warp] = rows;
    __syncwarp();   // this warp's rows of block b have landed
    const uint8_t* stage = f4_smem + (b & 1) * L::kStage;
    __half* pb = pf + (b & 1) * L::kHeads * L::kPRow;
    float s[NT][4];
    const uint32_t mask = rows;
    const int rho = (g & 4) | ((g & 1) << 1) | ((g >> 1) & 1);
    const bool v0 = (mask >> rho) & 1u, v1 = (mask >> (rho + 8)) & 1u;
    if (mask != 0u) f4_scores<NT>(stage + warp * kF4TileBytes, reinterpret_cast<const uint4*>(qbytes), s, lane, p.kv_scale, f);
    // Scores in log2 units; a maximum moves only when a score passes it by
    // 2^8, always with a unit's first rows.  (The difference is exact where it matters;
    // a sum m + 15 would be rounded to the step of large scores, and P pass f16's range.)
    bool need = false;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s[n][i] = (i < 2 ? v0 : v1) ? s[n][i] * p.scale_log2 : -INFINITY;
        need |= s[n][i] - m[n][i & 1] > 8.0f + kF4PBits;
      }
    // P of row r of this warp's tile sits at 16 warp + 4 (r % 4) + r / 4
    const int at = 16 * warp + 4 * (rho & 3) + (rho >> 2);
    float e[NT][4];
    auto weights = [&]() {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float ms = m[n][k] == -INFINITY ? 0.f : m[n][k];
          e[n][k] = fast_exp2(s[n][k] - ms);
          e[n][2 + k] = fast_exp2(s[n][2 + k] - ms);
          __half* d = pb + (8 * n + 2 * c + k) * L::kPRow + at;
          d[0] = __float2half_rn(e[n][k]);
          d[2] = __float2half_rn(e[n][2 + k]);
        }
    };
    weights();
    // Every warp's P and rows are there, and block b - 1 has been read.
    if (__syncthreads_or(need)) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float top = fmaxf(s[n][k], s[n][2 + k]);
#pragma unroll
          for (int x = 4; x < 32; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
          if (g == 0) red[warp * L::kHeads + 8 * n + 2 * c + k] = top;
        }
      __syncthreads();
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float mn = m[n][k];
#pragma unroll
          for (int w = 0; w < W; ++w) mn = fmaxf(mn, red[w * L::kHeads + 8 * n + 2 * c + k] - kF4PBits);
          const float a = m[n][k] == mn ? 1.f : fast_exp2(m[n][k] - mn);
          m[n][k] = mn;
          l[n][k] *= a;
#pragma unroll
          for (int t = 0; t < 32 / W; ++t) {
            o[t][n][k] *= a;
            o[t][n][2 + k] *= a;
          }
        }
      weights();
      __syncthreads();
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int k = 0; k < 2; ++k) l[n][k] += e[n][k] + e[n][2 + k];
    // Block b + 1 goes where block b - 1 was.
    if ((b & 1) == 0) {
      rows = copy(slots_a, 1, 1, b + 1 < n_blocks);
    } else {
      rows = copy(slots_b, 0, 0, b + 1 < n_blocks);
      slots_a = slots_b;
      resolve();
      slots_b = slot_n;
      look_up();
      read_entry();
    }
    if (b + 1 < n_blocks && j == p.nb - 1) prefetch_q(unit + 1);
    uint32_t any = 0u;   // a block without a valid row adds nothing
#pragma unroll
    for (int w = 0; w < W; ++w) any |= lw[w];
    if (any != 0u) f4_values<NT, W, L::kPRow>(stage, pb, o, warp, lane);
    ++j;
    if (j == p.nb || b == n_blocks - 1) {
      // End of the unit, or of this CTA's piece of it.
      const int tok = unit / p.groups, h0 = (unit % p.groups) * L::kHeads;
      const int heads = min(L::kHeads, p.h_q - h0);
      const bool whole = p.cluster == 0 && j == p.nb && (unit > unit0 || j0 == 0);
      const size_t slot = 2 * static_cast<size_t>(blockIdx.x) + (unit > unit0 ? 1 : 0);
      // (a cluster's piece: the ring and Q are free, every warp past the barrier below is done with them)
      float* part = p.cluster > 0 ? reinterpret_cast<float*>(f4_smem) : p.part_o + slot * p.part_rows * kDv;
      float* part_lse = p.cluster > 0 ? reinterpret_cast<float*>(qbytes) : p.part_lse + slot * p.part_rows;
      const int part_row = p.cluster > 0 ? kF4PartRow : kDv;
      // sums over this warp's rows, then over the warps
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float v = l[n][k];
#pragma unroll
          for (int x = 4; x < 32; x <<= 1) v += __shfl_xor_sync(0xffffffffu, v, x);
          if (g == 0) red[warp * L::kHeads + 8 * n + 2 * c + k] = v;
        }
      __syncthreads();
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int h = 8 * n + 2 * c + k;
          float sum = 0.f;
#pragma unroll
          for (int w = 0; w < W; ++w) sum += red[w * L::kHeads + h];
          const float inv = sum == 0.f ? 0.f : p.kv_scale / sum;
          if (h < heads) {
            if (warp == 0 && g == 0) {
              const float v = sum == 0.f ? -INFINITY : (m[n][k] + log2f(sum)) * 0.69314718055994530942f;
              if (whole) p.lse[static_cast<size_t>(tok) * p.h_q + h0 + h] = v;
              else part_lse[h] = v;
            }
#pragma unroll
            for (int q = 0; q < 8 / W; ++q) {
              float y[8];
#pragma unroll
              for (int t = 0; t < 4; ++t) {
                y[2 * t] = sum == 0.f ? 0.f : o[4 * q + t][n][k] * inv;
                y[2 * t + 1] = sum == 0.f ? 0.f : o[4 * q + t][n][2 + k] * inv;
              }
              const int col = (512 / W) * warp + (64 / W) * g + 8 * q;
              if (whole) {
                *reinterpret_cast<uint4*>(p.out + (static_cast<size_t>(tok) * p.h_q + h0 + h) * kDv + col) = pack8(y);
              } else {
                float4* d = reinterpret_cast<float4*>(part + h * part_row + col);
                d[0] = make_float4(y[0], y[1], y[2], y[3]);
                d[1] = make_float4(y[4], y[5], y[6], y[7]);
              }
            }
          }
        }
      if (j == p.nb) {
        j = 0;
        ++unit;
      }
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  if (p.cluster > 0) {
    cluster_sync();   // every piece is in its CTA's shared memory
    float* lse = reinterpret_cast<float*>(qbytes);
    f4_cluster_merge<L>(p, unit0, rank, reinterpret_cast<const float*>(f4_smem), lse, lse + L::kHeads);
    cluster_sync();   // and stays there until all have read it
  }
}

}  // namespace smla
