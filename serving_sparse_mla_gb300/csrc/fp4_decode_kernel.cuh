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
// code * scale is exact in f16.  Q is brought to f16 by a power of two per
// head (bf16 has 8 significant bits; values below 2^-14 of the head's largest
// lose bits below 2^-25 of it, the size of an fp32 sum's own rounding), P is
// f16 (11 bits).  The rotated part stays bf16 (its own MMAs).  All sums are
// fp32.
//
// 256 threads, 64-row blocks in a ring of three (2 x 26 KB in flight per CTA,
// two CTAs per SM): warp w takes rows 16 (w % 4) .. of S^T over half of the
// columns (w / 4), then heads w, w + 8 of the softmax, then columns 64 w .. of
// O^T.  Work is dealt as in the paged forward (block ranges, fwd_kernel.cuh):
// the units' lists laid end to end and cut into one equal range per CTA; the
// CTA that writes a cut unit's last piece merges its pieces.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>

#include "fwd_kernel.cuh"
#include "norm_rope_kernel.cuh"

namespace smla {

constexpr int kF4Threads = 256;
constexpr int kF4Stages = 3;
constexpr int kF4StageBytes = kBlk * kFp4Slot;
constexpr int kF4SRow = kBlk + 4;    // floats of one head's partial scores (the 4 spread the banks)
constexpr int kF4PRow = kBlk + 16;   // f16 values of one head's P

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
  int32_t* merge_count;        // [units], zeroed before the launch
  int n_tok, h_q, topk, s_next, page_size, max_blocks, num_blocks;
  int groups;                  // head groups of a token
  int nb;                      // 64-entry blocks of a list
  int ctas, part_rows;
  float scale_log2;            // sm_scale * log2(e)
  float kv_scale;
};

template <int NT>   // heads / 8 of a group
struct Fp4Layout {
  static constexpr int kHeads = 8 * NT;
  static constexpr int kQOff = kF4Stages * kF4StageBytes;
  static constexpr int kQBytes = 18 * NT * 512;   // 16 latent + 2 rope fragments of 32 lanes x 16 bytes
  static constexpr int kSOff = kQOff + kQBytes;
  static constexpr int kPOff = kSOff + 2 * kHeads * kF4SRow * 4;
  static constexpr int kMiscOff = kPOff + kHeads * kF4PRow * 2;
  static constexpr int kBytes = kMiscOff + 4 * kHeads * 4 + kF4Stages * kBlk * 4 + 64 * 4;
};

// A row of the list, prepared ahead of its copy: the list entry, then its
// page-table entry, then the slot.
struct Fp4Cursor {
  int unit, j;   // unit and block of the list
};

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

// S^T: this warp's 16 rows over its half of the columns.  The MMA's row g is
// row rho(g) = g with bits 0 and 1 swapped, so that the two rows a quarter of
// a warp reads together lie 832 bytes apart: their 16-byte reads fall into
// different banks (416-byte rows step by 8 of 32 banks).  Lane (g, c) owns
// codes 128 c .. 128 c + 127 of its rows, the four 32-code chunks taken in
// an order rotated by c for the same reason; Q's fragments are laid out to
// match (f4_load_q).
template <int NT>
__device__ __forceinline__ void f4_scores(const uint8_t* stage, const uint4* qf, float* s_out, int warp, int lane,
                                          float kv_scale) {
  const int g = lane >> 2, c = lane & 3;
  const int mt = warp & 3, kh = warp >> 2;
  const int rho = (g & 4) | ((g & 1) << 1) | ((g >> 1) & 1);
  const uint8_t* row0 = stage + (16 * mt + rho) * kFp4Slot;
  const uint8_t* row1 = row0 + 8 * kFp4Slot;
  float acc[NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[n][i] = 0.f;
#pragma unroll
  for (int it = 0; it < 2; ++it) {
    const int i0 = 2 * kh + it;
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
        mma_f16(acc[n], fb, b.z, b.w);
      }
    }
  }
  // the rotated part (bf16), after the latent part took kv_scale
  const int piece = 2 * c + ((kh + (c >> 1)) & 1);
  const uint4 r0 = *reinterpret_cast<const uint4*>(row0 + kFp4RopeAt + 16 * piece);
  const uint4 r1 = *reinterpret_cast<const uint4*>(row1 + kFp4RopeAt + 16 * piece);
  const uint32_t fa[4] = {r0.x, r1.x, r0.y, r1.y};
  const uint32_t fb[4] = {r0.z, r1.z, r0.w, r1.w};
#pragma unroll
  for (int n = 0; n < NT; ++n) {
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[n][i] *= kv_scale;
    const uint4 b = qf[((16 + kh) * NT + n) * 32 + lane];
    mma_bf16(acc[n], fa, b.x, b.y);
    mma_bf16(acc[n], fb, b.z, b.w);
  }
  float* dst = s_out + kh * (8 * NT * kF4SRow) + 16 * mt + rho;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    float* d = dst + (8 * n + 2 * c) * kF4SRow;
    d[0] = acc[n][0];
    d[kF4SRow] = acc[n][1];
    d[8] = acc[n][2];
    d[kF4SRow + 8] = acc[n][3];
  }
}

// O^T: columns 64 warp .. 64 warp + 63 over the block's 64 rows.  The MMA's
// K slots 2c, 2c + 1, 2c + 8, 2c + 9 are rows c, c + 4, c + 8, c + 12 of a
// 16-row tile: the four lanes' reads of one row each then fall into different
// banks.  Lane (g, c) widens columns 8 g .. 8 g + 7 of the warp's 64 (half a
// scale group): MMA tile t takes columns 8 g + 2 t (its row g) and 8 g + 2 t + 1
// (its row g + 8).  P of a head is stored in the order of the slots.
template <int NT>
__device__ __forceinline__ void f4_values(const uint8_t* stage, const __half* pf, float (&o)[4][NT][4], int warp,
                                          int lane) {
  const int g = lane >> 2, c = lane & 3;
  const uint8_t* base = stage + c * kFp4Slot;
  const int code_at = 32 * warp + 4 * g, scale_at = kFp4ScaleAt + 4 * warp + (g >> 1);
#pragma unroll
  for (int kt = 0; kt < 4; ++kt) {
    const uint8_t* r = base + 16 * kt * kFp4Slot;
    uint32_t w[4], s[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[i] = *reinterpret_cast<const uint32_t*>(r + 4 * i * kFp4Slot + code_at);
      s[i] = r[4 * i * kFp4Slot + scale_at];
    }
    uint2 b[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n)
      b[n] = *reinterpret_cast<const uint2*>(pf + (8 * n + g) * kF4PRow + 16 * kt + 4 * c);
    const uint32_t f0 = e4m3x2_f16x2(s[0] | (s[1] << 8)), f1 = e4m3x2_f16x2(s[2] | (s[3] << 8));
    // byte t: the codes of column 2t (even) or 2t + 1 (odd) of two rows
    uint32_t e0[4], o0[4], e1[4], o1[4];
    e2m1x8_value((w[0] & 0x0f0f0f0fu) | ((w[1] << 4) & 0xf0f0f0f0u), e0);
    e2m1x8_value(((w[0] >> 4) & 0x0f0f0f0fu) | (w[1] & 0xf0f0f0f0u), o0);
    e2m1x8_value((w[2] & 0x0f0f0f0fu) | ((w[3] << 4) & 0xf0f0f0f0u), e1);
    e2m1x8_value(((w[2] >> 4) & 0x0f0f0f0fu) | (w[3] & 0xf0f0f0f0u), o1);
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const uint32_t a[4] = {mul_f16x2(e0[t], f0), mul_f16x2(o0[t], f0), mul_f16x2(e1[t], f1), mul_f16x2(o1[t], f1)};
#pragma unroll
      for (int n = 0; n < NT; ++n) mma_f16(o[t][n], a, b[n].x, b[n].y);
    }
  }
}

// Q of a unit: warp w brings heads w, w + 8 .. to f16 / bf16 by 2^-e (the
// exponent of the head's largest value) and stores them as MMA fragments;
// qscale[h] = sm_scale log2(e) 2^e.  Heads past h_q are zero.
template <int NT>
__device__ __forceinline__ void f4_load_q(const Fp4Params& p, int unit, uint8_t* qbytes, float* qscale, int warp,
                                          int lane) {
  const int tok = unit / p.groups, h0 = (unit % p.groups) * (8 * NT);
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int h = h0 + 8 * n + warp;
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
        top = fmaxf(top, fabsf(x[k][i]));
      }
    }
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
    int e = static_cast<int>(__float_as_uint(top) >> 23) - 127;
    e = top > 0.f && top <= 3.402823466e38f ? min(max(e, -126), 126) : 0;
    const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
    if (lane == 0) qscale[8 * n + warp] = p.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
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
      *reinterpret_cast<uint4*>(qbytes + (((i0 * 4 + j) * NT + n) * 32 + 4 * warp + c) * 16) =
          make_uint4(h2[0], h2[1], h2[2], h2[3]);
    }
    if (lane < 8) {   // rotated part: piece `lane` belongs to owner c = lane / 2, half kh with (kh + c / 2) % 2 = lane % 2
      const int c = lane >> 1, kh = (lane + (c >> 1)) & 1;
      float y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = x[2][i] * down;
      *reinterpret_cast<uint4*>(qbytes + (((16 + kh) * NT + n) * 32 + 4 * warp + c) * 16) = pack8(y);
    }
  }
}

// The pieces of a cut unit merged, as merge_unit in fwd_kernel.cuh:
// LSE = ln sum exp(LSE_s), out = sum exp(LSE_s - LSE) O_s, in piece order.
// 16 threads per head row.
__device__ __forceinline__ void f4_merge(const Fp4Params& p, int unit, int h0, int heads, int c_first, int pieces) {
  const long long total = static_cast<long long>(p.n_tok) * p.groups * p.nb;
  const long long ub = static_cast<long long>(unit) * p.nb;
  const int tok = unit / p.groups;
  const int c16 = static_cast<int>(threadIdx.x) & 15;
  for (int h = static_cast<int>(threadIdx.x) >> 4; h < heads; h += kF4Threads / 16) {
    float m = -INFINITY, l = 0.f;
    float4 acc[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
    for (int i = 0; i < pieces; ++i) {
      const int cta = c_first + i;
      const size_t slot = 2 * static_cast<size_t>(cta) + (range_start(cta, total, p.ctas) < ub ? 1 : 0);
      const float ls = __ldcg(p.part_lse + slot * p.part_rows + h);
      const float4* src = reinterpret_cast<const float4*>(p.part_o + (slot * p.part_rows + h) * kDv) + c16;
      float4 v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = __ldcg(src + 16 * k);
      if (ls == -INFINITY) continue;
      const float mn = fmaxf(m, ls);
      const float a = expf(m - mn), w = expf(ls - mn);
      l = l * a + w;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        acc[k].x = acc[k].x * a + w * v[k].x;
        acc[k].y = acc[k].y * a + w * v[k].y;
        acc[k].z = acc[k].z * a + w * v[k].z;
        acc[k].w = acc[k].w * a + w * v[k].w;
      }
      m = mn;
    }
    const size_t row = static_cast<size_t>(tok) * p.h_q + h0 + h;
    const float inv = m == -INFINITY ? 0.f : 1.f / l;
    if (c16 == 0) p.lse[row] = m == -INFINITY ? -INFINITY : m + logf(l);
    uint2* o = reinterpret_cast<uint2*>(p.out + row * kDv) + c16;
#pragma unroll
    for (int k = 0; k < 8; ++k)
      o[16 * k] = make_uint2(pack_bf16x2(acc[k].x * inv, acc[k].y * inv), pack_bf16x2(acc[k].z * inv, acc[k].w * inv));
  }
}

template <int NT>
__global__ void __launch_bounds__(kF4Threads, 2) fp4_decode_kernel(const __grid_constant__ Fp4Params p) {
  using L = Fp4Layout<NT>;
  extern __shared__ __align__(128) uint8_t f4_smem[];
  uint8_t* qbytes = f4_smem + L::kQOff;
  float* s_part = reinterpret_cast<float*>(f4_smem + L::kSOff);
  __half* pf = reinterpret_cast<__half*>(f4_smem + L::kPOff);
  float* alpha = reinterpret_cast<float*>(f4_smem + L::kMiscOff);   // [heads] rescale of O
  float* qscale = alpha + L::kHeads;
  float* fin = qscale + L::kHeads;                                  // [heads] 1 / l
  float* lse_s = fin + L::kHeads;
  int* valid = reinterpret_cast<int*>(lse_s + L::kHeads);           // [stages][64]
  int* flag = valid + kF4Stages * kBlk;
  const int tid = static_cast<int>(threadIdx.x), warp = tid >> 5, lane = tid & 31;

  const long long total = static_cast<long long>(p.n_tok) * p.groups * p.nb;
  const long long x0 = range_start(static_cast<int>(blockIdx.x), total, p.ctas);
  const int n_blocks = static_cast<int>(range_start(static_cast<int>(blockIdx.x) + 1, total, p.ctas) - x0);
  const int unit0 = static_cast<int>(x0 / p.nb), j0 = static_cast<int>(x0 % p.nb);

  // Gather: four threads per row.  The list entry of block b + 4, the
  // page-table entry of block b + 3 and the copy of block b + 2 go out
  // together, so none waits for the one before it.
  const int grow = tid >> 2, part = tid & 3;
  Fp4Cursor ci = {unit0, j0};   // next list entry to read
  int n_read = 0;
  int tok_t = 0, idx_t = -1;    // token and entry whose page is looked up next
  int tok_n = 0, idx_n = -1;
  auto read_entry = [&]() {
    idx_n = -1;
    if (n_read < n_blocks) {
      tok_n = ci.unit / p.groups;
      const int e = ci.j * kBlk + grow;
      if (e < p.topk) idx_n = __ldg(p.indices + static_cast<size_t>(tok_n) * p.topk + e);
      if (++ci.j == p.nb) {
        ci.j = 0;
        ++ci.unit;
      }
    }
    ++n_read;
  };
  int page = -1, idx_p = -1;    // page-table entry read, and its list entry
  auto look_up = [&]() {        // list entry (idx_t) -> its page
    page = -1;
    idx_p = idx_t;
    if (idx_t >= 0) {
      const int b = tok_t / p.s_next;
      const int pg = idx_t / p.page_size;
      if (idx_t < __ldg(p.seqlens + b) && pg < p.max_blocks)
        page = __ldg(p.block_table + static_cast<size_t>(b) * p.max_blocks + pg);
    }
  };
  auto copy = [&](int b) {      // block b of this CTA into its ring slot
    const int st = b % kF4Stages;
    const bool ok = page >= 0 && page < p.num_blocks;
    const int row = ok ? page * p.page_size + idx_p % p.page_size : 0;
    const uint8_t* src = p.cache + static_cast<size_t>(row) * kFp4Slot;
    const uint32_t dst = smem_u32(f4_smem + st * kF4StageBytes + grow * kFp4Slot);
    const uint32_t bytes = ok ? 16u : 0u;   // masked rows are zeros and are not read
#pragma unroll
    for (int k = 0; k < 7; ++k)
      if (k < 6 || part < 2) cp_async_16(dst + 16 * (part + 4 * k), src + 16 * (part + 4 * k), bytes);
    if (part == 0) valid[st * kBlk + grow] = ok ? 1 : 0;
    return ok;
  };
  auto advance = [&]() {
    tok_t = tok_n;
    idx_t = idx_n;
  };
  bool ok0, ok1;   // validity of this thread's row in blocks b and b + 1
  read_entry();
  advance();
  read_entry();
  look_up();
  ok0 = copy(0);
  asm volatile("cp.async.commit_group;" ::: "memory");
  advance();
  read_entry();
  look_up();
  ok1 = copy(1);
  asm volatile("cp.async.commit_group;" ::: "memory");
  advance();
  read_entry();
  look_up();

  float o[4][NT][4];
  float m_run[NT], l_run[NT];   // this warp's heads (warp, warp + 8, ..)
  bool any = false;             // a valid row was met in this unit
  int unit = unit0, j = j0;
  for (int b = 0; b < n_blocks; ++b) {
    if (b == 0 || j == 0) {     // a new unit
      if (b > 0) __syncthreads();   // qscale and the fragments of the last unit have been read
      f4_load_q<NT>(p, unit, qbytes, qscale, warp, lane);
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[t][n][i] = 0.f;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        m_run[n] = -INFINITY;
        l_run[n] = 0.f;
      }
      any = false;
    }
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    // block b has landed for every thread, and block b - 1 has been read
    const bool live = __syncthreads_or(ok0) != 0;
    ok0 = ok1;
    ok1 = copy(b + 2);
    asm volatile("cp.async.commit_group;" ::: "memory");
    advance();
    read_entry();
    look_up();
    const uint8_t* stage = f4_smem + (b % kF4Stages) * kF4StageBytes;
    if (live) {
      any = true;
      f4_scores<NT>(stage, reinterpret_cast<const uint4*>(qbytes), s_part, warp, lane, p.kv_scale);
      __syncthreads();
      // Softmax of heads warp, warp + 8, ..: lane l has rows l and l + 32.
      const int* vrow = valid + (b % kF4Stages) * kBlk;
      const bool v0 = vrow[lane] != 0, v1 = vrow[lane + 32] != 0;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int h = 8 * n + warp;
        const float* sa = s_part + h * kF4SRow;
        const float* sb = sa + L::kHeads * kF4SRow;
        const float f = qscale[h];
        const float s0 = v0 ? (sa[lane] + sb[lane]) * f : -INFINITY;
        const float s1 = v1 ? (sa[lane + 32] + sb[lane + 32]) * f : -INFINITY;
        float top = fmaxf(s0, s1);
#pragma unroll
        for (int k = 16; k > 0; k >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
        const float mn = fmaxf(m_run[n], top);
        const float ms = mn == -INFINITY ? 0.f : mn;
        const float a = fast_exp2(m_run[n] - ms);
        const float e0 = fast_exp2(s0 - ms), e1 = fast_exp2(s1 - ms);
        m_run[n] = mn;
        l_run[n] = l_run[n] * a + (e0 + e1);
        // row r of a 16-row tile sits at 4 (r % 4) + r / 4
        const int at = (lane & 16) + 4 * (lane & 3) + ((lane >> 2) & 3);
        pf[h * kF4PRow + at] = __float2half_rn(e0);
        pf[h * kF4PRow + 32 + at] = __float2half_rn(e1);
        if (lane == 0) alpha[h] = a;
      }
      __syncthreads();
      const int c = lane & 3;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float a0 = alpha[8 * n + 2 * c], a1 = alpha[8 * n + 2 * c + 1];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          o[t][n][0] *= a0;
          o[t][n][1] *= a1;
          o[t][n][2] *= a0;
          o[t][n][3] *= a1;
        }
      }
      f4_values<NT>(stage, pf, o, warp, lane);
    }
    ++j;
    if (j == p.nb || b == n_blocks - 1) {
      // End of the unit, or of this CTA's piece of it.
      const int je = j;
      const int tok = unit / p.groups, h0 = (unit % p.groups) * L::kHeads;
      const int heads = min(L::kHeads, p.h_q - h0);
      const long long ub = static_cast<long long>(unit) * p.nb;
      const int c_first = range_cta(ub, total, p.ctas);
      const int pieces = range_cta(ub + p.nb - 1, total, p.ctas) - c_first + 1;
      const bool whole = pieces == 1;
      const size_t slot = 2 * static_cast<size_t>(blockIdx.x) + (x0 < ub ? 1 : 0);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int h = 8 * n + warp;
        const float l = warp_sum(l_run[n]);
        if (lane == 0) {
          const bool some = any && l != 0.f;
          const float v = some ? (m_run[n] + log2f(l)) * 0.69314718055994530942f : -INFINITY;
          fin[h] = some ? p.kv_scale / l : 0.f;
          if (h < heads) {
            if (whole) p.lse[static_cast<size_t>(tok) * p.h_q + h0 + h] = v;
            else p.part_lse[slot * p.part_rows + h] = v;
          }
        }
      }
      __syncthreads();
      const int g = lane >> 2, c = lane & 3;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int h = 8 * n + 2 * c + k;
          if (h < heads) {
            const float f = fin[h];
            float y[8];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
              y[2 * t] = f == 0.f ? 0.f : o[t][n][k] * f;
              y[2 * t + 1] = f == 0.f ? 0.f : o[t][n][k + 2] * f;
            }
            const int col = 64 * warp + 8 * g;
            if (whole) {
              *reinterpret_cast<uint4*>(p.out + (static_cast<size_t>(tok) * p.h_q + h0 + h) * kDv + col) = pack8(y);
            } else {
              float4* d = reinterpret_cast<float4*>(p.part_o + (slot * p.part_rows + h) * kDv + col);
              d[0] = make_float4(y[0], y[1], y[2], y[3]);
              d[1] = make_float4(y[4], y[5], y[6], y[7]);
            }
          }
        }
      if (!whole) {
        // One thread counts the piece with a release add after the barrier
        // that orders every thread's writes before it; the CTA that completes
        // the unit acquires the others' and merges.
        __syncthreads();
        if (tid == 0) {
          const int last = atomic_add_release_gpu(p.merge_count + unit, 1) + 1 == pieces;
          if (last) fence_acquire_gpu();
          *flag = last;
        }
        __syncthreads();
        if (*flag) f4_merge(p, unit, h0, heads, c_first, pieces);
      }
      if (je == p.nb) {
        j = 0;
        ++unit;
      }
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

}  // namespace smla
