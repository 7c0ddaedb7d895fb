// RMS norm, position rotation and cache write of the latent attention's rows,
// and the gradients of the first two.
//
// A row has 576 values: a latent part a (512) and a rotated part r (64).
//
//   y  = a * rsqrt(mean(a^2) + eps) * w        (no weight: y = a)
//   r' = R(position) r                         (32 planes, each turned by its angle)
//
// Query rows ([n_tok, h_q, 576]) take q_weight, the token's latent row
// ([n_tok, 576]) takes kv_weight and goes into its cache slot as well.
//
// One warp takes one row: 8 values of either half of the latent part per lane
// (two 16-byte loads, each 512 contiguous bytes per warp) and one 4-byte pair
// of the rotated part, so that a row is read once and written once and every
// statistic is a warp reduction.  Both directions are bound by memory: 8192
// tokens x 64 heads take 185 us forward (1.23 GB, 6640 GB/s, 0.98 of the rate
// measured for a copy) and 363 us backward (2.46 GB, 6760 GB/s, 0.995); 2119 x 8
// takes 11.9 and 20.6 us (3840 and 4290 GB/s: a launch's start and end are 4 us of
// it); one token 3.4 us, a launch.
//
// 512 squares are summed as fp32 numbers before they are divided: a row whose mean
// square is 2^119 or more is outside of what the norm is made for.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>

#include "ptx.cuh"

namespace smla {

constexpr int kRowW = 576;    // values of a row
constexpr int kLatW = 512;    // its latent part
constexpr int kFp4Slot = 416;       // bytes of a 4-bit cache slot: 256 of codes,
constexpr int kFp4ScaleAt = 256;    // 32 scales,
constexpr int kFp4RopeAt = 288;     // 64 bf16 values
constexpr int kFp8Slot = 656;       // FP8 slot: 512 codes, 4 fp32 scales, 64 bf16 values
constexpr int kFp8ScaleAt = 512;
constexpr int kFp8RopeAt = 528;
constexpr int kNormWarps = 8;       // warps per CTA

enum CacheFormat : int { kCacheBf16 = 0, kCacheFp8 = 1, kCacheFp4 = 2 };

struct NormParams {
  const __nv_bfloat16* q;    // rows at q + t * q_tok + h * q_head
  const __nv_bfloat16* kv;   // rows at kv + t * kv_tok
  long long q_tok, q_head, kv_tok;
  const int32_t* positions;  // [n_tok]
  const float* cos_sin;      // [n_pos, 64]: 32 cosines, 32 sines
  const __nv_bfloat16* q_weight;
  const __nv_bfloat16* kv_weight;
  float eps;
  int interleaved, n_pos, n_tok, h_q;
  // forward
  __nv_bfloat16* q_out;      // [n_tok, h_q, 576]
  __nv_bfloat16* kv_out;     // [n_tok, 576] or null
  uint8_t* cache;
  const int32_t* slots;      // [n_tok]
  int format, n_slots;
  int zero_q, zero_kv;       // padding rows of q_out / kv_out are written with zeros
  float kv_scale, kv_scale6;
  // backward
  const float* dq;           // [n_tok, h_q, 576]
  const float* dkv;          // [n_tok, 576]
  __nv_bfloat16* dq_in;      // [n_tok, h_q, 576]
  __nv_bfloat16* dkv_in;     // [n_tok, 576]
  float* part_q;             // [CTAs, 512] sums of the q weight's gradient
  float* part_kv;            // [CTAs, 512]
};

__device__ __forceinline__ float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

__device__ __forceinline__ void unpack8(const uint4& v, float* x) {
  x[0] = bf16_lo(v.x); x[1] = bf16_hi(v.x); x[2] = bf16_lo(v.y); x[3] = bf16_hi(v.y);
  x[4] = bf16_lo(v.z); x[5] = bf16_hi(v.z); x[6] = bf16_lo(v.w); x[7] = bf16_hi(v.w);
}
__device__ __forceinline__ uint4 pack8(const float* x) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                    pack_bf16x2(x[6], x[7]));
}

__device__ __forceinline__ void zero_row(__nv_bfloat16* row, int lane) {
  const uint4 z = make_uint4(0, 0, 0, 0);
  *reinterpret_cast<uint4*>(row + 8 * lane) = z;
  *reinterpret_cast<uint4*>(row + 256 + 8 * lane) = z;
  *reinterpret_cast<uint32_t*>(row + kLatW + 2 * lane) = 0u;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The two rotated values of this lane (values 2 lane and 2 lane + 1 of the
// rotated part), turned by the position's angles; sign = -1 turns back.
// Interleaved: the lane holds a whole plane, number `lane`.  Else plane i is
// values i and i + 32: lanes l and l + 16 hold the two sides of planes
// 2 (l % 16) and 2 (l % 16) + 1 and swap them.
__device__ __forceinline__ float2 rotate_pair(float2 x, const float* table, int lane, bool interleaved, float sign) {
  if (interleaved) {
    const float c = __ldg(table + lane), s = sign * __ldg(table + 32 + lane);
    return make_float2(x.x * c - x.y * s, x.x * s + x.y * c);
  }
  const int i = 2 * (lane & 15);
  const float2 c = __ldg(reinterpret_cast<const float2*>(table + i));
  float2 s = __ldg(reinterpret_cast<const float2*>(table + 32 + i));
  const float ox = __shfl_xor_sync(0xffffffffu, x.x, 16), oy = __shfl_xor_sync(0xffffffffu, x.y, 16);
  const float t = lane < 16 ? -sign : sign;   // first side: a c - b s, second: b c + a s
  return make_float2(x.x * c.x + t * s.x * ox, x.y * c.y + t * s.y * oy);
}

// ------------------------------------------------------------------ two-float sums
// The latent row's values are rounded to cache codes.  A value next to a
// code's border falls on one side or the other by its last bits, so the norm
// of that row is carried to about 46 bits (pairs hi + lo of floats, with the
// error-free sum and product) and rounded once: the codes then follow from
// the formula alone, not from the order of a sum.  This is 1 row in h_q + 1.
// (Sums: Knuth's, The Art of Computer Programming 2, 4.2.2; products: Dekker's, A
// floating-point technique for extending the available precision, 1971, with a fused
// multiply-add.  46 bits where the low parts are normal numbers: mean squares within
// [2^-100, 2^100]; outside of that fewer.)
struct Two {
  float hi, lo;
};

__device__ __forceinline__ Two two_add(Two a, float b) {   // a + b, the error of the high parts kept
  const float s = __fadd_rn(a.hi, b);
  const float t = __fsub_rn(s, a.hi);
  const float e = __fadd_rn(__fsub_rn(a.hi, __fsub_rn(s, t)), __fsub_rn(b, t));
  return {s, __fadd_rn(a.lo, e)};
}

// (a + b)^-1/2 as hi + lo: the hardware's estimate r and one Newton step whose
// residual 1 - v r^2 is formed with fused multiply-adds.
__device__ __forceinline__ Two two_rsqrt(Two v) {
  const float h = __fadd_rn(v.hi, v.lo);
  const float l = __fsub_rn(v.lo, __fsub_rn(h, v.hi));
  const float r = rsqrtf(h);
  const float p = __fmul_rn(r, r), pl = __fmaf_rn(r, r, -p);
  float t = __fmaf_rn(-h, p, 1.0f);
  t = __fmaf_rn(-h, pl, t);
  t = __fmaf_rn(-l, p, t);
  return {r, __fmul_rn(r, __fmaf_rn(0.375f * t, t, 0.5f * t))};
}

// u * r rounded once to bf16 (nearest even), u an exact float.  After the
// renormalisation |lo| <= half an ulp of hi, so lo matters only where hi lies
// halfway between two bf16 numbers.
__device__ __forceinline__ float two_mul_bf16(float u, Two r) {
  const float p = __fmul_rn(u, r.hi);
  const float e = __fmaf_rn(u, r.lo, __fmaf_rn(u, r.hi, -p));
  const float h = __fadd_rn(p, e);
  const float l = __fsub_rn(e, __fsub_rn(h, p));
  uint32_t b = __float_as_uint(h);
  if ((b & 0xffffu) == 0x8000u && l != 0.f) b += (l > 0.f) == (h > 0.f) ? 1u : 0xffffffffu;
  return __bfloat162float(__float2bfloat16_rn(__uint_as_float(b)));
}

// ------------------------------------------------------------------ codes

__device__ __forceinline__ uint32_t e4m3x2_of(float lo, float hi) {
  unsigned short v;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(v) : "f"(hi), "f"(lo));
  return v;
}
__device__ __forceinline__ float2 e4m3x2_value(uint32_t v) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<unsigned short>(v)));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
// Eight values as e2m1 codes, the first in the lowest four bits.
__device__ __forceinline__ uint32_t e2m1x8_of(const float* x) {
  uint32_t v;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(v)
      : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
  return v;
}
// The four bytes of v, two codes each, as f16 pairs (exact).
__device__ __forceinline__ void e2m1x8_value(uint32_t v, uint32_t* h) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(v));
}

// Eight values y of half `half` of a row (columns 256 half + 8 lane ..) into
// the slot; y becomes what the slot stands for.
//
// FP8: the 16 lanes of a 128-column tile share the scale 2^k, the smallest
// with largest / 2^k <= 448 (k kept in [-64, 31]; 1 for a tile of zeros):
// code * 2^k is then exact in bf16.
__device__ __forceinline__ void store_fp8(uint8_t* slot, bool keep, int half, int lane, float* y) {
  float top = 0.f;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    top = fmaxf(top, fabsf(y[i]));
    bad |= !(fabsf(y[i]) <= 3.402823466e38f);
  }
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  bad = (__ballot_sync(0xffffffffu, bad) & (lane < 16 ? 0xffffu : 0xffff0000u)) != 0u;
  const uint32_t b = __float_as_uint(top);
  int k = static_cast<int>(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);   // 448 = 1.75 * 2^8
  k = top > 0.f ? min(max(k, -64), 31) : 0;
  const float up = __uint_as_float(static_cast<uint32_t>(127 + k) << 23);
  const float down = __uint_as_float(static_cast<uint32_t>(127 - k) << 23);
  const float scale = bad ? __uint_as_float(0x7fc00000u) : up;
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    c[i] = bad ? 0u : e4m3x2_of(y[2 * i] * down, y[2 * i + 1] * down);
    const float2 v = e4m3x2_value(c[i]);
    y[2 * i] = v.x * scale;
    y[2 * i + 1] = v.y * scale;
  }
  if (keep) {
    *reinterpret_cast<uint2*>(slot + 256 * half + 8 * lane) = make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
    if ((lane & 15) == 0) *reinterpret_cast<float*>(slot + kFp8ScaleAt + 4 * (2 * half + (lane >> 4))) = scale;
  }
}

// 4 bits: two lanes share a group of 16 and its scale
// e4m3(largest / (6 kv_scale)), at least 2^-9; code = e2m1(y / step), step = scale
// kv_scale.  6 kv_scale, the step and both quotients are fp32, rounded to nearest:
// with a factor that is not a power of two quotients near a code's border are
// common, and that rounding is part of the cache's definition.  y / step is one
// multiplication by the rounded reciprocal and its correction by the remainder
// (Markstein, Computation of elementary functions on the IBM RISC System/6000
// processor, 1990), the correctly rounded quotient; values past 8 steps, all of code
// 6, are cut there, so that it stays finite where the scale is at its largest.
__device__ __forceinline__ void store_fp4(uint8_t* slot, bool keep, int half, int lane, float kv_scale, float kv_scale6,
                                          float* y) {
  float top = 0.f;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    top = fmaxf(top, fabsf(y[i]));
    bad |= !(fabsf(y[i]) <= 3.402823466e38f);
  }
  top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
  bad = (__ballot_sync(0xffffffffu, bad) & (3u << (lane & 30))) != 0u;
  const uint32_t sc = bad ? 0x7fu : (e4m3x2_of(fmaxf(top / kv_scale6, 0x1p-9f), 0.f) & 0xffu);
  const float step = e4m3x2_value(sc).x * kv_scale;
  const float inv = 1.0f / step;
  float x[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float v = fminf(fmaxf(y[i], -8.f * step), 8.f * step);
    const float t = __fmul_rn(v, inv);
    x[i] = __fmaf_rn(__fmaf_rn(-t, step, v), inv, t);
  }
  const uint32_t c = bad ? 0u : e2m1x8_of(x);
  uint32_t h[4];
  e2m1x8_value(c, h);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
    y[2 * i] = v.x * step;
    y[2 * i + 1] = v.y * step;
  }
  if (keep) {
    *reinterpret_cast<uint32_t*>(slot + 128 * half + 4 * lane) = c;
    if ((lane & 1) == 0) slot[kFp4ScaleAt + 16 * half + (lane >> 1)] = static_cast<uint8_t>(sc);
  }
}

// ------------------------------------------------------------------ forward

// A row as this lane holds it: 8 values of either latent half, one pair of the
// rotated part, and where the row belongs.
struct NormRow {
  uint4 v0, v1;
  uint32_t vr;
  int t, h, pos;
};

__device__ __forceinline__ NormRow load_row(const NormParams& p, long long r, int lane) {
  NormRow x;
  x.t = static_cast<int>(r / (p.h_q + 1));
  x.h = static_cast<int>(r - static_cast<long long>(x.t) * (p.h_q + 1));
  const __nv_bfloat16* row = x.h == p.h_q ? p.kv + static_cast<long long>(x.t) * p.kv_tok
                                          : p.q + static_cast<long long>(x.t) * p.q_tok + static_cast<long long>(x.h) * p.q_head;
  x.v0 = *reinterpret_cast<const uint4*>(row + 8 * lane);
  x.v1 = *reinterpret_cast<const uint4*>(row + 256 + 8 * lane);
  x.vr = *reinterpret_cast<const uint32_t*>(row + kLatW + 2 * lane);
  x.pos = __ldg(p.positions + x.t);
  return x;
}

// The latent row of token t: norm carried in two floats, rotation, kv_out and
// the slot.
__device__ __forceinline__ void norm_kv_row(const NormParams& p, const NormRow& x, int lane) {
  const int t = x.t, pos = x.pos;
  const uint4 v0 = x.v0, v1 = x.v1;
  const uint32_t vr = x.vr;
  float y[16];
  unpack8(v0, y);
  unpack8(v1, y + 8);
  if (p.kv_weight != nullptr) {
    Two ss = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 16; ++i) ss = two_add(ss, __fmul_rn(y[i], y[i]));   // squares of 8-bit numbers: exact
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float h = __shfl_xor_sync(0xffffffffu, ss.hi, o), l = __shfl_xor_sync(0xffffffffu, ss.lo, o);
      ss = two_add({ss.hi, __fadd_rn(ss.lo, l)}, h);
    }
    const Two r = two_rsqrt(two_add({ss.hi * (1.f / kLatW), ss.lo * (1.f / kLatW)}, p.eps));
    float w[16];
    unpack8(__ldg(reinterpret_cast<const uint4*>(p.kv_weight + 8 * lane)), w);
    unpack8(__ldg(reinterpret_cast<const uint4*>(p.kv_weight + 256 + 8 * lane)), w + 8);
#pragma unroll
    for (int i = 0; i < 16; ++i) y[i] = two_mul_bf16(__fmul_rn(y[i], w[i]), r);   // 8 x 8 bits: exact
  }
  const float2 rr = rotate_pair(make_float2(bf16_lo(vr), bf16_hi(vr)), p.cos_sin + static_cast<size_t>(pos) * 64, lane,
                                p.interleaved != 0, 1.f);
  const uint32_t rope = pack_bf16x2(rr.x, rr.y);
  // without a cache n_slots is 0 and slots may be null
  const int s = p.n_slots > 0 ? __ldg(p.slots + t) : -1;
  const bool keep = s >= 0 && s < p.n_slots;
  if (p.format == kCacheBf16) {
    if (keep) {
      uint8_t* slot = p.cache + static_cast<size_t>(s) * (2 * kRowW);
      *reinterpret_cast<uint4*>(slot + 16 * lane) = pack8(y);
      *reinterpret_cast<uint4*>(slot + 512 + 16 * lane) = pack8(y + 8);
      *reinterpret_cast<uint32_t*>(slot + 2 * kLatW + 4 * lane) = rope;
    }
  } else {
    const bool fp8 = p.format == kCacheFp8;
    uint8_t* slot = p.cache + static_cast<size_t>(keep ? s : 0) * (fp8 ? kFp8Slot : kFp4Slot);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      if (fp8) store_fp8(slot, keep, half, lane, y + 8 * half);
      else store_fp4(slot, keep, half, lane, p.kv_scale, p.kv_scale6, y + 8 * half);
    }
    if (keep) *reinterpret_cast<uint32_t*>(slot + (fp8 ? kFp8RopeAt : kFp4RopeAt) + 4 * lane) = rope;
  }
  if (p.kv_out != nullptr) {
    __nv_bfloat16* o = p.kv_out + static_cast<size_t>(t) * kRowW;
    *reinterpret_cast<uint4*>(o + 8 * lane) = pack8(y);
    *reinterpret_cast<uint4*>(o + 256 + 8 * lane) = pack8(y + 8);
    *reinterpret_cast<uint32_t*>(o + kLatW + 2 * lane) = rope;
  }
}

__device__ __forceinline__ void norm_q_row(const NormParams& p, const NormRow& x, int lane) {
  const int t = x.t, h = x.h, pos = x.pos;
  uint4 v0 = x.v0, v1 = x.v1;
  const uint32_t vr = x.vr;
  if (p.q_weight != nullptr) {
    float y[16], w[16];
    unpack8(v0, y);
    unpack8(v1, y + 8);
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) ss += y[i] * y[i];
    const float r = rsqrtf(warp_sum(ss) * (1.f / kLatW) + p.eps);
    unpack8(__ldg(reinterpret_cast<const uint4*>(p.q_weight + 8 * lane)), w);
    unpack8(__ldg(reinterpret_cast<const uint4*>(p.q_weight + 256 + 8 * lane)), w + 8);
#pragma unroll
    for (int i = 0; i < 16; ++i) y[i] = y[i] * r * w[i];
    v0 = pack8(y);
    v1 = pack8(y + 8);
  }
  const float2 rr = rotate_pair(make_float2(bf16_lo(vr), bf16_hi(vr)), p.cos_sin + static_cast<size_t>(pos) * 64, lane,
                                p.interleaved != 0, 1.f);
  __nv_bfloat16* o = p.q_out + (static_cast<size_t>(t) * p.h_q + h) * kRowW;
  *reinterpret_cast<uint4*>(o + 8 * lane) = v0;
  *reinterpret_cast<uint4*>(o + 256 + 8 * lane) = v1;
  *reinterpret_cast<uint32_t*>(o + kLatW + 2 * lane) = pack_bf16x2(rr.x, rr.y);
}

// Rows t (h_q + 1) + h; h = h_q is the latent row.  A warp reads its next row
// before it works on the one it has.
__global__ void __launch_bounds__(kNormWarps * 32) norm_rope_kernel(const __grid_constant__ NormParams p) {
  const int lane = static_cast<int>(lane_id());
  const long long rows = static_cast<long long>(p.n_tok) * (p.h_q + 1);
  const long long step = static_cast<long long>(gridDim.x) * kNormWarps;
  long long r = static_cast<long long>(blockIdx.x) * kNormWarps + (threadIdx.x >> 5);
  if (r >= rows) return;
  NormRow next = load_row(p, r, lane);
  for (; r < rows; r += step) {
    const NormRow x = next;
    if (r + step < rows) next = load_row(p, r + step, lane);
    if (x.pos < 0 || x.pos >= p.n_pos) {   // a padding row: left as it was, or zeros
      if (x.h == p.h_q ? p.zero_kv : p.zero_q)
        zero_row(x.h == p.h_q ? p.kv_out + static_cast<size_t>(x.t) * kRowW
                              : p.q_out + (static_cast<size_t>(x.t) * p.h_q + x.h) * kRowW, lane);
      continue;
    }
    if (x.h == p.h_q) norm_kv_row(p, x, lane);
    else norm_q_row(p, x, lane);
  }
}

// ------------------------------------------------------------------ backward

// A row of the backward as this lane holds it: 16 latent gradients, the pair of
// the rotated part and (normed rows) the 16 latent values.
struct GradRow {
  float4 g[4];
  float2 gr;
  uint4 x0, x1;
  int pos;
};

template <bool kNorm>
__device__ __forceinline__ GradRow load_grad_row(const __nv_bfloat16* x, const float* dy, const int32_t* pos,
                                                 int lane) {
  GradRow v;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    v.g[i] = __ldg(reinterpret_cast<const float4*>(dy + 256 * (i >> 1) + 8 * lane + 4 * (i & 1)));
  v.gr = __ldg(reinterpret_cast<const float2*>(dy + kLatW + 2 * lane));
  if constexpr (kNorm) {
    v.x0 = __ldg(reinterpret_cast<const uint4*>(x + 8 * lane));
    v.x1 = __ldg(reinterpret_cast<const uint4*>(x + 256 + 8 * lane));
  }
  v.pos = __ldg(pos);
  return v;
}

// With g = w dy and xhat = a r, r = rsqrt(mean a^2 + eps):
//   da = r (g - xhat mean(g xhat)),  dw = sum over rows of dy xhat,
// and the rotated part turns back.  One row per warp; acc keeps this warp's
// rows' shares of dw.
template <bool kNorm>
__device__ __forceinline__ void grad_row(const NormParams& p, const GradRow& v, __nv_bfloat16* dx,
                                         const __nv_bfloat16* weight, int lane, float (&acc)[16]) {
  if (v.pos < 0 || v.pos >= p.n_pos) {   // a padding row takes no part in the output
    zero_row(dx, lane);
    return;
  }
  float g[16];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    g[4 * i] = v.g[i].x;
    g[4 * i + 1] = v.g[i].y;
    g[4 * i + 2] = v.g[i].z;
    g[4 * i + 3] = v.g[i].w;
  }
  if constexpr (kNorm) {
    float a[16], w[16];
    unpack8(v.x0, a);
    unpack8(v.x1, a + 8);
    unpack8(__ldg(reinterpret_cast<const uint4*>(weight + 8 * lane)), w);
    unpack8(__ldg(reinterpret_cast<const uint4*>(weight + 256 + 8 * lane)), w + 8);
    float ss = 0.f, dot = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      ss += a[i] * a[i];
      dot += (g[i] * w[i]) * a[i];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      ss += __shfl_xor_sync(0xffffffffu, ss, o);
      dot += __shfl_xor_sync(0xffffffffu, dot, o);
    }
    const float r = rsqrtf(ss * (1.f / kLatW) + p.eps);
    const float c = (dot * (1.f / kLatW)) * r * r;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      acc[i] += g[i] * (a[i] * r);
      g[i] = r * (g[i] * w[i] - a[i] * c);
    }
  }
  *reinterpret_cast<uint4*>(dx + 8 * lane) = pack8(g);
  *reinterpret_cast<uint4*>(dx + 256 + 8 * lane) = pack8(g + 8);
  const float2 rr = rotate_pair(v.gr, p.cos_sin + static_cast<size_t>(v.pos) * 64, lane, p.interleaved != 0, -1.f);
  *reinterpret_cast<uint32_t*>(dx + kLatW + 2 * lane) = pack_bf16x2(rr.x, rr.y);
}

// The CTA's share of dw: its warps' sums added in warp order.
__device__ __forceinline__ void store_part(float (&sums)[kNormWarps][kLatW], float (&acc)[16], float* part, int warp,
                                           int lane) {
  __syncthreads();   // an earlier use of `sums` has been read
#pragma unroll
  for (int i = 0; i < 4; ++i)
    *reinterpret_cast<float4*>(&sums[warp][256 * (i >> 1) + 8 * lane + 4 * (i & 1)]) =
        make_float4(acc[4 * i], acc[4 * i + 1], acc[4 * i + 2], acc[4 * i + 3]);
  __syncthreads();
  for (int c = static_cast<int>(threadIdx.x); c < kLatW; c += kNormWarps * 32) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kNormWarps; ++w) s += sums[w][c];
    part[static_cast<size_t>(blockIdx.x) * kLatW + c] = s;
  }
}

// Query rows first, then the latent rows; a warp reads its next row before it
// works on the one it has.
template <bool kQNorm, bool kKvNorm>
__global__ void __launch_bounds__(kNormWarps * 32, 2) norm_rope_bwd_kernel(const __grid_constant__ NormParams p) {
  __shared__ float sums[kNormWarps][kLatW];
  const int lane = static_cast<int>(lane_id()), warp = static_cast<int>(threadIdx.x >> 5);
  if constexpr (kQNorm || kKvNorm)
    asm volatile("griddepcontrol.launch_dependents;");   // the weights' sums may be set up (they wait for this grid's end)
  const long long step = static_cast<long long>(gridDim.x) * kNormWarps;
  const long long first = static_cast<long long>(blockIdx.x) * kNormWarps + warp;
  float acc[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) acc[i] = 0.f;
  const long long rows = static_cast<long long>(p.n_tok) * p.h_q;
  auto load_q = [&](long long r) {
    const int t = static_cast<int>(r / p.h_q);
    const int h = static_cast<int>(r - static_cast<long long>(t) * p.h_q);
    return load_grad_row<kQNorm>(p.q + static_cast<long long>(t) * p.q_tok + static_cast<long long>(h) * p.q_head,
                                 p.dq + r * kRowW, p.positions + t, lane);
  };
  auto load_kv = [&](long long r) {
    return load_grad_row<kKvNorm>(p.kv + r * p.kv_tok, p.dkv + r * kRowW, p.positions + r, lane);
  };
  if (first < rows) {
    GradRow next = load_q(first);
    for (long long r = first; r < rows; r += step) {
      const GradRow v = next;
      if (r + step < rows) next = load_q(r + step);
      grad_row<kQNorm>(p, v, p.dq_in + r * kRowW, p.q_weight, lane, acc);
    }
  }
  if constexpr (kQNorm) {
    store_part(sums, acc, p.part_q, warp, lane);
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i] = 0.f;
  }
  for (long long r = first; r < p.n_tok; r += step)
    grad_row<kKvNorm>(p, load_kv(r), p.dkv_in + r * kRowW, p.kv_weight, lane, acc);
  if constexpr (kKvNorm) store_part(sums, acc, p.part_kv, warp, lane);
}

// dw = the CTAs' shares added in a fixed order: 32 warps take every 32nd share
// of 32 columns, then add their sums.  Launched as a dependent of the kernel
// above; it reads only after that has completed.
__global__ void __launch_bounds__(1024) norm_weight_grad_kernel(const float* part_q, const float* part_kv, float* dw_q,
                                                                float* dw_kv, int ctas) {
  __shared__ float sums[32][33];
  const float* part = blockIdx.y == 0 ? part_q : part_kv;
  float* dw = blockIdx.y == 0 ? dw_q : dw_kv;
  const int lane = static_cast<int>(lane_id()), warp = static_cast<int>(threadIdx.x >> 5);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (dw == nullptr) return;
  const int c = static_cast<int>(blockIdx.x) * 32 + lane;
  float s = 0.f;
#pragma unroll 8
  for (int i = warp; i < ctas; i += 32) s += __ldcg(part + static_cast<size_t>(i) * kLatW + c);
  sums[warp][lane] = s;
  __syncthreads();
  s = warp_sum(sums[lane][warp]);   // column `warp`, one share per lane
  if (lane == 0) dw[static_cast<int>(blockIdx.x) * 32 + warp] = s;
}

}  // namespace smla
