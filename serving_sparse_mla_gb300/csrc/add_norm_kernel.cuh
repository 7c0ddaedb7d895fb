// The residual's addition, the RMS norm of the sum and its gradients, over whole
// rows of a model's hidden width.
//
//   z = bf16(x + residual)                       (no residual: z = x)
//   y = bf16(z * rsqrt(mean(z^2) + eps) * w)
//
// and, where 8-bit rows are asked for, codes e4m3(y / 2^k) with the smallest 2^k that
// brings the largest of 128 values (or of the row) to at most 448.  The norm's factor
// is carried to about 46 bits and y rounded once, so that the codes follow from the
// formula alone, not from the order of a sum, and the 8-bit form is the 16-bit form's
// rows in codes.
//
// One CTA takes a row at a time: V vectors of 8 values per thread, vector i of thread t
// at t + i * (threads), so that loads are contiguous and 16 neighbouring lanes hold
// the 128 values under one scale.  A CTA reads its next row before it works on the
// one it has, and a row costs one barrier (two where a scale spans the row).
//
// What bounds it: 16-bit rows and gradients wait for memory (8192 x 7168: 73 us for 470 MB,
// 0.94 of a copy's rate, and 74 to 82 us for the gradients), 8-bit rows for issue (93 us for
// 412 MB): per value some six packed operations on pairs, and per scale four shuffles.  A
// single row takes 4 us, a launch and one trip to memory and back.
#pragma once
#include <cuda_bf16.h>
#include <cstdint>

#include "norm_rope_kernel.cuh"
#include "ptx.cuh"

namespace smla {

constexpr int kAddNormMaxWidth = 16384;
constexpr int kAddNormGroup = 128;   // values under one scale

// Registers of a thread of the forward: 2 CTAs of 448 threads an SM at 7168 values a row.
// 8192 x 7168 in 16 bits and groups: 84.5 and 103.7 us with 40, 75.7 and 95.3 with 48, 73.4
// and 92.9 with 56, 72.3 and 93.2 with 64.
constexpr int kAddNormRegs = 56;

enum AddNormForm : int { kAddNormBf16 = 0, kAddNormGroups = 1, kAddNormRow = 2 };

struct AddNormParams {
  const __nv_bfloat16* x;         // row r at x + r * x_step (backward: z)
  const __nv_bfloat16* residual;  // or null
  const __nv_bfloat16* weight;    // [d]
  long long x_step, residual_step;
  __nv_bfloat16* z;               // [n, d], or null without a residual
  void* out;                      // [n, d] bf16 or e4m3
  float* scales;                  // [n, ceil(d / 128)] or [n]
  int n, d;
  Two sqrt_d, d_eps;              // sqrt(d), d eps
  // backward
  const __nv_bfloat16* dout;
  const __nv_bfloat16* dresidual; // or null
  long long dout_step, dresidual_step;
  __nv_bfloat16* dx;              // [n, d]
  float* part;                    // [CTAs, d] sums of the weight's gradient
  float eps;
};

// Two floats side by side, each operation rounded as on its own.
struct Pair {
  unsigned long long v;
};
__device__ __forceinline__ Pair pair_of(float a, float b) {
  Pair p;
  asm("mov.b64 %0, {%1, %2};" : "=l"(p.v) : "f"(a), "f"(b));
  return p;
}
__device__ __forceinline__ float2 halves(Pair p) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(p.v));
  return f;
}
__device__ __forceinline__ Pair operator+(Pair a, Pair b) {
  Pair p;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(p.v) : "l"(a.v), "l"(b.v));
  return p;
}
__device__ __forceinline__ Pair operator-(Pair a, Pair b) {
  Pair p;
  asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(p.v) : "l"(a.v), "l"(b.v));
  return p;
}
__device__ __forceinline__ Pair operator*(Pair a, Pair b) {
  Pair p;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(p.v) : "l"(a.v), "l"(b.v));
  return p;
}
__device__ __forceinline__ Pair fma(Pair a, Pair b, Pair c) {
  Pair p;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(p.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return p;
}

// Two bf16 values as a pair of floats.
__device__ __forceinline__ Pair unpack2(uint32_t v) { return pair_of(bf16_lo(v), bf16_hi(v)); }
__device__ __forceinline__ uint32_t pack2(Pair p) {
  const float2 f = halves(p);
  return pack_bf16x2(f.x, f.y);
}

// hi + lo += b, two sums side by side (two_add's steps).
__device__ __forceinline__ void pair_two_add(Pair& hi, Pair& lo, Pair b) {
  const Pair s = hi + b, t = s - hi;
  lo = lo + ((hi - (s - t)) + (b - t));
  hi = s;
}

__device__ __forceinline__ Two two_sum(Two a, Two b) { return two_add({a.hi, __fadd_rn(a.lo, b.lo)}, b.hi); }

__device__ __forceinline__ Two two_mul(Two a, Two b) {
  const float p = __fmul_rn(a.hi, b.hi);
  const float e = __fadd_rn(__fmaf_rn(a.hi, b.hi, -p), __fmaf_rn(a.hi, b.lo, __fmul_rn(a.lo, b.hi)));
  return {p, e};
}

// sqrt(d) / sqrt(ss + d eps); where the sum is not finite, what the formula gives in one float.
__device__ __forceinline__ Two norm_factor(Two ss, const AddNormParams& p) {
  const Two s = two_sum(ss, p.d_eps);
  if (!(s.hi <= 3.402823466e38f)) return {rsqrtf(s.hi), 0.f};
  return two_mul(two_rsqrt(s), p.sqrt_d);
}

__device__ __forceinline__ uint4 load_vec(const __nv_bfloat16* row, int vec, int nvec) {
  return vec < nvec ? *reinterpret_cast<const uint4*>(row + 8 * static_cast<size_t>(vec)) : make_uint4(0, 0, 0, 0);
}

// The power of two under which `top` is at most 448 (k kept in [-64, 31]; 1 for zeros).
__device__ __forceinline__ int scale_exponent(float top) {
  const uint32_t b = __float_as_uint(top);
  const int k = static_cast<int>(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);   // 448 = 1.75 * 2^8
  return top > 0.f ? min(max(k, -64), 31) : 0;
}

// Eight products u (exact floats) times the factor hi + lo, rounded once to bf16 (nearest
// even).  |lo| of a renormalised product is at most half an ulp of its high part, so it
// matters only where that lies halfway between two bf16 numbers, which is seldom: one
// test for all eight.
__device__ __forceinline__ uint4 times_factor(const Pair (&u)[4], Two f) {
  const Pair fh = pair_of(f.hi, f.hi), fl = pair_of(f.lo, f.lo), minus = pair_of(-1.f, -1.f);
  uint32_t out[4];
  bool tie = false;
  Pair h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const Pair p = u[i] * fh;
    h[i] = p + fma(u[i], fl, fma(u[i], fh, p * minus));
    const float2 x = halves(h[i]);
    out[i] = pack_bf16x2(x.x, x.y);
    tie |= (__float_as_uint(x.x) & 0xffffu) == 0x8000u || (__float_as_uint(x.y) & 0xffffu) == 0x8000u;
  }
  if (tie) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 x = halves(u[i]);
      out[i] = pack_bf16x2(two_mul_bf16(x.x, f), two_mul_bf16(x.y, f));
    }
  }
  return make_uint4(out[0], out[1], out[2], out[3]);
}

// The largest magnitude of eight bf16 values as a bf16 bit pattern: a NaN's is above an
// infinity's, and that above every number's.
__device__ __forceinline__ uint32_t largest8(const uint4& v) {
  const uint32_t m = 0x7fff7fffu;
  const uint32_t a = __vmaxu2(__vmaxu2(v.x & m, v.y & m), __vmaxu2(v.z & m, v.w & m));
  return max(a & 0xffffu, a >> 16);
}

// Codes of eight bf16 values times 2^-k.
__device__ __forceinline__ uint2 codes8(const uint4& v, float down) {
  const Pair d = pair_of(down, down);
  const float2 a = halves(unpack2(v.x) * d), b = halves(unpack2(v.y) * d), c = halves(unpack2(v.z) * d),
               e = halves(unpack2(v.w) * d);
  return make_uint2(e4m3x2_of(a.x, a.y) | (e4m3x2_of(b.x, b.y) << 16), e4m3x2_of(c.x, c.y) | (e4m3x2_of(e.x, e.y) << 16));
}

template <int V, int FORM>
__global__ void __maxnreg__(kAddNormRegs) add_norm_kernel(const __grid_constant__ AddNormParams p) {
  __shared__ Two sums[2][32];
  __shared__ uint32_t tops[2][32];
  const int lane = static_cast<int>(lane_id()), warp = static_cast<int>(threadIdx.x >> 5);
  const int warps = static_cast<int>(blockDim.x >> 5), nvec = p.d >> 3;
  const int groups = (p.d + kAddNormGroup - 1) / kAddNormGroup;
  uint4 nx[V], nr[V];
  auto fetch = [&](long long r) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int vec = static_cast<int>(threadIdx.x + i * blockDim.x);
      nx[i] = load_vec(p.x + r * p.x_step, vec, nvec);
      if (p.residual != nullptr) nr[i] = load_vec(p.residual + r * p.residual_step, vec, nvec);
    }
  };
  int buf = 0;
  long long r = blockIdx.x;
  fetch(r);
  for (; r < p.n; r += gridDim.x, buf ^= 1) {
    uint4 z[V];
    Pair hi = pair_of(0.f, 0.f), lo = hi;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int vec = static_cast<int>(threadIdx.x + i * blockDim.x);
      z[i] = nx[i];
      if (p.residual != nullptr) {
        z[i] = make_uint4(pack2(unpack2(nx[i].x) + unpack2(nr[i].x)), pack2(unpack2(nx[i].y) + unpack2(nr[i].y)),
                          pack2(unpack2(nx[i].z) + unpack2(nr[i].z)), pack2(unpack2(nx[i].w) + unpack2(nr[i].w)));
        if (vec < nvec) *reinterpret_cast<uint4*>(p.z + r * p.d + 8 * static_cast<size_t>(vec)) = z[i];
      }
      const Pair a[4] = {unpack2(z[i].x), unpack2(z[i].y), unpack2(z[i].z), unpack2(z[i].w)};
#pragma unroll
      for (int j = 0; j < 4; ++j) pair_two_add(hi, lo, a[j] * a[j]);   // squares of 8-bit numbers: exact
    }
    const float2 sh = halves(hi), sl = halves(lo);
    Two ss = two_sum({sh.x, sl.x}, {sh.y, sl.y});
    if (r + gridDim.x < p.n) fetch(r + gridDim.x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      ss = two_sum(ss, {__shfl_xor_sync(0xffffffffu, ss.hi, o), __shfl_xor_sync(0xffffffffu, ss.lo, o)});
    if (lane == 0) sums[buf][warp] = ss;
    __syncthreads();
    ss = lane < warps ? sums[buf][lane] : Two{0.f, 0.f};
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      ss = two_sum(ss, {__shfl_xor_sync(0xffffffffu, ss.hi, o), __shfl_xor_sync(0xffffffffu, ss.lo, o)});
    const Two f = norm_factor(ss, p);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int vec = static_cast<int>(threadIdx.x + i * blockDim.x);
      const uint4 w = vec < nvec ? __ldg(reinterpret_cast<const uint4*>(p.weight) + vec) : make_uint4(0, 0, 0, 0);
      // 8 x 8 bits: exact
      const Pair u[4] = {unpack2(z[i].x) * unpack2(w.x), unpack2(z[i].y) * unpack2(w.y),
                         unpack2(z[i].z) * unpack2(w.z), unpack2(z[i].w) * unpack2(w.w)};
      z[i] = times_factor(u, f);
      if (FORM == kAddNormBf16 && vec < nvec) reinterpret_cast<uint4*>(p.out)[r * nvec + vec] = z[i];
    }
    if (FORM == kAddNormGroups) {
      uint32_t top = 0;   // of either vector, side by side
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (static_cast<int>(threadIdx.x + i * blockDim.x) < nvec) top |= largest8(z[i]) << (16 * i);
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, o));
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int vec = static_cast<int>(threadIdx.x + i * blockDim.x);
        const uint32_t t = i == 0 ? top << 16 : top & 0xffff0000u;
        const bool bad = t >= 0x7f800000u;
        const int k = scale_exponent(__uint_as_float(t));
        const float down = __uint_as_float(static_cast<uint32_t>(127 - k) << 23);
        if (vec < nvec) {
          reinterpret_cast<uint2*>(p.out)[r * nvec + vec] = bad ? make_uint2(0, 0) : codes8(z[i], down);
          if ((lane & 15) == 0)
            p.scales[r * groups + (vec >> 4)] =
                __uint_as_float(bad ? 0x7fc00000u : static_cast<uint32_t>(127 + k) << 23);
        }
      }
    }
    if (FORM == kAddNormRow) {
      uint32_t row_top = 0;
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (static_cast<int>(threadIdx.x + i * blockDim.x) < nvec) row_top = max(row_top, largest8(z[i]));
      row_top = __reduce_max_sync(0xffffffffu, row_top);
      if (lane == 0) tops[buf][warp] = row_top;
      __syncthreads();
      row_top = __reduce_max_sync(0xffffffffu, lane < warps ? tops[buf][lane] : 0u);
      const bool bad = row_top >= 0x7f80u;
      const int k = scale_exponent(__uint_as_float(row_top << 16));
      const float down = __uint_as_float(static_cast<uint32_t>(127 - k) << 23);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int vec = static_cast<int>(threadIdx.x + i * blockDim.x);
        if (vec < nvec) reinterpret_cast<uint2*>(p.out)[r * nvec + vec] = bad ? make_uint2(0, 0) : codes8(z[i], down);
      }
      if (threadIdx.x == 0) p.scales[r] = __uint_as_float(bad ? 0x7fc00000u : static_cast<uint32_t>(127 + k) << 23);
    }
  }
}

// With g = w dout and zhat = z r, r = rsqrt(mean z^2 + eps):
//   dx = r (g - zhat mean(g zhat)) + dresidual,   dw = sum over rows of dout zhat.
// A thread's columns are the same in every row, so its share of dw stays in registers.
template <int V>
__global__ void __launch_bounds__(1024) add_norm_bwd_kernel(const __grid_constant__ AddNormParams p) {
  __shared__ float2 sums[2][32];
  asm volatile("griddepcontrol.launch_dependents;");   // the weight's sums may be set up (they wait for this grid's end)
  const int lane = static_cast<int>(lane_id()), warp = static_cast<int>(threadIdx.x >> 5);
  const int warps = static_cast<int>(blockDim.x >> 5), nvec = p.d >> 3;
  const float inv_d = 1.f / static_cast<float>(p.d);
  Pair acc[V][4];
  uint4 nz[V], ng[V], nr[V];
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = pair_of(0.f, 0.f);
  auto fetch = [&](long long r) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int vec = static_cast<int>(threadIdx.x + i * blockDim.x);
      nz[i] = load_vec(p.x + r * p.x_step, vec, nvec);
      ng[i] = load_vec(p.dout + r * p.dout_step, vec, nvec);
      if (p.dresidual != nullptr) nr[i] = load_vec(p.dresidual + r * p.dresidual_step, vec, nvec);
    }
  };
  auto weight = [&](int vec) {
    return vec < nvec ? __ldg(reinterpret_cast<const uint4*>(p.weight) + vec) : make_uint4(0, 0, 0, 0);
  };
  int buf = 0;
  long long r = blockIdx.x;
  fetch(r);
  for (; r < p.n; r += gridDim.x, buf ^= 1) {
    uint4 zv[V], gv[V], rv[V];
    Pair sq = pair_of(0.f, 0.f), pr = sq;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      zv[i] = nz[i];
      gv[i] = ng[i];
      rv[i] = nr[i];
      const uint4 w = weight(static_cast<int>(threadIdx.x + i * blockDim.x));
      auto step = [&](uint32_t z, uint32_t g, uint32_t u) {
        const Pair a = unpack2(z);
        sq = fma(a, a, sq);
        pr = fma(unpack2(g) * unpack2(u), a, pr);
      };
      step(zv[i].x, gv[i].x, w.x);
      step(zv[i].y, gv[i].y, w.y);
      step(zv[i].z, gv[i].z, w.z);
      step(zv[i].w, gv[i].w, w.w);
    }
    if (r + gridDim.x < p.n) fetch(r + gridDim.x);
    float ss = halves(sq).x + halves(sq).y, dot = halves(pr).x + halves(pr).y;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      ss += __shfl_xor_sync(0xffffffffu, ss, o);
      dot += __shfl_xor_sync(0xffffffffu, dot, o);
    }
    if (lane == 0) sums[buf][warp] = make_float2(ss, dot);
    __syncthreads();
    const float2 t = lane < warps ? sums[buf][lane] : make_float2(0.f, 0.f);
    ss = warp_sum(t.x);
    dot = warp_sum(t.y);
    const float f = rsqrtf(ss * inv_d + p.eps);
    const Pair f2 = pair_of(f, f), c2 = pair_of(-dot * inv_d * f * f, -dot * inv_d * f * f);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int vec = static_cast<int>(threadIdx.x + i * blockDim.x);
      if (vec >= nvec) continue;
      const uint4 w = weight(vec);
      auto step = [&](uint32_t z, uint32_t g, uint32_t u, uint32_t later, Pair& sum) -> uint32_t {
        const Pair a = unpack2(z), y = unpack2(g);
        sum = fma(y, a * f2, sum);
        Pair d = f2 * fma(a, c2, y * unpack2(u));
        if (p.dresidual != nullptr) d = d + unpack2(later);
        return pack2(d);
      };
      uint4 o;
      o.x = step(zv[i].x, gv[i].x, w.x, rv[i].x, acc[i][0]);
      o.y = step(zv[i].y, gv[i].y, w.y, rv[i].y, acc[i][1]);
      o.z = step(zv[i].z, gv[i].z, w.z, rv[i].z, acc[i][2]);
      o.w = step(zv[i].w, gv[i].w, w.w, rv[i].w, acc[i][3]);
      *reinterpret_cast<uint4*>(p.dx + r * p.d + 8 * static_cast<size_t>(vec)) = o;
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int vec = static_cast<int>(threadIdx.x + i * blockDim.x);
    if (vec >= nvec) continue;
    float4* o = reinterpret_cast<float4*>(p.part + static_cast<size_t>(blockIdx.x) * p.d + 8 * static_cast<size_t>(vec));
    o[0] = make_float4(halves(acc[i][0]).x, halves(acc[i][0]).y, halves(acc[i][1]).x, halves(acc[i][1]).y);
    o[1] = make_float4(halves(acc[i][2]).x, halves(acc[i][2]).y, halves(acc[i][3]).x, halves(acc[i][3]).y);
  }
}

// dw = the CTAs' shares added in a fixed order: 32 warps take every 32nd share of 32
// columns, then add their sums.  Launched as a dependent of the kernel above; it reads
// only after that has completed.
__global__ void __launch_bounds__(1024) add_norm_weight_grad_kernel(const float* part, float* dw, int ctas, int d) {
  __shared__ float sums[32][33];
  const int lane = static_cast<int>(lane_id()), warp = static_cast<int>(threadIdx.x >> 5);
  const int c = static_cast<int>(blockIdx.x) * 32 + lane;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float s = 0.f;
  if (c < d) {
#pragma unroll 8
    for (int i = warp; i < ctas; i += 32) s += __ldcg(part + static_cast<size_t>(i) * d + c);
  }
  sums[warp][lane] = s;
  __syncthreads();
  s = warp_sum(sums[lane][warp]);   // column `warp`, one share per lane
  const int o = static_cast<int>(blockIdx.x) * 32 + warp;
  if (lane == 0 && o < d) dw[o] = s;
}

}  // namespace smla
