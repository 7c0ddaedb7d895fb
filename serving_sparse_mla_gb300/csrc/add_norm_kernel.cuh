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
#pragma once
#include <cuda_bf16.h>
#include <cstdint>

#include "norm_rope_kernel.cuh"
#include "ptx.cuh"

namespace smla {

constexpr int kAddNormMaxWidth = 16384;
constexpr int kAddNormGroup = 128;   // values under one scale

enum AddNormForm : int { kAddNormBf16 = 0, kAddNormGroups = 1, kAddNormRow = 2 };

struct AddNormParams {
  const __nv_bfloat16* x;         // row r at x + r * x_step (backward: z)
  const __nv_bfloat16* residual;  // or null
  const __nv_bfloat16* weight;    // [d]
  long long x_step, residual_step;
  __nv_bfloat16* z;               // [n, d], or null without a residual
  void* out;                      // [n, d] bf16 or e4m3
  float* scales;                  // [n, ceil(d / 128)] or [n]
  int n, d, form;
  Two sqrt_d, d_eps;              // sqrt(d), d eps
  // backward
  const __nv_bfloat16* dout;
  const __nv_bfloat16* dresidual; // or null
  long long dout_step, dresidual_step;
  __nv_bfloat16* dx;              // [n, d]
  float* part;                    // [CTAs, d] sums of the weight's gradient
  float eps;
};

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

template <int V>
__global__ void __launch_bounds__(V == 4 ? 512 : 1024) add_norm_kernel(const __grid_constant__ AddNormParams p) {
  __shared__ Two sums[2][32];
  __shared__ float tops[2][32];
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
    Two ss = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int vec = static_cast<int>(threadIdx.x + i * blockDim.x);
      float a[8];
      unpack8(nx[i], a);
      z[i] = nx[i];
      if (p.residual != nullptr) {
        float b[8];
        unpack8(nr[i], b);
#pragma unroll
        for (int j = 0; j < 8; ++j) a[j] += b[j];
        z[i] = pack8(a);
        unpack8(z[i], a);
        if (vec < nvec) *reinterpret_cast<uint4*>(p.z + r * p.d + 8 * static_cast<size_t>(vec)) = z[i];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = two_add(ss, __fmul_rn(a[j], a[j]));   // squares of 8-bit numbers: exact
    }
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
    float row_top = 0.f;   // NaN where a value of the row is not finite
    uint4 y[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int vec = static_cast<int>(threadIdx.x + i * blockDim.x);
      float a[8], w[8];
      unpack8(z[i], a);
      unpack8(vec < nvec ? __ldg(reinterpret_cast<const uint4*>(p.weight) + vec) : make_uint4(0, 0, 0, 0), w);
      bool bad = false;
      float top = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        a[j] = vec < nvec ? two_mul_bf16(__fmul_rn(a[j], w[j]), f) : 0.f;   // 8 x 8 bits: exact
        top = fmaxf(top, fabsf(a[j]));
        bad |= !(fabsf(a[j]) <= 3.402823466e38f);
      }
      if (p.form == kAddNormBf16) {
        if (vec < nvec) reinterpret_cast<uint4*>(p.out)[r * nvec + vec] = pack8(a);
        continue;
      }
      if (p.form == kAddNormRow) {
        y[i] = pack8(a);
        row_top = bad || row_top != row_top ? __uint_as_float(0x7fc00000u) : fmaxf(row_top, top);
        continue;
      }
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      bad = (__ballot_sync(0xffffffffu, bad) & (lane < 16 ? 0xffffu : 0xffff0000u)) != 0u;
      const int k = scale_exponent(top);
      const float down = __uint_as_float(static_cast<uint32_t>(127 - k) << 23);
      uint32_t c[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) c[j] = bad ? 0u : e4m3x2_of(a[2 * j] * down, a[2 * j + 1] * down);
      if (vec < nvec) {
        reinterpret_cast<uint2*>(p.out)[r * nvec + vec] = make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
        if ((lane & 15) == 0)
          p.scales[r * groups + (vec >> 4)] =
              __uint_as_float(bad ? 0x7fc00000u : static_cast<uint32_t>(127 + k) << 23);
      }
    }
    if (p.form == kAddNormRow) {
      // a NaN's image is the largest of the bit patterns of numbers without a sign
      uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(row_top));
      if (lane == 0) tops[buf][warp] = __uint_as_float(top);
      __syncthreads();
      top = __reduce_max_sync(0xffffffffu, lane < warps ? __float_as_uint(tops[buf][lane]) : 0u);
      const bool bad = top > 0x7f800000u;
      const int k = scale_exponent(__uint_as_float(top));
      const float down = __uint_as_float(static_cast<uint32_t>(127 - k) << 23);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int vec = static_cast<int>(threadIdx.x + i * blockDim.x);
        float a[8];
        unpack8(y[i], a);
        uint32_t c[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) c[j] = bad ? 0u : e4m3x2_of(a[2 * j] * down, a[2 * j + 1] * down);
        if (vec < nvec)
          reinterpret_cast<uint2*>(p.out)[r * nvec + vec] = make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
      }
      if (threadIdx.x == 0) p.scales[r] = __uint_as_float(bad ? 0x7fc00000u : static_cast<uint32_t>(127 + k) << 23);
    }
  }
}

// With g = w dout and zhat = z r, r = rsqrt(mean z^2 + eps):
//   dx = r (g - zhat mean(g zhat)) + dresidual,   dw = sum over rows of dout zhat.
// A thread's columns are the same in every row, so its share of dw stays in registers.
template <int V>
__global__ void __launch_bounds__(V == 4 ? 512 : 1024) add_norm_bwd_kernel(const __grid_constant__ AddNormParams p) {
  __shared__ float2 sums[2][32];
  asm volatile("griddepcontrol.launch_dependents;");   // the weight's sums may be set up (they wait for this grid's end)
  const int lane = static_cast<int>(lane_id()), warp = static_cast<int>(threadIdx.x >> 5);
  const int warps = static_cast<int>(blockDim.x >> 5), nvec = p.d >> 3;
  const float inv_d = 1.f / static_cast<float>(p.d);
  float acc[V][8];
  uint4 nz[V], ng[V], nr[V], w[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int vec = static_cast<int>(threadIdx.x + i * blockDim.x);
    w[i] = vec < nvec ? __ldg(reinterpret_cast<const uint4*>(p.weight) + vec) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[i][j] = 0.f;
  }
  auto fetch = [&](long long r) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int vec = static_cast<int>(threadIdx.x + i * blockDim.x);
      nz[i] = load_vec(p.x + r * p.x_step, vec, nvec);
      ng[i] = load_vec(p.dout + r * p.dout_step, vec, nvec);
      if (p.dresidual != nullptr) nr[i] = load_vec(p.dresidual + r * p.dresidual_step, vec, nvec);
    }
  };
  int buf = 0;
  long long r = blockIdx.x;
  fetch(r);
  for (; r < p.n; r += gridDim.x, buf ^= 1) {
    uint4 zv[V], gv[V], rv[V];
    float ss = 0.f, dot = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      zv[i] = nz[i];
      gv[i] = ng[i];
      rv[i] = nr[i];
      float a[8], g[8], u[8];
      unpack8(zv[i], a);
      unpack8(gv[i], g);
      unpack8(w[i], u);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        ss += a[j] * a[j];
        dot += g[j] * u[j] * a[j];
      }
    }
    if (r + gridDim.x < p.n) fetch(r + gridDim.x);
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
    const float c = dot * inv_d * f * f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int vec = static_cast<int>(threadIdx.x + i * blockDim.x);
      if (vec >= nvec) continue;
      float a[8], g[8], u[8];
      unpack8(zv[i], a);
      unpack8(gv[i], g);
      unpack8(w[i], u);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        acc[i][j] += g[j] * (a[j] * f);
        g[j] = f * (g[j] * u[j] - a[j] * c);
      }
      if (p.dresidual != nullptr) {
        unpack8(rv[i], a);
#pragma unroll
        for (int j = 0; j < 8; ++j) g[j] += a[j];
      }
      *reinterpret_cast<uint4*>(p.dx + r * p.d + 8 * static_cast<size_t>(vec)) = pack8(g);
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int vec = static_cast<int>(threadIdx.x + i * blockDim.x);
    if (vec >= nvec) continue;
    float4* o = reinterpret_cast<float4*>(p.part + static_cast<size_t>(blockIdx.x) * p.d + 8 * static_cast<size_t>(vec));
    o[0] = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
    o[1] = make_float4(acc[i][4], acc[i][5], acc[i][6], acc[i][7]);
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
