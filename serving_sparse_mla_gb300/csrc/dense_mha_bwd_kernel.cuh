// Gradients of causal attention over whole prompts in the heads' own space.
//
//   s_ij = scale q_i . k_j  over the keys j that query i sees,
//   lse_i = ln sum_j exp(s_ij),   out_i = sum_j exp(s_ij - lse_i) v_j
//
// A sequence's lq queries are the last lq of its lk positions: local query i sees keys
// 0 .. i + lk - lq.  h_q / h_kv query heads share a key and value head.
#pragma once
#include <cuda_bf16.h>
#include <cstdint>

#include "dense_mha_kernel.cuh"
#include "norm_rope_kernel.cuh"
#include "ptx.cuh"

namespace smla {

struct MhaParams {
  const __nv_bfloat16 *q, *k, *v;          // row (t, h) at q + t q_tok + h q_head
  long long q_tok, q_head, k_tok, k_head, v_tok, v_head;
  const int32_t *cu_q, *cu_kv;             // [batch + 1], null for one dense sequence
  int batch, total_q, total_kv, h_q, h_kv;
  float scale;
  __nv_bfloat16* out;                      // [total_q, h_q, d_v]
  float* lse;                              // [total_q, h_q]
  const __nv_bfloat16* dout;
  long long do_tok, do_head;
  __nv_bfloat16 *dq, *dk, *dv;             // [total, h, d]
  float* delta;                            // [total_q, h_q]: rowsum(dout out)
};

struct MhaSeq {
  int q0, q1, k0, k1;
};

__device__ __forceinline__ MhaSeq mha_seq(const MhaParams& p, int b) {
  if (p.cu_q == nullptr) return {0, p.total_q, 0, p.total_kv};
  MhaSeq s;
  s.q0 = mha_offset(p.cu_q, b, p.total_q);
  s.q1 = max(s.q0, mha_offset(p.cu_q, b + 1, p.total_q));
  s.k0 = mha_offset(p.cu_kv, b, p.total_kv);
  s.k1 = max(s.k0, mha_offset(p.cu_kv, b + 1, p.total_kv));
  return s;
}

// The sequence that holds row r of the offsets `cu` (the last b with cu[b] <= r), or -1.
__device__ __forceinline__ int mha_seq_of(const int32_t* cu, int batch, int r) {
  if (cu == nullptr) return 0;
  int lo = 0, hi = batch - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldg(cu + mid) <= r) lo = mid;
    else hi = mid - 1;
  }
  return __ldg(cu + lo) <= r && r < __ldg(cu + lo + 1) ? lo : -1;
}

// A row of N * 64 values, two per lane and 64.
template <int N>
__device__ __forceinline__ void mha_row(const __nv_bfloat16* row, int lane, float (&x)[2 * N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint32_t v = *reinterpret_cast<const uint32_t*>(row + 64 * i + 2 * lane);
    x[2 * i] = bf16_lo(v);
    x[2 * i + 1] = bf16_hi(v);
  }
}

template <int N>
__device__ __forceinline__ void mha_store(__nv_bfloat16* row, int lane, const float (&x)[2 * N], float f) {
#pragma unroll
  for (int i = 0; i < N; ++i)
    *reinterpret_cast<uint32_t*>(row + 64 * i + 2 * lane) = pack_bf16x2(x[2 * i] * f, x[2 * i + 1] * f);
}

template <int N>
__device__ __forceinline__ float mha_dot(const float (&a)[2 * N], const float (&b)[2 * N]) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < 2 * N; ++i) s += a[i] * b[i];
  return warp_sum(s);
}

// One warp per (query row, head): D = rowsum(dout out) and dq.
template <int NQK>
__global__ void __launch_bounds__(256) dense_mha_dq_kernel(const __grid_constant__ MhaParams p) {
  const int lane = static_cast<int>(lane_id());
  const long long rows = static_cast<long long>(p.total_q) * p.h_q, step = static_cast<long long>(gridDim.x) * 8;
  for (long long r = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5); r < rows; r += step) {
    const int t = static_cast<int>(r / p.h_q), h = static_cast<int>(r % p.h_q);
    float acc[2 * NQK];
#pragma unroll
    for (int i = 0; i < 2 * NQK; ++i) acc[i] = 0.f;
    const int b = mha_seq_of(p.cu_q, p.batch, t);
    if (b >= 0) {
      const MhaSeq s = mha_seq(p, b);
      const int lk = s.k1 - s.k0;
      const int sees = min(lk, t - s.q0 + lk - (s.q1 - s.q0) + 1);
      float q[2 * NQK], k[2 * NQK], v[4], g[4], o[4];
      mha_row<NQK>(p.q + t * p.q_tok + h * p.q_head, lane, q);
      mha_row<2>(p.dout + t * p.do_tok + h * p.do_head, lane, g);
      mha_row<2>(p.out + r * 128, lane, o);
      const float delta = mha_dot<2>(g, o), lse = p.lse[r];
      if (lane == 0) p.delta[r] = delta;
      const int hk = h / (p.h_q / p.h_kv);
      for (int j = 0; j < sees; ++j) {
        mha_row<NQK>(p.k + (s.k0 + j) * p.k_tok + hk * p.k_head, lane, k);
        mha_row<2>(p.v + (s.k0 + j) * p.v_tok + hk * p.v_head, lane, v);
        const float e = __expf(mha_dot<NQK>(q, k) * p.scale - lse);
        const float ds = e * (mha_dot<2>(g, v) - delta);
#pragma unroll
        for (int i = 0; i < 2 * NQK; ++i) acc[i] += ds * k[i];
      }
    }
    mha_store<NQK>(p.dq + r * (64 * NQK), lane, acc, p.scale);
  }
}

// One warp per (key row, key head): dk and dv over the rows that see the key, of every head of the group.
template <int NQK>
__global__ void __launch_bounds__(256) dense_mha_dkv_kernel(const __grid_constant__ MhaParams p) {
  const int lane = static_cast<int>(lane_id());
  const int share = p.h_q / p.h_kv;
  const long long rows = static_cast<long long>(p.total_kv) * p.h_kv, step = static_cast<long long>(gridDim.x) * 8;
  for (long long r = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5); r < rows; r += step) {
    const int t = static_cast<int>(r / p.h_kv), hk = static_cast<int>(r % p.h_kv);
    float dk[2 * NQK], dv[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 2 * NQK; ++i) dk[i] = 0.f;
    const int b = mha_seq_of(p.cu_kv, p.batch, t);
    if (b >= 0) {
      const MhaSeq s = mha_seq(p, b);
      float q[2 * NQK], k[2 * NQK], v[4], g[4];
      mha_row<NQK>(p.k + t * p.k_tok + hk * p.k_head, lane, k);
      mha_row<2>(p.v + t * p.v_tok + hk * p.v_head, lane, v);
      const int first = max(0, t - s.k0 - (s.k1 - s.k0) + (s.q1 - s.q0));
      for (int h = hk * share; h < (hk + 1) * share; ++h) {
        for (int i = s.q0 + first; i < s.q1; ++i) {
          const long long qr = static_cast<long long>(i) * p.h_q + h;
          mha_row<NQK>(p.q + i * p.q_tok + h * p.q_head, lane, q);
          mha_row<2>(p.dout + i * p.do_tok + h * p.do_head, lane, g);
          const float e = __expf(mha_dot<NQK>(q, k) * p.scale - p.lse[qr]);
          const float ds = e * (mha_dot<2>(g, v) - p.delta[qr]);
#pragma unroll
          for (int j = 0; j < 2 * NQK; ++j) dk[j] += ds * q[j];
#pragma unroll
          for (int j = 0; j < 4; ++j) dv[j] += e * g[j];
        }
      }
    }
    mha_store<NQK>(p.dk + r * (64 * NQK), lane, dk, p.scale);
    mha_store<2>(p.dv + r * 128, lane, dv, 1.f);
  }
}

}  // namespace smla
