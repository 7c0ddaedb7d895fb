// Gradients of causal attention over whole prompts in the heads' own space (tcgen05 + TMA).
//
//   P = exp(scale q k^T - lse),  D = rowsum(dout out),  dS = P (dout V^T - D),
//   dq = scale dS K,   dk = scale dS^T q,   dv = P^T dout
//
// A row that sees one key has P = 1 and out = v, so its dS is 0: T is taken for D there, where
// two sums of the same products, added up in different orders, would leave their rounding.
//
// dk and dv are sums over the queries, dq over the keys: two kernels, each with its own
// accumulators in TMEM and in a fixed order, at the price of forming S and dout V^T
// twice (512 + 640 products a pair at 192 columns where one pass would have 832, but
// that pass would need 640 columns of TMEM where there are 512, and would add dq up
// across CTAs in an order that changes).
//
// dense_mha_dq_kernel: a tile of 128 query rows ((token, head) pairs, as in the forward)
// against the keys that they see, 128 (at 192 columns 96) at a time.
//   warps 0 .. 7   a thread per row and half of the columns.  First dout's row into TMEM
//                  (A of the second product) and D; then per block P from S, and dS from
//                  P and T; dq's rows at the end
//   warps 8, 10    issue   S = Q K^T and T = dout V^T;   dQ += dS K
//   warp 9         one thread issues the TMA loads (K three blocks deep)
//
// dense_mha_dkv_kernel: a tile of 128 keys against the query rows that see them, 64 at a
// time, of every head of the group.
//   warps 0 .. 7   a thread per key and half of the columns: P^T and dS^T
//   warps 8, 11    issue   S^T = K Q^T and T^T = V dout^T;   dV += P^T dout and dK += dS^T Q
//   warp 9         the TMA loads
//   warp 10        the rows' lse and D into shared memory
//
// A signal from the tensor core to the threads that wait for it and back takes about 1000
// cycles, as long as two products of a block.  So P and dS have columns of their own in
// TMEM, and the next block's S and T are formed as soon as this one's have been read: with
// P and dS in the columns of S and T a block of 64 rows took 2250 cycles where 1280 are
// products.  That is what sets the blocks: at 192 columns 96 keys (dq; 2 x 96 + 48 + 192 + 64 columns of TMEM) and
// 64 query rows (dk, dv; 128 + 192 + 2 x 64 + 2 x 32).
//
// What bounds dk and dv at 192 columns: a block's products are 1280 cycles, but 1600 as both
// operands of S^T and T^T come from shared memory and N = 64 (48 cycles for each 16 columns
// where the product itself takes 32).  8192 tokens of 32 heads: 960 us, 2110 cycles a block
// with all that a tile costs once (8000 cycles to the first scores, 5500 for the sums' way
// out); dq 630 us.  At 128 columns K stays in TMEM as A of S^T and a block is 1152 cycles.
//
// Every wait is bounded, as in the forward.  dk's and dv's kernel waits for dq's grid, which has
// a bound of its own, outside of these waits: no warp has one for D under way before.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cstdint>

#include "dense_mha_kernel.cuh"

namespace smla {

enum MhaBwdErrCode : int {
  kErrMhaDqLoadWait = 0x711,
  kErrMhaDqMmaWait = 0x712,
  kErrMhaDqRowsWait = 0x713,
  kErrMhaDkvLoadWait = 0x721,
  kErrMhaDkvMmaWait = 0x722,
  kErrMhaDkvRowsWait = 0x723,
  kErrMhaDkvStatWait = 0x724,
};

struct MhaBwdParams {
  CUtensorMap map_q, map_do, map_o;        // [token, head, d]: boxes 64 x pack x tok_tile
  CUtensorMap map_k, map_v;                // boxes 64 x 1 x the keys of a block (dq: 128, at 192 columns 96; dk, dv: 128)
  const int32_t *cu_q, *cu_kv;             // [batch + 1], null for one dense sequence
  int batch, total_q, total_kv, h_q, h_kv, group;
  int pack, tok_tile;                      // rows of a query tile: tok_tile tokens x pack heads
  MhaDiv per;                              // tok_tile
  int slots;                               // tiles per head (pack) that the grid has room for
  MhaHeads order;
  float scale, scale_log2;
  const __nv_bfloat16 *k, *dout;           // row (t, h) at k + t k_tok + h k_head
  long long k_tok, k_head, do_tok, do_head;
  const float* lse;                        // [total_q, h_q]
  float* delta;                            // [total_q, h_q]: D
  __nv_bfloat16 *dq, *dk, *dv;             // [total, h, d]
  unsigned long long timeout_ns;
};

// Half a row of 128 values as A of a product: 32 columns of TMEM.
__device__ __forceinline__ void mha_row_to_tmem(uint32_t taddr, const uint4 (&x)[8]) {
  const float* f = reinterpret_cast<const float*>(&x[0]);
  tmem_st16(taddr, f);
  tmem_st16(taddr + 16, f + 16);
}

// ------------------------------------------------------------------ dq

constexpr int kMhaDqK = 3, kMhaDqV = 2;   // stages of K and of V

struct __align__(16) MhaDqMisc {
  uint64_t q_full, o_full, k_full[kMhaDqK], k_empty[kMhaDqK], v_full[kMhaDqV], v_empty[kMhaDqV], do_ready, s_full, s_free, t_full, t_free, ds_full, dq_full, drain[2];
  uint32_t tmem_base;
  int abort_flag;
  int prior_error;
  int cleared;   // values of K that are not finite were taken out of a block that some rows do not see all of
  MhaWork work;
  float part[2][kMhaTile];
};

template <int DQK>
struct MhaDqShape {
  static constexpr int kN = DQK == 192 ? 96 : 128;             // keys of a block
  static constexpr int kSub = DQK / 64;
  static constexpr int kKStages = kMhaDqK, kVStages = kMhaDqV;
  static constexpr uint32_t kKUnit = kN * 128;                 // 64 columns of a block
  static constexpr uint32_t kKBytes = kSub * kKUnit, kVBytes = 2 * kKUnit;
  static constexpr uint32_t kKOff = kSub * kMhaUnit, kVOff = kKOff + kKStages * kKBytes;
  // dout and out, until they have been read: in the last stage of K, and behind the first of V
  static constexpr uint32_t kDoOff = kKOff + 2 * kKBytes, kOOff = kVOff + kVBytes;
  static constexpr uint32_t kMiscOff = kOOff + (kVBytes > 2 * kMhaUnit ? kVBytes : 2 * kMhaUnit);
  static constexpr int kBytes = static_cast<int>(kMiscOff) + static_cast<int>(sizeof(MhaDqMisc)) + 1024;
  static constexpr int kThreads = 11 * 32;
  static_assert(kVStages == 2 && kKStages == 3 && kKBytes >= 2 * kMhaUnit, "dout and out");
  // columns of TMEM
  static constexpr uint32_t kS = 0, kT = kN, kDq = 2 * kN, kDs = kDq + DQK, kDo = 448;
  static_assert(kBytes <= kMaxSmem, "shared memory");
  static_assert(kDs + kN / 2 <= kDo, "TMEM");
  static_assert(kMiscOff >= 256 * mha_stage_row<DQK / 64>(), "stage");
};

template <class Misc>
__device__ __forceinline__ void mha_bwd_raise(Misc& m, int code) {
  *reinterpret_cast<volatile int*>(&m.abort_flag) = 1;
  atomicCAS(&g_device_error, 0, code);
}

template <int DQK>
__device__ __forceinline__ bool mha_dq_load(const MhaBwdParams& p, MhaDqMisc& m, uint32_t sb, const MhaWork& w, int t0,
                                            int blocks, int pack0, int& k_fills, int& v_fills) {
  using C = MhaDqShape<DQK>;
  const volatile int* ab = &m.abort_flag;
  uint64_t deadline = global_timer_ns() + p.timeout_ns;
  const int kvh = pack0 / p.group;
  uint32_t bar = smem_u32(&m.q_full);
  mbar_arrive_expect_tx(bar, C::kSub * static_cast<uint32_t>(p.pack * p.tok_tile) * 128u);
  for (int c = 0; c < C::kSub; ++c) tma_load_3d(sb + c * kMhaUnit, &p.map_q, 64 * c, pack0, w.q0 + t0, bar);
  // dout and out for the threads, where block 2's keys and block 1's values come later
  const uint32_t bytes = static_cast<uint32_t>(p.pack * p.tok_tile) * 128u;
  bar = smem_u32(&m.o_full);
  mbar_arrive_expect_tx(bar, 4 * bytes);
  for (int c = 0; c < 2; ++c) {
    tma_load_3d(sb + C::kDoOff + c * kMhaUnit, &p.map_do, 64 * c, pack0, w.q0 + t0, bar);
    tma_load_3d(sb + C::kOOff + c * kMhaUnit, &p.map_o, 64 * c, pack0, w.q0 + t0, bar);
  }
  for (int j = 0; j < blocks; ++j) {
    deadline = global_timer_ns() + p.timeout_ns;
    if (j == 1 && !mbar_wait(smem_u32(&m.do_ready), 0, deadline, ab)) return false;
    const int ks = j % C::kKStages, vs = j % C::kVStages, row = w.k0 + j * C::kN;
    if (!mbar_wait(smem_u32(&m.k_empty[ks]), (j / C::kKStages & 1) ^ 1, deadline, ab)) return false;
    bar = smem_u32(&m.k_full[ks]);
    mbar_arrive_expect_tx(bar, C::kKBytes);
    ++k_fills;
    for (int c = 0; c < C::kSub; ++c)
      tma_load_3d(sb + C::kKOff + ks * C::kKBytes + c * C::kKUnit, &p.map_k, 64 * c, kvh, row, bar);
    if (!mbar_wait(smem_u32(&m.v_empty[vs]), (j / C::kVStages & 1) ^ 1, deadline, ab)) return false;
    bar = smem_u32(&m.v_full[vs]);
    mbar_arrive_expect_tx(bar, C::kVBytes);
    ++v_fills;
    for (int c = 0; c < 2; ++c)
      tma_load_3d(sb + C::kVOff + vs * C::kVBytes + c * C::kKUnit, &p.map_v, 64 * c, kvh, row, bar);
  }
  return true;
}

// S and T of the blocks, each as soon as the one before has been read.
template <int DQK>
__device__ __forceinline__ bool mha_dq_scores(const MhaBwdParams& p, MhaDqMisc& m, uint32_t sb, int blocks) {
  using C = MhaDqShape<DQK>;
  constexpr uint32_t kIdesc = idesc_bf16_f32(kMhaTile, C::kN, false, false);
  const uint64_t q_desc = smem_desc(sb, 16, 1024, SWZ_128B), k_desc = smem_desc(sb + C::kKOff, 16, 1024, SWZ_128B),
                 v_desc = smem_desc(sb + C::kVOff, 16, 1024, SWZ_128B);
  const uint32_t chosen = elect_one();
  const volatile int* ab = &m.abort_flag;
  uint64_t deadline = global_timer_ns() + p.timeout_ns;
  if (!warp_wait(smem_u32(&m.q_full), 0, deadline, ab)) return false;
  for (int j = 0; j < blocks; ++j) {
    deadline = global_timer_ns() + p.timeout_ns;
    const int ks = j % C::kKStages, vs = j % C::kVStages;
    if (!warp_wait(smem_u32(&m.k_full[ks]), j / C::kKStages & 1, deadline, ab)) return false;
    if (j > 0 && !warp_wait(smem_u32(&m.s_free), (j - 1) & 1, deadline, ab)) return false;
    tc_fence_after();
    const uint64_t k = desc_plus(k_desc, ks * C::kKBytes), v = desc_plus(v_desc, vs * C::kVBytes);
#pragma unroll
    for (int kk = 0; kk < DQK / 16; ++kk)
      mma_ss(chosen, C::kS, desc_plus(q_desc, (kk >> 2) * kMhaUnit + (kk & 3) * 32),
             desc_plus(k, (kk >> 2) * C::kKUnit + (kk & 3) * 32), kIdesc, kk > 0 ? 1u : 0u);
    commit_to(chosen, &m.s_full);
    if (!warp_wait(smem_u32(&m.v_full[vs]), j / C::kVStages & 1, deadline, ab)) return false;
    if (!warp_wait(smem_u32(j == 0 ? &m.do_ready : &m.t_free), j == 0 ? 0 : (j - 1) & 1, deadline, ab)) return false;
    tc_fence_after();
#pragma unroll
    for (int kk = 0; kk < kMhaDv / 16; ++kk)
      mma_ts(chosen, C::kT, C::kDo + 8 * kk, desc_plus(v, (kk >> 2) * C::kKUnit + (kk & 3) * 32), kIdesc, kk > 0 ? 1u : 0u);
    commit_to(chosen, &m.t_full);
    commit_to(chosen, &m.v_empty[vs]);
  }
  return true;
}

// dQ += dS K of the blocks.
template <int DQK>
__device__ __forceinline__ bool mha_dq_sums(const MhaBwdParams& p, MhaDqMisc& m, uint32_t sb, int blocks) {
  using C = MhaDqShape<DQK>;
  constexpr uint32_t kIdesc = idesc_bf16_f32(kMhaTile, DQK, false, true);
  const uint64_t k_desc = smem_desc(sb + C::kKOff, C::kKUnit, 1024, SWZ_128B);   // its rows as columns
  const uint32_t chosen = elect_one();
  const volatile int* ab = &m.abort_flag;
  uint64_t deadline = global_timer_ns() + p.timeout_ns;
  for (int j = 0; j < blocks; ++j) {
    deadline = global_timer_ns() + p.timeout_ns;
    const int ks = j % C::kKStages;
    const uint64_t k = desc_plus(k_desc, ks * C::kKBytes);
    if (!warp_wait(smem_u32(&m.ds_full), j & 1, deadline, ab)) return false;
    if (!warp_wait(smem_u32(&m.k_full[ks]), j / C::kKStages & 1, deadline, ab)) return false;   // long past
    tc_fence_after();
#pragma unroll
    for (int kk = 0; kk < C::kN / 16; ++kk)
      mma_ts(chosen, C::kDq, C::kDs + 8 * kk, desc_plus(k, kk * 2048), kIdesc, j + kk > 0 ? 1u : 0u);
    commit_to(chosen, &m.k_empty[ks]);
  }
  commit_to(chosen, &m.dq_full);
  return true;
}

// A key that is not finite and that a row with a finite lse sees has the score -infinite: its dS
// is 0, and 0 times an infinity or a NaN is NaN.  So it is where the product meets the key; for
// keys of the blocks from which such values were taken out, first .. end - 1, the 32 N columns of
// the rows of `asked` are made so here.  One warp, a row per lane; a lane's end is its row's, and
// does not fall from lane to lane.
template <int N>
__device__ __forceinline__ void mha_restore_dq(uint32_t asked, const __nv_bfloat16* keys, long long step, int first, int end,
                                               __nv_bfloat16* out) {
  __syncwarp();   // the rows' own threads have written them
  for (int c = 0; c < N; ++c) {
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    int from = first;
    for (uint32_t left = asked; left != 0u; left &= left - 1) {
      const int row = __ffs(left) - 1, upto = __shfl_sync(0xffffffffu, end, row);
      __nv_bfloat16* o = reinterpret_cast<__nv_bfloat16*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(out), row));
      mha_take_odd<4>(keys + 32 * c, step, from, upto, acc);
      from = max(from, upto);
      float sum[8];
      mha_sum_odd<4>(acc, sum);
      if (lane_id() < 4) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (sum[k] != 0.f) o[32 * c + 8 * lane_id() + k] = __ushort_as_bfloat16(0x7fff);
      }
    }
  }
}

template <int DQK>
__device__ __forceinline__ bool mha_dq_rows(const MhaBwdParams& p, MhaDqMisc& m, uint32_t sb, uint32_t tmem,
                                            const MhaWork& w, int t0, int blocks, int pack0) {
  using C = MhaDqShape<DQK>;
  const volatile int* ab = &m.abort_flag;
  uint64_t deadline = global_timer_ns() + p.timeout_ns;
  const int row = static_cast<int>(threadIdx.x) & 127, half = static_cast<int>(threadIdx.x) >> 7;
  const int lq = w.q1 - w.q0, lk = w.k1 - w.k0;
  const int tok = t0 + row / p.pack, head = pack0 + row % p.pack;
  const bool live = row < p.pack * p.tok_tile && tok < lq;
  const uint32_t lane0 = tmem + (static_cast<uint32_t>((row >> 5) * 32) << 16);
  const size_t at = live ? static_cast<size_t>(w.q0 + tok) * p.h_q + head : 0;
  float lse2 = 0.f, delta = 0.f;
  if (blocks > 0) {
    uint4 g[8];
    float dot = 0.f;
    if (live) lse2 = p.lse[at] * 1.4426950408889634f;
    const bool there = warp_wait(smem_u32(&m.o_full), 0, deadline, ab);   // all threads go on to their barrier
    const uint32_t from = sb + half * kMhaUnit + row * 128;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t at16 = static_cast<uint32_t>((i ^ (row & 7)) * 16);   // 128B swizzle
      uint4 x = ld_shared_v4(from + C::kOOff + at16);
      g[i] = live ? ld_shared_v4(from + C::kDoOff + at16) : make_uint4(0, 0, 0, 0);
      if (!live) x = make_uint4(0, 0, 0, 0);
      float a[8], b[8];
      unpack8(g[i], a);
      unpack8(x, b);
#pragma unroll
      for (int k = 0; k < 8; ++k) dot += a[k] * b[k];
    }
    mha_row_to_tmem(lane0 + C::kDo + 32 * half, g);
    tmem_wait_st();
    tc_fence_before();
    __syncwarp();
    if (lane_id() == 0) mbar_arrive(smem_u32(&m.do_ready));
    m.part[half][row] = dot;
    named_bar_sync(1, 256);
    if (!there) return false;
    delta = m.part[0][row] + m.part[1][row];
    if (!mha_finite(delta)) delta = __uint_as_float(0x7fc00000u);   // all of the row's dS is then NaN
    if (live && half == 0) p.delta[at] = delta;
  }
  constexpr int kHalf = C::kN / 2;
  const bool one = tok + lk == lq;   // the row sees one key: out is its value, and T is D
  const int whole = max(0, t0 + lk - lq + 1) / C::kN;
  const uint32_t ts = lane0 + C::kS + kHalf * half, tt = lane0 + C::kT + kHalf * half,
                 td = lane0 + C::kDs + kHalf / 2 * half;
  for (int j = 0; j < blocks; ++j) {
    deadline = global_timer_ns() + p.timeout_ns;
    if (!warp_wait(smem_u32(&m.s_full), j & 1, deadline, ab)) return false;
    tc_fence_after();
    float s[kHalf], x[kHalf];
    tmem_load<kHalf>(ts, s);
    tc_fence_before();
    __syncwarp();
    if (lane_id() == 0) mbar_arrive(smem_u32(&m.s_free));
    const bool edge = j >= whole;
    if (edge) {   // the product with dS must not meet what is not finite in a hidden key
      const int st = j % C::kKStages;
      if (!warp_wait(smem_u32(&m.k_full[st]), j / C::kKStages & 1, deadline, ab)) return false;
      mha_clear<256>(sb + C::kKOff + st * C::kKBytes, C::kKBytes, &m.cleared);
    }
    const int sees = edge ? tok + lk - lq + 1 - j * C::kN - kHalf * half : kHalf;
#pragma unroll
    for (int i = 0; i < kHalf; i += 2) {
      scale_shift2(s[i], s[i + 1], p.scale_log2, -lse2, -lse2);
      s[i] = fast_exp2(s[i]);
      s[i + 1] = fast_exp2(s[i + 1]);
    }
    if (!warp_wait(smem_u32(&m.t_full), j & 1, deadline, ab)) return false;
    tc_fence_after();
    tmem_load<kHalf>(tt, x);
    tc_fence_before();
    __syncwarp();
    if (lane_id() == 0) mbar_arrive(smem_u32(&m.t_free));
    x[0] = one ? delta : x[0];
#pragma unroll
    for (int i = 0; i < kHalf; i += 2) weigh2(s[i], s[i + 1], x[i], x[i + 1], -delta, -delta);
    if (edge) {
#pragma unroll
      for (int i = 0; i < kHalf; ++i) x[i] = i < sees ? x[i] : 0.f;
    }
    // the product with the dS before has ended when that block's keys are free
    if (j > 0 && !warp_wait(smem_u32(&m.k_empty[(j - 1) % C::kKStages]), (j - 1) / C::kKStages & 1, deadline, ab)) return false;
    tc_fence_after();
    tmem_store_bf16<kHalf>(td, x);
    tmem_wait_st();
    tc_fence_before();
    __syncwarp();
    if (lane_id() == 0) mbar_arrive(smem_u32(&m.ds_full));
  }
  if (blocks > 0) {
    if (!warp_wait(smem_u32(&m.dq_full), 0, deadline, ab)) return false;
    tc_fence_after();
  }
  // Q and K are not needed any more: their memory is the stage
  mha_store_sums<DQK / 64>(p.dq + at * DQK + half * (DQK / 2), sb + threadIdx.x * mha_stage_row<DQK / 64>(),
                           lane0 + C::kDq + half * (DQK / 2), p.scale, blocks > 0, live);
  bulk_wait();
  if (blocks > whole) {   // long past: the other warps' arrivals with their dS of the last block, and what they have found by then
    if (!warp_wait(smem_u32(&m.ds_full), (blocks - 1) & 1, deadline, ab)) return false;
    const uint32_t rows = __ballot_sync(0xffffffffu, live && *reinterpret_cast<volatile int*>(&m.cleared));
    if (rows != 0u)
      mha_restore_dq<DQK / 64>(rows, p.k + w.k0 * p.k_tok + pack0 / p.group * p.k_head + half * (DQK / 2), p.k_tok,
                               whole * C::kN, tok + lk - lq + 1, p.dq + at * DQK + half * (DQK / 2));
  }
  return true;
}

template <int DQK>
__global__ void __launch_bounds__(MhaDqShape<DQK>::kThreads, 1) dense_mha_dq_kernel(const __grid_constant__ MhaBwdParams p) {
  using C = MhaDqShape<DQK>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sbase = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  MhaDqMisc& m = *reinterpret_cast<MhaDqMisc*>(sbase + C::kMiscOff);
  const int warp = static_cast<int>(threadIdx.x >> 5);
  const uint32_t sb = smem_u32(sbase);
  asm volatile("griddepcontrol.launch_dependents;");   // dk's and dv's kernel may be set up (it waits for this grid's end)
  int slot, head;
  mha_unit(static_cast<int>(blockIdx.x), p.slots, p.order, slot, head);
  const int pack0 = head * p.pack;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kKStages; ++i) {
      mbar_init(smem_u32(&m.k_full[i]), 1);
      mbar_init(smem_u32(&m.k_empty[i]), 1);
    }
    for (int i = 0; i < C::kVStages; ++i) {
      mbar_init(smem_u32(&m.v_full[i]), 1);
      mbar_init(smem_u32(&m.v_empty[i]), 1);
    }
    mbar_init(smem_u32(&m.q_full), 1);
    mbar_init(smem_u32(&m.o_full), 1);
    mbar_init(smem_u32(&m.do_ready), 8);   // one arrival per row warp
    mbar_init(smem_u32(&m.s_full), 1);
    mbar_init(smem_u32(&m.s_free), 8);
    mbar_init(smem_u32(&m.t_full), 1);
    mbar_init(smem_u32(&m.t_free), 8);
    mbar_init(smem_u32(&m.ds_full), 8);
    mbar_init(smem_u32(&m.dq_full), 1);
    mbar_init(smem_u32(&m.drain[0]), 1);
    mbar_init(smem_u32(&m.drain[1]), 1);
    m.abort_flag = 0;
    m.cleared = 0;
    m.prior_error = *reinterpret_cast<volatile int*>(&g_device_error);
    fence_mbar_init();
    prefetch_tmap(&p.map_q);
    prefetch_tmap(&p.map_do);
    prefetch_tmap(&p.map_o);
    prefetch_tmap(&p.map_k);
    prefetch_tmap(&p.map_v);
  }
  if (warp == 8) {
    tmem_alloc(smem_u32(&m.tmem_base), 512);
    tmem_relinquish();
  }
  if (warp == 9) {
    const MhaWork w = mha_find<false>(p.cu_q, p.cu_kv, p.batch, p.total_q, p.total_kv, slot, p.per);
    if (lane_id() == 0) m.work = w;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = m.tmem_base;
  const MhaWork w = m.work;

  // rows of no sequence
  if (warp == 9 && w.end < p.total_q && m.prior_error == 0)
    mha_fill_rows(p.dq, static_cast<long long>(p.h_q) * (DQK / 2), w.end, p.total_q, 0u);
  if (m.prior_error == 0 && w.q1 > w.q0) {
    const int lq = w.q1 - w.q0, t0 = w.tile * p.tok_tile;
    const int sees = min(t0 + p.tok_tile, lq) + (w.k1 - w.k0) - lq;   // of the tile's last row
    const int blocks = sees > 0 ? (sees + C::kN - 1) / C::kN : 0;
    const int never = 0;
    if (warp < 8) {
      if (!mha_dq_rows<DQK>(p, m, sb, tmem, w, t0, blocks, pack0)) mha_bwd_raise(m, kErrMhaDqRowsWait);
    } else if ((warp == 8 || warp == 10) && blocks > 0) {
      if (!(warp == 8 ? mha_dq_scores<DQK>(p, m, sb, blocks) : mha_dq_sums<DQK>(p, m, sb, blocks)))
        mha_bwd_raise(m, kErrMhaDqMmaWait);
      uint64_t* drain = &m.drain[warp == 8 ? 0 : 1];
      commit_to(elect_one(), drain);   // every MMA issued completes before TMEM is freed
      mbar_wait(smem_u32(drain), 0, global_timer_ns() + 100000000ull, &never);
    } else if (blocks > 0) {
      if (lane_id() == 0) {
        int kf = 0, vf = 0;
        if (!mha_dq_load<DQK>(p, m, sb, w, t0, blocks, pack0, kf, vf)) mha_bwd_raise(m, kErrMhaDqLoadWait);
        // every copy issued has landed before the CTA exits
        const uint64_t dl = global_timer_ns() + 100000000ull;
        mbar_wait(smem_u32(&m.q_full), 0, dl, &never);
        mbar_wait(smem_u32(&m.o_full), 0, dl, &never);
        for (int i = max(0, kf - C::kKStages); i < kf; ++i)
          mbar_wait(smem_u32(&m.k_full[i % C::kKStages]), i / C::kKStages & 1, dl, &never);
        for (int i = max(0, vf - C::kVStages); i < vf; ++i)
          mbar_wait(smem_u32(&m.v_full[i % C::kVStages]), i / C::kVStages & 1, dl, &never);
      }
      __syncwarp();
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 8) tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------------------ dk, dv

// Until the grid before (dq's) has ended, and all that it has written is there.
__device__ __forceinline__ void mha_other_grid() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

struct __align__(16) MhaDkvMisc {
  uint64_t k_full, k_ready, q_full[4], do_full[4], empty[4];
  uint64_t s_full, s_free, p_full, p_free, t_full, t_free, ds_full, out_full, drain[2];
  uint32_t tmem_base;
  int abort_flag;
  int prior_error;
  int cleared;   // values of dout that are not finite were taken out of a block of which some rows do not see all keys
  MhaWork work;
  alignas(16) float shift[4][64];     // -lse in powers of two and -D of a block's rows, read four at a time
  alignas(16) float minus_d[4][64];
};

template <int DQK>
struct MhaDkvShape {
  static constexpr int kN = 64;                                // query rows of a block
  static constexpr bool kKTmem = DQK == 128;                   // K, A of S^T, in TMEM
  static constexpr int kSub = DQK / 64;
  static constexpr int kStages = DQK == 192 ? 3 : 4;
  static constexpr uint32_t kQUnit = kN * 128;                 // 64 columns of a block
  static constexpr uint32_t kQBytes = kSub * kQUnit, kDoBytes = 2 * kQUnit;
  static constexpr uint32_t kVOff = kKTmem ? 0 : kSub * kMhaUnit;
  static constexpr uint32_t kQOff = kVOff + 2 * kMhaUnit, kDoOff = kQOff + kStages * kQBytes;
  static constexpr uint32_t kMiscOff = kDoOff + kStages * kDoBytes;
  static constexpr int kBytes = static_cast<int>(kMiscOff) + static_cast<int>(sizeof(MhaDkvMisc)) + 1024;
  static constexpr int kThreads = 12 * 32;
  static_assert(kN == 64 && kStages <= 4, "rows and barriers of MhaDkvMisc");
  // columns of TMEM
  static constexpr uint32_t kDv = 0, kDk = 128, kS = 128 + DQK, kT = kS + kN, kP = kT + kN, kDs = kP + kN / 2, kK = 448;
  static_assert(kBytes <= kMaxSmem, "shared memory");
  static_assert(kDs + kN / 2 <= (kKTmem ? kK : 512), "TMEM");
  static_assert(kMiscOff >= 256 * (mha_stage_row<2>() + mha_stage_row<DQK / 64>()), "stage");
};

// The query blocks of one key tile: blocks of tok_tile tokens from the first that sees
// its first key, for each pack of heads of the group.
struct MhaQueries {
  int first, blocks, total;
  __device__ __forceinline__ MhaQueries(const MhaBwdParams& p, const MhaWork& w) {
    const int lq = w.q1 - w.q0, lk = w.k1 - w.k0;
    first = max(0, w.tile * kMhaTile - (lk - lq));
    blocks = first < lq ? p.per.of(lq - first + p.tok_tile - 1) : 0;
    total = blocks * (p.group / p.pack);
  }
};

template <int DQK>
__device__ __forceinline__ bool mha_dkv_load(const MhaBwdParams& p, MhaDkvMisc& m, uint32_t sb, const MhaWork& w,
                                             const MhaQueries& s, int kvh, int& fills) {
  using C = MhaDkvShape<DQK>;
  const volatile int* ab = &m.abort_flag;
  uint64_t deadline = global_timer_ns() + p.timeout_ns;
  const uint32_t kb = smem_u32(&m.k_full);
  mbar_arrive_expect_tx(kb, (C::kKTmem ? 2 : C::kSub + 2) * kMhaUnit);
  for (int c = 0; c < C::kSub && !C::kKTmem; ++c)
    tma_load_3d(sb + c * kMhaUnit, &p.map_k, 64 * c, kvh, w.k0 + w.tile * kMhaTile, kb);
  for (int c = 0; c < 2; ++c) tma_load_3d(sb + C::kVOff + c * kMhaUnit, &p.map_v, 64 * c, kvh, w.k0 + w.tile * kMhaTile, kb);
  const uint32_t bytes = static_cast<uint32_t>(p.pack * p.tok_tile) * 128u;
  int head = kvh * p.group, b = 0, st = 0, turn = 0;
  for (int j = 0; j < s.total; ++j) {
    deadline = global_timer_ns() + p.timeout_ns;
    if (j == C::kStages) {   // the first stages' copies wait for nothing
      mha_other_grid();
      deadline = global_timer_ns() + p.timeout_ns;
    }
    const int tok = w.q0 + s.first + b * p.tok_tile;
    if (!mbar_wait(smem_u32(&m.empty[st]), turn ^ 1, deadline, ab)) return false;
    uint32_t bar = smem_u32(&m.q_full[st]);
    mbar_arrive_expect_tx(bar, C::kSub * bytes);
    for (int c = 0; c < C::kSub; ++c)
      tma_load_3d(sb + C::kQOff + st * C::kQBytes + c * C::kQUnit, &p.map_q, 64 * c, head, tok, bar);
    bar = smem_u32(&m.do_full[st]);
    mbar_arrive_expect_tx(bar, 2 * bytes);
    ++fills;
    for (int c = 0; c < 2; ++c)
      tma_load_3d(sb + C::kDoOff + st * C::kDoBytes + c * C::kQUnit, &p.map_do, 64 * c, head, tok, bar);
    if (++st == C::kStages) {
      st = 0;
      turn ^= 1;
    }
    if (++b == s.blocks) {
      b = 0;
      head += p.pack;
    }
  }
  return true;
}

// S^T and T^T of the blocks, each as soon as the one before has been read.
template <int DQK>
__device__ __forceinline__ bool mha_dkv_scores(const MhaBwdParams& p, MhaDkvMisc& m, uint32_t sb, int total) {
  using C = MhaDkvShape<DQK>;
  constexpr uint32_t kIdesc = idesc_bf16_f32(kMhaTile, C::kN, false, false);
  const uint64_t k_desc = smem_desc(sb, 16, 1024, SWZ_128B), v_desc = smem_desc(sb + C::kVOff, 16, 1024, SWZ_128B),
                 q_desc = smem_desc(sb + C::kQOff, 16, 1024, SWZ_128B), g_desc = smem_desc(sb + C::kDoOff, 16, 1024, SWZ_128B);
  const uint32_t chosen = elect_one();
  const volatile int* ab = &m.abort_flag;
  uint64_t deadline = global_timer_ns() + p.timeout_ns;
  if (!warp_wait(smem_u32(&m.k_full), 0, deadline, ab)) return false;
  if (C::kKTmem && !warp_wait(smem_u32(&m.k_ready), 0, deadline, ab)) return false;
  mha_other_grid();
  int st = 0, turn = 0;
  for (int j = 0; j < total; ++j) {
    deadline = global_timer_ns() + p.timeout_ns;
    const uint64_t q = desc_plus(q_desc, st * C::kQBytes), g = desc_plus(g_desc, st * C::kDoBytes);
    if (!warp_wait(smem_u32(&m.q_full[st]), turn, deadline, ab)) return false;
    if (j > 0 && !warp_wait(smem_u32(&m.s_free), (j - 1) & 1, deadline, ab)) return false;
    tc_fence_after();
#pragma unroll
    for (int kk = 0; kk < DQK / 16; ++kk) {
      const uint64_t b = desc_plus(q, (kk >> 2) * C::kQUnit + (kk & 3) * 32);
      if (C::kKTmem) mma_ts(chosen, C::kS, C::kK + 8 * kk, b, kIdesc, kk > 0 ? 1u : 0u);
      else mma_ss(chosen, C::kS, desc_plus(k_desc, (kk >> 2) * kMhaUnit + (kk & 3) * 32), b, kIdesc, kk > 0 ? 1u : 0u);
    }
    commit_to(chosen, &m.s_full);
    if (!warp_wait(smem_u32(&m.do_full[st]), turn, deadline, ab)) return false;
    if (j > 0 && !warp_wait(smem_u32(&m.t_free), (j - 1) & 1, deadline, ab)) return false;
    tc_fence_after();
#pragma unroll
    for (int kk = 0; kk < kMhaDv / 16; ++kk)
      mma_ss(chosen, C::kT, desc_plus(v_desc, (kk >> 2) * kMhaUnit + (kk & 3) * 32),
             desc_plus(g, (kk >> 2) * C::kQUnit + (kk & 3) * 32), kIdesc, kk > 0 ? 1u : 0u);
    commit_to(chosen, &m.t_full);
    if (++st == C::kStages) {
      st = 0;
      turn ^= 1;
    }
  }
  return true;
}

// dV += P^T dout and dK += dS^T Q of the blocks.  A block's copies are free behind them: S
// and T have been read by then.
template <int DQK>
__device__ __forceinline__ bool mha_dkv_sums(const MhaBwdParams& p, MhaDkvMisc& m, uint32_t sb, int total) {
  using C = MhaDkvShape<DQK>;
  constexpr uint32_t kIdescV = idesc_bf16_f32(kMhaTile, kMhaDv, false, true);
  constexpr uint32_t kIdescK = idesc_bf16_f32(kMhaTile, DQK, false, true);
  const uint64_t q_desc = smem_desc(sb + C::kQOff, C::kQUnit, 1024, SWZ_128B),    // their rows as columns
                 g_desc = smem_desc(sb + C::kDoOff, C::kQUnit, 1024, SWZ_128B);
  mha_other_grid();
  const uint32_t chosen = elect_one();
  const volatile int* ab = &m.abort_flag;
  uint64_t deadline = global_timer_ns() + p.timeout_ns;
  int st = 0, turn = 0;
  for (int j = 0; j < total; ++j) {
    deadline = global_timer_ns() + p.timeout_ns;
    const uint64_t q = desc_plus(q_desc, st * C::kQBytes), g = desc_plus(g_desc, st * C::kDoBytes);
    if (!warp_wait(smem_u32(&m.p_full), j & 1, deadline, ab)) return false;
    if (!warp_wait(smem_u32(&m.do_full[st]), turn, deadline, ab)) return false;
    tc_fence_after();
#pragma unroll
    for (int kk = 0; kk < C::kN / 16; ++kk)
      mma_ts(chosen, C::kDv, C::kP + 8 * kk, desc_plus(g, kk * 2048), kIdescV, j + kk > 0 ? 1u : 0u);
    commit_to(chosen, &m.p_free);
    if (!warp_wait(smem_u32(&m.ds_full), j & 1, deadline, ab)) return false;
    if (!warp_wait(smem_u32(&m.q_full[st]), turn, deadline, ab)) return false;   // long past
    tc_fence_after();
#pragma unroll
    for (int kk = 0; kk < C::kN / 16; ++kk)
      mma_ts(chosen, C::kDk, C::kDs + 8 * kk, desc_plus(q, kk * 2048), kIdescK, j + kk > 0 ? 1u : 0u);
    commit_to(chosen, &m.empty[st]);
    if (++st == C::kStages) {
      st = 0;
      turn ^= 1;
    }
  }
  commit_to(chosen, &m.out_full);
  return true;
}

// The rows' lse (in powers of two) and D, there with the block's copy of Q.  Rows of no token
// weigh nothing.
template <int DQK>
__device__ __forceinline__ bool mha_dkv_stats(const MhaBwdParams& p, MhaDkvMisc& m, const MhaWork& w, const MhaQueries& s,
                                              int kvh) {
  using C = MhaDkvShape<DQK>;
  const volatile int* ab = &m.abort_flag;
  uint64_t deadline = global_timer_ns() + p.timeout_ns;
  const int lane = static_cast<int>(lane_id()), lq = w.q1 - w.q0;
  int head = kvh * p.group, b = 0, st = 0, turn = 0;
  for (int j = 0; j < s.total; ++j) {
    deadline = global_timer_ns() + p.timeout_ns;
    float l[C::kN / 32], d[C::kN / 32];
#pragma unroll
    for (int i = 0; i < C::kN / 32; ++i) {
      const int r = 32 * i + lane, tok = s.first + b * p.tok_tile + r / p.pack;
      l[i] = -INFINITY;
      d[i] = 0.f;
      if (r < p.pack * p.tok_tile && tok < lq) {
        const size_t at = static_cast<size_t>(w.q0 + tok) * p.h_q + head + r % p.pack;
        l[i] = __ldg(p.lse + at) * -1.4426950408889634f;
        d[i] = -__ldcg(p.delta + at);
      }
    }
    if (!warp_wait(smem_u32(&m.empty[st]), turn ^ 1, deadline, ab)) return false;
#pragma unroll
    for (int i = 0; i < C::kN / 32; ++i) {
      m.shift[st][32 * i + lane] = l[i];
      m.minus_d[st][32 * i + lane] = d[i];
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&m.q_full[st]));
    if (++st == C::kStages) {
      st = 0;
      turn ^= 1;
    }
    if (++b == s.blocks) {
      b = 0;
      head += p.pack;
    }
  }
  return true;
}

// As mha_restore, for dv and what is not finite in dout: the columns (64 from `col0` on) of the
// keys of `asked` become the sums of what is not finite in the rows that see the key, of all heads
// of the group; NaN where such a row's lse is not finite, since its weights are NaN.  One warp, a
// key per lane.
__device__ __forceinline__ void mha_restore_dv(const MhaBwdParams& p, uint32_t asked, const MhaWork& w, int key, int kvh,
                                               __nv_bfloat16* out, int col0) {
  const int lane = static_cast<int>(lane_id()), lq = w.q1 - w.q0, lk = w.k1 - w.k0, heads = kvh * p.group;
  int end = lq;
  bool odd = false;   // an lse is not finite
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  __syncwarp();   // the keys' own threads have written them
  while (asked != 0u) {   // from the last key, which the fewest rows see
    const int of = 31 - __clz(asked), first = max(0, __shfl_sync(0xffffffffu, key, of) - (lk - lq));
    __nv_bfloat16* o = reinterpret_cast<__nv_bfloat16*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(out), of));
    asked &= ~(1u << of);
    for (int h = heads; h < heads + p.group; ++h) {
      mha_take_odd<8>(p.dout + w.q0 * p.do_tok + h * p.do_head + col0, p.do_tok, first, end, acc);
      for (int r = first + lane; r < end; r += 32) odd |= !mha_finite(__ldg(p.lse + static_cast<size_t>(w.q0 + r) * p.h_q + h));
    }
    end = first;
    if (__any_sync(0xffffffffu, odd)) acc[0] = acc[1] = acc[2] = acc[3] = acc[4] = acc[5] = acc[6] = acc[7] = __uint_as_float(0x7fc00000u);
    float sum[8];
    mha_sum_odd<8>(acc, sum);
    if (lane < 8) {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (sum[k] != 0.f) o[8 * lane + k] = __float2bfloat16_rn(sum[k]);
    }
  }
}

template <int DQK>
__device__ __forceinline__ bool mha_dkv_rows(const MhaBwdParams& p, MhaDkvMisc& m, uint32_t sb, uint32_t tmem,
                                             const MhaWork& w, const MhaQueries& s, int kvh) {
  using C = MhaDkvShape<DQK>;
  constexpr int kHalf = C::kN / 2;
  const volatile int* ab = &m.abort_flag;
  uint64_t deadline = global_timer_ns() + p.timeout_ns;
  const int row = static_cast<int>(threadIdx.x) & 127, half = static_cast<int>(threadIdx.x) >> 7;
  const int lq = w.q1 - w.q0, lk = w.k1 - w.k0;
  const int key = w.tile * kMhaTile + row;
  const bool live = key < lk;
  const uint32_t lane0 = tmem + (static_cast<uint32_t>((row >> 5) * 32) << 16);
  if (C::kKTmem && s.total > 0) {
    uint4 k[8];
    const uint4* kp = reinterpret_cast<const uint4*>(p.k + (w.k0 + key) * p.k_tok + kvh * p.k_head + 64 * half);
#pragma unroll
    for (int i = 0; i < 8; ++i) k[i] = live ? __ldg(kp + i) : make_uint4(0, 0, 0, 0);
    mha_row_to_tmem(lane0 + C::kK + 32 * half, k);
    tmem_wait_st();
    tc_fence_before();
    __syncwarp();
    if (lane_id() == 0) mbar_arrive(smem_u32(&m.k_ready));
  }
  if (s.total > 0) mha_other_grid();
  const int last_key = min((w.tile + 1) * kMhaTile, lk) - 1;
  const uint32_t ts = lane0 + C::kS + kHalf * half, tt = lane0 + C::kT + kHalf * half,
                 tp = lane0 + C::kP + kHalf / 2 * half, td = lane0 + C::kDs + kHalf / 2 * half;
  static_assert(kMhaSpare <= 4, "columns that are masked");
  // the bits of the last columns that are rows; in the others, zeros, a key that is not finite has a score of NaN
  const int used = p.pack * p.tok_tile - kHalf * half;
  auto bits = [&](int col) { return (col < used ? 0xffffu : 0u) | (col + 1 < used ? 0xffff0000u : 0u); };
  const uint32_t rows[2] = {bits(kHalf - 4), bits(kHalf - 2)};
  int b = 0, st = 0, turn = 0, before = 0, turn_before = 0;   // where the block is, and the one before
  for (int j = 0; j < s.total; ++j) {
    deadline = global_timer_ns() + p.timeout_ns;
    const int t0 = s.first + b * p.tok_tile;
    if (++b == s.blocks) b = 0;
    const bool edge = t0 + lk - lq < last_key || t0 + p.tok_tile > lq;   // some rows do not see all of the keys
    // the columns that see this thread's key, from a token of the block to another (0 to kN: `pack` of them could pass 32 bits)
    const int lo = edge ? p.pack * max(0, key - (lk - lq) - t0) - kHalf * half : 0;
    const int hi = edge ? p.pack * min(C::kN, lq - t0) - kHalf * half : kHalf;
    // the rows' numbers are another warp's plain stores: what tells that they are there is its arrival beside the copy
    // of Q, not the tensor core's on s_full
    if (!warp_wait_both(smem_u32(&m.q_full[st]), turn, smem_u32(&m.s_full), j & 1, deadline, ab)) return false;
    tc_fence_after();
    float x[kHalf], y[kHalf];
    tmem_load<kHalf>(ts, x);
    tc_fence_before();
    __syncwarp();
    if (lane_id() == 0) mbar_arrive(smem_u32(&m.s_free));
    if (edge) {
      // the products with P and dS must not meet what is not finite in a row that does not
      // see a key; the product that gives T has read dout by then
      if (!warp_wait(smem_u32(&m.t_full), j & 1, deadline, ab)) return false;
      if (!warp_wait(smem_u32(&m.do_full[st]), turn, deadline, ab)) return false;
      mha_clear<256>(sb + C::kQOff + st * C::kQBytes, C::kQBytes);
      mha_clear<256>(sb + C::kDoOff + st * C::kDoBytes, C::kDoBytes, &m.cleared);
    }
    const float4* l4 = reinterpret_cast<const float4*>(&m.shift[st][kHalf * half]);
#pragma unroll
    for (int i = 0; i < kHalf; i += 4) {
      const float4 l = l4[i >> 2];
      scale_shift2(x[i], x[i + 1], p.scale_log2, l.x, l.y);
      scale_shift2(x[i + 2], x[i + 3], p.scale_log2, l.z, l.w);
#pragma unroll
      for (int n = 0; n < 4; ++n) x[i + n] = fast_exp2(x[i + n]);
    }
    if (edge) {
#pragma unroll
      for (int i = 0; i < kHalf; ++i) x[i] = i >= lo && i < hi ? x[i] : 0.f;
    }
    if (j > 0 && !warp_wait(smem_u32(&m.p_free), (j - 1) & 1, deadline, ab)) return false;
    tc_fence_after();
    tmem_store_bf16<kHalf>(tp, x, rows);
    tmem_wait_st();
    tc_fence_before();
    __syncwarp();
    if (lane_id() == 0) mbar_arrive(smem_u32(&m.p_full));
    if (!warp_wait(smem_u32(&m.t_full), j & 1, deadline, ab)) return false;
    tc_fence_after();
    tmem_load<kHalf>(tt, y);
    tc_fence_before();
    __syncwarp();
    if (lane_id() == 0) mbar_arrive(smem_u32(&m.t_free));
    const float4* d4 = reinterpret_cast<const float4*>(&m.minus_d[st][kHalf * half]);
    if (t0 == lq - lk && row < 32) {   // the block's first token sees the first key alone, and T is D
      const int ones = key == 0 ? p.pack - kHalf * half : 0;
#pragma unroll
      for (int i = 0; i < kHalf; ++i) y[i] = i < ones ? -m.minus_d[st][kHalf * half + i] : y[i];
    }
#pragma unroll
    for (int i = 0; i < kHalf; i += 4) {
      const float4 d = d4[i >> 2];
      weigh2(x[i], x[i + 1], y[i], y[i + 1], d.x, d.y);
      weigh2(x[i + 2], x[i + 3], y[i + 2], y[i + 3], d.z, d.w);
    }
    if (edge) {
#pragma unroll
      for (int i = 0; i < kHalf; ++i) y[i] = i >= lo && i < hi ? y[i] : 0.f;
    }
    // the product with the dS before has ended when that block is free
    if (j > 0 && !warp_wait(smem_u32(&m.empty[before]), turn_before, deadline, ab)) return false;
    tc_fence_after();
    tmem_store_bf16<kHalf>(td, y, rows);
    tmem_wait_st();
    tc_fence_before();
    __syncwarp();
    if (lane_id() == 0) mbar_arrive(smem_u32(&m.ds_full));
    before = st;
    turn_before = turn;
    if (++st == C::kStages) {
      st = 0;
      turn ^= 1;
    }
  }
  if (s.total > 0) {
    if (!warp_wait(smem_u32(&m.out_full), 0, deadline, ab)) return false;
    tc_fence_after();
  }
  const size_t at = live ? static_cast<size_t>(w.k0 + key) * p.h_kv + kvh : 0;
  // the copies are not needed any more: their memory is the stage
  const bool odd = mha_store_sums<2, true>(p.dv + at * kMhaDv + 64 * half, sb + threadIdx.x * mha_stage_row<2>(),
                                           lane0 + C::kDv + 64 * half, 1.f, s.total > 0, live);
  mha_store_sums<DQK / 64>(p.dk + at * DQK + half * (DQK / 2),
                           sb + 256 * mha_stage_row<2>() + threadIdx.x * mha_stage_row<DQK / 64>(),
                           lane0 + C::kDk + half * (DQK / 2), p.scale, s.total > 0, live);
  bulk_wait();
  if (s.total > 0) {   // long past: the other warps' arrivals with their weights of the last block, and what they have found by then
    if (!warp_wait(smem_u32(&m.p_full), (s.total - 1) & 1, deadline, ab)) return false;
    const uint32_t keys = __ballot_sync(0xffffffffu, live && (odd || *reinterpret_cast<volatile int*>(&m.cleared)));
    if (keys != 0u) mha_restore_dv(p, keys, w, key, kvh, p.dv + at * kMhaDv + 64 * half, 64 * half);
  }
  return true;
}

template <int DQK>
__global__ void __launch_bounds__(MhaDkvShape<DQK>::kThreads, 1) dense_mha_dkv_kernel(
    const __grid_constant__ MhaBwdParams p) {
  using C = MhaDkvShape<DQK>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sbase = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  MhaDkvMisc& m = *reinterpret_cast<MhaDkvMisc*>(sbase + C::kMiscOff);
  const int warp = static_cast<int>(threadIdx.x >> 5);
  const uint32_t sb = smem_u32(sbase);
  int slot, kvh;
  mha_unit(static_cast<int>(blockIdx.x), p.slots, p.order, slot, kvh);

  if (threadIdx.x == 0) {
    for (int i = 0; i < 4; ++i) {
      mbar_init(smem_u32(&m.q_full[i]), 2);   // the copy and its rows' numbers
      mbar_init(smem_u32(&m.do_full[i]), 1);
      mbar_init(smem_u32(&m.empty[i]), 1);
    }
    mbar_init(smem_u32(&m.k_full), 1);
    mbar_init(smem_u32(&m.k_ready), 8);   // one arrival per row warp
    mbar_init(smem_u32(&m.s_full), 1);
    mbar_init(smem_u32(&m.s_free), 8);
    mbar_init(smem_u32(&m.p_full), 8);
    mbar_init(smem_u32(&m.p_free), 1);
    mbar_init(smem_u32(&m.t_full), 1);
    mbar_init(smem_u32(&m.t_free), 8);
    mbar_init(smem_u32(&m.ds_full), 8);
    mbar_init(smem_u32(&m.out_full), 1);
    mbar_init(smem_u32(&m.drain[0]), 1);
    mbar_init(smem_u32(&m.drain[1]), 1);
    m.abort_flag = 0;
    m.cleared = 0;
    m.prior_error = *reinterpret_cast<volatile int*>(&g_device_error);
    fence_mbar_init();
    prefetch_tmap(&p.map_q);
    prefetch_tmap(&p.map_do);
    prefetch_tmap(&p.map_k);
    prefetch_tmap(&p.map_v);
  }
  if (warp == 8) {
    tmem_alloc(smem_u32(&m.tmem_base), 512);
    tmem_relinquish();
  }
  if (warp == 9) {
    const MhaWork w = mha_find<true>(p.cu_q, p.cu_kv, p.batch, p.total_q, p.total_kv, slot, p.per);
    if (lane_id() == 0) m.work = w;
  }
  if (p.pack * p.tok_tile < C::kN) {
    // rows that no copy writes: a block's last ones, which weigh nothing, have to be numbers
    for (uint32_t i = threadIdx.x * 16; i < C::kStages * (C::kQBytes + C::kDoBytes); i += C::kThreads * 16)
      *reinterpret_cast<uint4*>(sbase + C::kQOff + i) = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = m.tmem_base;
  const MhaWork w = m.work;

  // rows of no sequence
  if (warp == 9 && w.end < p.total_kv && m.prior_error == 0) {
    mha_fill_rows(p.dk, static_cast<long long>(p.h_kv) * (DQK / 2), w.end, p.total_kv, 0u);
    mha_fill_rows(p.dv, static_cast<long long>(p.h_kv) * (kMhaDv / 2), w.end, p.total_kv, 0u);
  }
  // D is there, and dq too when this grid ends
  if (warp == 10) mha_other_grid();
  if (m.prior_error == 0 && w.k1 > w.k0) {
    const MhaQueries s(p, w);
    const int never = 0;
    if (warp < 8) {
      if (!mha_dkv_rows<DQK>(p, m, sb, tmem, w, s, kvh)) mha_bwd_raise(m, kErrMhaDkvRowsWait);
    } else if (s.total > 0) {
      if (warp == 10) {
        if (!mha_dkv_stats<DQK>(p, m, w, s, kvh)) mha_bwd_raise(m, kErrMhaDkvStatWait);
      } else if (warp == 8 || warp == 11) {
        if (!(warp == 8 ? mha_dkv_scores<DQK>(p, m, sb, s.total) : mha_dkv_sums<DQK>(p, m, sb, s.total)))
          mha_bwd_raise(m, kErrMhaDkvMmaWait);
        uint64_t* drain = &m.drain[warp == 8 ? 0 : 1];
        commit_to(elect_one(), drain);   // every MMA issued completes before TMEM is freed
        mbar_wait(smem_u32(drain), 0, global_timer_ns() + 100000000ull, &never);
      } else if (lane_id() == 0) {
        int fills = 0;
        if (!mha_dkv_load<DQK>(p, m, sb, w, s, kvh, fills)) mha_bwd_raise(m, kErrMhaDkvLoadWait);
        mha_other_grid();   // q_full takes the statistics' arrivals too
        // every copy issued has landed before the CTA exits
        const uint64_t dl = global_timer_ns() + 100000000ull;
        mbar_wait(smem_u32(&m.k_full), 0, dl, &never);
        for (int i = max(0, fills - C::kStages); i < fills; ++i) {
          mbar_wait(smem_u32(&m.q_full[i % C::kStages]), i / C::kStages & 1, dl, &never);
          mbar_wait(smem_u32(&m.do_full[i % C::kStages]), i / C::kStages & 1, dl, &never);
        }
      }
      __syncwarp();
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 8) tmem_dealloc(tmem, 512);
}

}  // namespace smla
