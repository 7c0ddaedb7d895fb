// Causal attention over whole prompts in the heads' own space (tcgen05 + TMA).
//
//   s_ij = scale q_i . k_j  over the keys j that query i sees,
//   lse_i = ln sum_j exp(s_ij),   out_i = sum_j exp(s_ij - lse_i) v_j
//
// A sequence's lq queries are the last lq of its lk positions: local query i sees keys
// 0 .. i + lk - lq.  h_q / h_kv query heads share a key and value head.
//
// A CTA takes NT tiles of 128 query rows against all keys that they see, 128 at a time.
// A tile's rows are (token, head) pairs: `pack` heads of one group side by side, so that
// a group of query heads reads its keys once and few tokens still fill a tile.
//
//   warps 0 .. 4 NT - 1  softmax, a thread per row: S from TMEM, running maximum and
//                        sum, P (bf16) back into the same TMEM columns; the epilogue
//   warp 4 NT            issues the MMAs (one thread, chosen by the whole warp):
//                          S_t = Q_t K_j^T   (both operands in shared memory)
//                          O_t += P_t V_j    (P_t in TMEM)
//   warp 4 NT + 1        one thread issues the TMA loads: Q once, then K and V through
//                        a ring of 16 KB units (K: 128 keys x 64 columns, V: 64 keys x
//                        128 columns)
//
// With two tiles the tensor core works on one while the softmax works on the other (a published
// way for this generation of tensor cores, as is the late rescaling below).  Where
// there are few tiles a CTA takes one, and a cluster of CTAs shares its keys out: each
// leaves its O, maximum and sum in its shared memory, and every CTA of the cluster joins a
// share of the rows from there.  O is
// rescaled only when a row's maximum has grown by more than 2^8: until then the weights
// are relative to the older maximum, which the sum and the LSE take into account exactly.
// P is rounded to bf16 for the product (2^-8 of each weight at most); scores, sums and O
// are fp32.
//
// What bounds it: the products (768 + 512 cycles a tile and block at 192 columns), as long
// as a softmax of one tile ends within the products of the other.  8192 tokens of 64 heads
// take 922 us, 1490 TFLOP/s or 79% of a large library product's rate; the rest is the
// pipeline's filling per tile and the diagonal's half-empty blocks.  Packed prompts of 3 to
// 2000 tokens take 150 us for 134 GFLOP: each CTA has some 5 to 15 blocks, and about 9000
// cycles go into starting (finding the tile, Q and K from memory) and the way out.  One
// token against 5001 keys is 14 us, of which the launch, the first loads and the join are
// all but 4.
//
// A weight of a key that is seen counts as above 0 where its value is not finite, even where it
// underflows: see mha_restore.
//
// Every wait is bounded; a CTA in which one runs out records an error, waits (bounded) for its
// copies and MMAs in flight, frees TMEM and returns.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cstdint>

#include "fp4_decode_kernel.cuh"
#include "fwd_kernel.cuh"
#include "norm_rope_kernel.cuh"
#include "ptx.cuh"

namespace smla {

constexpr int kMhaTile = 128;              // query rows of a tile, keys of a block
constexpr int kMhaDv = 128;
constexpr int kMhaMaxCluster = 16;
constexpr uint32_t kMhaUnit = 16384;       // bytes of a ring unit, and of 64 columns of a Q tile
constexpr int kMhaSpare = 4;               // rows of 64 that heads side by side leave unused at most (dk and dv mask as many)
constexpr float kMhaLazy = 8.f;            // log2 of the growth of a maximum that O is rescaled for

enum MhaErrCode : int {
  kErrMhaLoadWait = 0x701,
  kErrMhaMmaWait = 0x702,
  kErrMhaSoftmaxWait = 0x703,
};

// n / d for n < 2^31 as 2n m >> 32 + log: with log = log2 d (rounded up) and m = 2^(31 + log)
// / d + 1 (rounded down, below 2^32), m d is above 2^(31 + log) by d <= 2^log at most.
struct MhaDiv {
  unsigned m;
  int d, log;
  __device__ __forceinline__ int of(int n) const {
    return static_cast<int>(__umulhi(static_cast<unsigned>(n) << 1, m) >> log);
  }
};

// Heads (packs of them) whose tiles run side by side, the longest first: `near` at a time, so
// that what they read stays close, and behind the first `lead` all of the rest, so that the
// SMs end together.
struct MhaHeads {
  MhaDiv near, tiles, rest;   // tiles: of `near` heads; rest: heads behind the first `lead`
  int lead;
};

struct MhaFwdParams {
  CUtensorMap map_q, map_k, map_v;         // [token, head, d]: boxes 64 x pack x tok_tile, 64 x 1 x 128, 64 x 1 x 64
  const int32_t *cu_q, *cu_kv;             // [batch + 1], null for one dense sequence
  int batch, total_q, total_kv, h_q, group; // query heads per key head
  int pack, tok_tile;                      // a tile is tok_tile tokens x pack heads
  MhaDiv per;                              // tokens of a CTA (NT tiles)
  int slots;                               // tiles (of NT) per head pack that the grid has room for
  MhaHeads order;
  int cluster;                             // CTAs that share a tile's keys out (one tile a CTA; else 1)
  float scale_log2;
  const __nv_bfloat16* v;                  // row (t, h) at v + t v_tok + h v_head
  long long v_tok, v_head;
  __nv_bfloat16* out;                      // [total_q, h_q, 128]
  float* lse;                              // [total_q, h_q]
  int fill;                                // rows of no sequence: 1 out is zero, 2 lse is -inf
  unsigned long long timeout_ns;
};

// ------------------------------------------------------------------ sequences

// Offset b of `cu` within [0, total], whatever the array holds.
__device__ __forceinline__ int mha_offset(const int32_t* cu, int b, int total) {
  const int c = __ldg(cu + b);
  return c < 0 ? 0 : (c > total ? total : c);
}

// The rows of a sequence, and of one CTA's tile among those of one side.
struct MhaWork {
  int q0, q1, k0, k1;   // q1 <= q0: nothing to do
  int tile;             // from the sequence's first row
  int end;              // of the sequences' rows: the ones behind belong to none
};

// Tile `slot` of all sequences' tiles; q1 = k1 = 0 where there are not so many.  Up to 32
// sequences are taken from the longest to the shortest (of keys, whose tiles' work is the
// queries: by their queries), so that the SMs end together; more in their order.  A
// sequence's tiles come with the most work first: its last of queries, its first of keys.
// One warp, all lanes.  Every CTA goes through this before it can load anything, so it is
// kept short: with all tiles in the order of their work, by a search, 100 texts of 3 to 600
// tokens took 1.7 times as long and 15 of up to 2000 1.12 times; with every batch in its order
// the gradients of 9 texts of 122 to 2119 took 1.07 times as long.  It is CTAs times sequences
// all the same: 2000 texts of 1 to 30 tokens, 8 heads, take 2350 us, nearly all of it here.
template <bool KEYS>
__device__ __forceinline__ MhaWork mha_find(const int32_t* cu_q, const int32_t* cu_kv, int batch, int total_q,
                                            int total_kv, int slot, const MhaDiv& per) {
  MhaWork w = {0, 0, 0, 0, 0, KEYS ? total_kv : total_q};
  auto tiles = [&](int lq, int lk) { return KEYS ? (lk + kMhaTile - 1) >> 7 : per.of(lq + per.d - 1); };
  if (cu_q == nullptr) {
    const int n = tiles(total_q, total_kv);
    if (slot < n) {
      w.q1 = total_q;
      w.k1 = total_kv;
      w.tile = KEYS ? slot : n - 1 - slot;
    }
    return w;
  }
  const int lane = static_cast<int>(lane_id());
  int end = 0;
#pragma unroll 4
  for (int b = lane; b < batch; b += 32) end = max(end, KEYS ? mha_offset(cu_kv, b + 1, total_kv) : mha_offset(cu_q, b + 1, total_q));
  w.end = __reduce_max_sync(0xffffffffu, end);
  int4 x;          // a lane's sequence, its tiles, and the tiles before them
  int n, before;
  uint32_t past = 0u;
  for (int base = 0, all = 0; base < batch && past == 0u; base += 32) {
    x = make_int4(0, 0, 0, 0);
    if (const int b = base + lane; b < batch) {
      const int q0 = mha_offset(cu_q, b, total_q), k0 = mha_offset(cu_kv, b, total_kv);
      x = make_int4(q0, max(q0, mha_offset(cu_q, b + 1, total_q)), k0, max(k0, mha_offset(cu_kv, b + 1, total_kv)));
    }
    n = tiles(x.y - x.x, x.w - x.z);
    if (batch <= 32) {
      const int key = KEYS ? x.y - x.x : x.w - x.z;
      before = 0;
#pragma unroll 4
      for (int i = 0; i < batch; ++i) {
        const int other = __shfl_sync(0xffffffffu, key, i), m = __shfl_sync(0xffffffffu, n, i);
        before += other > key || (other == key && i < lane) ? m : 0;
      }
    } else {
      before = all + n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += y - all;
      }
      before -= n;
    }
    past = __ballot_sync(0xffffffffu, before <= slot && slot - before < n);
    all += __reduce_add_sync(0xffffffffu, n);
  }
  if (past != 0u) {
    const int at = __ffs(past) - 1;
    w.q0 = __shfl_sync(0xffffffffu, x.x, at);
    w.q1 = __shfl_sync(0xffffffffu, x.y, at);
    w.k0 = __shfl_sync(0xffffffffu, x.z, at);
    w.k1 = __shfl_sync(0xffffffffu, x.w, at);
    const int nth = slot - __shfl_sync(0xffffffffu, before, at);
    w.tile = KEYS ? nth : __shfl_sync(0xffffffffu, n, at) - 1 - nth;
  }
  return w;
}

// Rows first .. total - 1 of an output [total, words of 4 bytes] filled with a word, a share
// of them by each CTA of the grid.  One warp.
__device__ __forceinline__ void mha_fill_rows(void* out, long long words, int first, int total, uint32_t word) {
  for (long long r = static_cast<long long>(first) + blockIdx.x; r < total; r += gridDim.x)
    for (long long i = lane_id(); i < words; i += 32) static_cast<uint32_t*>(out)[r * words + i] = word;
}

// Unit -> tile and head (pack).
__device__ __forceinline__ void mha_unit(int unit, int slots, const MhaHeads& h, int& slot, int& head) {
  const int lead = h.lead * slots, turn = unit < lead ? h.tiles.of(unit) : 0;
  const int at = unit < lead ? unit - turn * h.tiles.d : unit - lead;
  slot = unit < lead ? h.near.of(at) : h.rest.of(at);
  head = unit < lead ? turn * h.near.d + at - slot * h.near.d : h.lead + at - slot * h.rest.d;
}

// ------------------------------------------------------------------ PTX

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void* tmap, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
      ::"r"(dst), "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

// Products are issued by a whole warp of which one thread is chosen: control and addresses
// are then the same for all of its threads, and the compiler keeps them in the registers
// that the instruction takes them from (one thread by itself needed 60 to 90 cycles more
// for each product, about as long as the product takes).
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t chosen;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(chosen));
  return chosen;
}

// A role's waits end at a deadline.  How long a tile takes has no bound, so the deadline is set
// anew with every block: what is bounded is a stay without progress, not the tile.  (Set by each
// wait in its own loop it took 4 % of packed prompts' time; so 0.3 %.)
//
// mbar_wait by all threads of a warp, with the same result for all.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, uint64_t deadline_ns,
                                          const volatile int* abort_flag) {
  while (!__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) {
    if (__any_sync(0xffffffffu, *abort_flag != 0 || global_timer_ns() > deadline_ns)) return false;
  }
  return true;
}
// For two barriers, of which the first has most likely been passed: their tries are under way together.
__device__ __forceinline__ bool warp_wait_both(uint32_t bar, uint32_t parity, uint32_t bar2, uint32_t parity2,
                                               uint64_t deadline_ns, const volatile int* abort_flag) {
  for (;;) {
    const bool one = mbar_try_wait(bar, parity), two = mbar_try_wait(bar2, parity2);
    if (__all_sync(0xffffffffu, one && two)) return true;
    if (__any_sync(0xffffffffu, *abort_flag != 0 || global_timer_ns() > deadline_ns)) return false;
  }
}

// D[tmem] (+)= A * B[smem] by the chosen thread, A in shared memory or (a row per lane, two
// bf16 values per column) in TMEM.
__device__ __forceinline__ void mma_ss(uint32_t chosen, uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
      ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(chosen) : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t chosen, uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
      ::"r"(d_tmem), "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(chosen) : "memory");
}
// Arrive on an mbarrier when every product that the chosen thread has issued so far has completed.
__device__ __forceinline__ void commit_to(uint32_t chosen, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}"
      ::"r"(smem_u32(bar)), "r"(chosen) : "memory");
}

// The descriptor of an operand `bytes` further on in shared memory (below 256 KB, so the
// address' field does not overflow): one addition, where forming it anew takes several
// and a block's products are issued by one thread.
__device__ __forceinline__ uint64_t desc_plus(uint64_t desc, uint32_t bytes) {
  uint32_t lo, hi;
  asm("mov.b64 {%0, %1}, %2;" : "=r"(lo), "=r"(hi) : "l"(desc));
  lo += bytes >> 4;
  asm("mov.b64 %0, {%1, %2};" : "=l"(desc) : "r"(lo), "r"(hi));
  return desc;
}

// This thread's TMEM lane, columns taddr .. taddr + N - 1, and the wait for them in one
// statement: nothing can be done with the registers before they hold the values.
__device__ __forceinline__ void tmem_load32(uint32_t taddr, float* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
      "%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31"
      "}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
        "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]),
        "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]),
        "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_load64(uint32_t taddr, float* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 {"
      "%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,"
      "%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,"
      "%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63"
      "}, [%64];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
        "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]),
        "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]),
        "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31]),
        "=f"(v[32]), "=f"(v[33]), "=f"(v[34]), "=f"(v[35]), "=f"(v[36]), "=f"(v[37]), "=f"(v[38]), "=f"(v[39]),
        "=f"(v[40]), "=f"(v[41]), "=f"(v[42]), "=f"(v[43]), "=f"(v[44]), "=f"(v[45]), "=f"(v[46]), "=f"(v[47]),
        "=f"(v[48]), "=f"(v[49]), "=f"(v[50]), "=f"(v[51]), "=f"(v[52]), "=f"(v[53]), "=f"(v[54]), "=f"(v[55]),
        "=f"(v[56]), "=f"(v[57]), "=f"(v[58]), "=f"(v[59]), "=f"(v[60]), "=f"(v[61]), "=f"(v[62]), "=f"(v[63])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_load128(uint32_t taddr, float* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x128.b32 {"
      "%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,"
      "%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,"
      "%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63,"
      "%64,%65,%66,%67,%68,%69,%70,%71,%72,%73,%74,%75,%76,%77,%78,%79,"
      "%80,%81,%82,%83,%84,%85,%86,%87,%88,%89,%90,%91,%92,%93,%94,%95,"
      "%96,%97,%98,%99,%100,%101,%102,%103,%104,%105,%106,%107,%108,%109,%110,%111,"
      "%112,%113,%114,%115,%116,%117,%118,%119,%120,%121,%122,%123,%124,%125,%126,%127"
      "}, [%128];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
        "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]),
        "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]),
        "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31]),
        "=f"(v[32]), "=f"(v[33]), "=f"(v[34]), "=f"(v[35]), "=f"(v[36]), "=f"(v[37]), "=f"(v[38]), "=f"(v[39]),
        "=f"(v[40]), "=f"(v[41]), "=f"(v[42]), "=f"(v[43]), "=f"(v[44]), "=f"(v[45]), "=f"(v[46]), "=f"(v[47]),
        "=f"(v[48]), "=f"(v[49]), "=f"(v[50]), "=f"(v[51]), "=f"(v[52]), "=f"(v[53]), "=f"(v[54]), "=f"(v[55]),
        "=f"(v[56]), "=f"(v[57]), "=f"(v[58]), "=f"(v[59]), "=f"(v[60]), "=f"(v[61]), "=f"(v[62]), "=f"(v[63]),
        "=f"(v[64]), "=f"(v[65]), "=f"(v[66]), "=f"(v[67]), "=f"(v[68]), "=f"(v[69]), "=f"(v[70]), "=f"(v[71]),
        "=f"(v[72]), "=f"(v[73]), "=f"(v[74]), "=f"(v[75]), "=f"(v[76]), "=f"(v[77]), "=f"(v[78]), "=f"(v[79]),
        "=f"(v[80]), "=f"(v[81]), "=f"(v[82]), "=f"(v[83]), "=f"(v[84]), "=f"(v[85]), "=f"(v[86]), "=f"(v[87]),
        "=f"(v[88]), "=f"(v[89]), "=f"(v[90]), "=f"(v[91]), "=f"(v[92]), "=f"(v[93]), "=f"(v[94]), "=f"(v[95]),
        "=f"(v[96]), "=f"(v[97]), "=f"(v[98]), "=f"(v[99]), "=f"(v[100]), "=f"(v[101]), "=f"(v[102]), "=f"(v[103]),
        "=f"(v[104]), "=f"(v[105]), "=f"(v[106]), "=f"(v[107]), "=f"(v[108]), "=f"(v[109]), "=f"(v[110]), "=f"(v[111]),
        "=f"(v[112]), "=f"(v[113]), "=f"(v[114]), "=f"(v[115]), "=f"(v[116]), "=f"(v[117]), "=f"(v[118]), "=f"(v[119]),
        "=f"(v[120]), "=f"(v[121]), "=f"(v[122]), "=f"(v[123]), "=f"(v[124]), "=f"(v[125]), "=f"(v[126]), "=f"(v[127])
      : "r"(taddr));
}

__device__ __forceinline__ void tmem_load48(uint32_t taddr, float* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
      "%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31"
      "}, [%48];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {"
      "%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47"
      "}, [%49];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
        "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]),
        "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]),
        "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31]),
        "=f"(v[32]), "=f"(v[33]), "=f"(v[34]), "=f"(v[35]), "=f"(v[36]), "=f"(v[37]), "=f"(v[38]), "=f"(v[39]),
        "=f"(v[40]), "=f"(v[41]), "=f"(v[42]), "=f"(v[43]), "=f"(v[44]), "=f"(v[45]), "=f"(v[46]), "=f"(v[47])
      : "r"(taddr), "r"(taddr + 32));
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const float* v) {
  const uint32_t* r = reinterpret_cast<const uint32_t*>(v);
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
               ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
// N (32, 48 or 64) columns of this thread's lane, all at once.
template <int N>
__device__ __forceinline__ void tmem_load(uint32_t taddr, float* v) {
  if constexpr (N == 64) tmem_load64(taddr, v);
  else if constexpr (N == 48) tmem_load48(taddr, v);
  else tmem_load32(taddr, v);
}
// N values rounded to bf16 into N / 2 columns, of the last two of which `keep` says what stays.
template <int N>
__device__ __forceinline__ void tmem_store_bf16(uint32_t taddr, const float* x, const uint32_t* keep = nullptr) {
  float pk[N / 2];
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    const uint32_t v = pack_bf16x2(x[2 * i], x[2 * i + 1]);
    pk[i] = __uint_as_float(keep != nullptr && i >= N / 2 - 2 ? v & keep[i - (N / 2 - 2)] : v);
  }
#pragma unroll
  for (int i = 0; i < N / 32; ++i) tmem_st16(taddr + 16 * i, pk + 16 * i);
  if constexpr (N % 32 != 0) tmem_st8(taddr + N / 2 - 8, pk + N / 2 - 8);
}

__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}

// `bytes` (a multiple of 16) of this CTA's shared memory to global memory, in the background;
// the thread's copies so far have ended.
__device__ __forceinline__ void bulk_store(void* to, uint32_t from, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;"
               ::"l"(reinterpret_cast<uint64_t>(to)), "r"(from), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bulk_wait() {
  asm volatile("cp.async.bulk.commit_group;\n\tcp.async.bulk.wait_group 0;" ::: "memory");
}

// Turns `odd` into NaN where one of 32 values is not finite (0 times it is a NaN).
__device__ __forceinline__ void mha_odd32(const float* x, float (&odd)[2]) {
#pragma unroll
  for (int k = 0; k < 32; k += 2)
    asm("{\n\t.reg .b64 px, pz, po;\n\t"
        "mov.b64 px, {%2, %3};\n\t"
        "mov.b64 pz, {%4, %4};\n\t"
        "mov.b64 po, {%0, %1};\n\t"
        "fma.rn.f32x2 po, px, pz, po;\n\t"
        "mov.b64 {%0, %1}, po;\n\t}"
        : "+f"(odd[0]), "+f"(odd[1])
        : "f"(x[k]), "f"(x[k + 1]), "f"(0.f));
}
__device__ __forceinline__ bool mha_finite(float x) { return fabsf(x) <= 3.402823466e38f; }
// Not 0 where one of eight bf16 values is not finite: the sign bit's place is carried into
// where the exponent is all ones.
__device__ __forceinline__ uint32_t odd_halves(const uint4& x) {
  return (((x.x & 0x7fff7fffu) + 0x00800080u) | ((x.y & 0x7fff7fffu) + 0x00800080u) | ((x.z & 0x7fff7fffu) + 0x00800080u) |
          ((x.w & 0x7fff7fffu) + 0x00800080u)) & 0x80008000u;
}

// Adds to acc, for this lane's 8 of 8 LANES columns (lane % LANES), what is not finite in rows
// from .. end - 1 at `rows`, `step` elements apart; the rows are dealt out over the warp's
// groups of LANES lanes.
template <int LANES>
__device__ __forceinline__ void mha_take_odd(const __nv_bfloat16* rows, long long step, int from, int end, float (&acc)[8]) {
  const int lane = static_cast<int>(lane_id());
#pragma unroll 4
  for (int r = from + lane / LANES; r < end; r += 32 / LANES) {
    const uint4 x = __ldg(reinterpret_cast<const uint4*>(rows + r * step) + lane % LANES);
    if (odd_halves(x) == 0u) continue;
    float y[8];
    unpack8(x, y);
#pragma unroll
    for (int k = 0; k < 8; ++k) acc[k] += mha_finite(y[k]) ? 0.f : y[k];
  }
}
// The groups' shares of acc together.
template <int LANES>
__device__ __forceinline__ void mha_sum_odd(const float (&acc)[8], float (&sum)[8]) {
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    sum[k] = acc[k];
#pragma unroll
    for (int o = LANES; o < 32; o <<= 1) sum[k] += __shfl_xor_sync(0xffffffffu, sum[k], o);
  }
}

// 32 N columns of this thread's TMEM lane times `f` as a bf16 row (zeros where there are no
// sums), put together in its own part of shared memory (`stage`) and copied from there:
// stored by the threads themselves, 32 rows' pieces of 16 bytes at a time, a tile's rows
// take about 2 us of the CTA's time.  Rows of the stage are 64 N + 16 bytes apart:
// neighbours are in other banks.  `sums` is the same for a whole warp.  Whether a value is not
// finite, where ODD asks for it.
template <int N, bool ODD = false>
__device__ __forceinline__ bool mha_store_sums(__nv_bfloat16* row, uint32_t stage, uint32_t taddr, float f, bool sums,
                                               bool live) {
  float odd[2] = {0.f, 0.f};
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float x[32];
    if (sums) tmem_load32(taddr + 32 * i, x);
#pragma unroll
    for (int k = 0; k < 32; ++k) x[k] = sums ? x[k] * f : 0.f;
    if (ODD) mha_odd32(x, odd);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint4 v = pack8(x + 8 * k);
      st_shared_v4(stage + 64 * i + 16 * k, v.x, v.y, v.z, v.w);
    }
  }
  fence_proxy_async_smem();
  if (live) bulk_store(row, stage, 64 * N);
  return odd[0] + odd[1] != 0.f;
}
template <int N>
__device__ constexpr uint32_t mha_stage_row() {
  return 64 * N + 16;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// (a0, a1) * b + (c0, c1) and (a0, a1) * ((b0, b1) + (c0, c1)), packed.
__device__ __forceinline__ void scale_shift2(float& a0, float& a1, float b, float c0, float c1) {
  asm("{\n\t.reg .b64 pa, pb, pc;\n\t"
      "mov.b64 pa, {%0, %1};\n\t"
      "mov.b64 pb, {%2, %2};\n\t"
      "mov.b64 pc, {%3, %4};\n\t"
      "fma.rn.f32x2 pa, pa, pb, pc;\n\t"
      "mov.b64 {%0, %1}, pa;\n\t}"
      : "+f"(a0), "+f"(a1)
      : "f"(b), "f"(c0), "f"(c1));
}
__device__ __forceinline__ void weigh2(float a0, float a1, float& b0, float& b1, float c0, float c1) {
  asm("{\n\t.reg .b64 pa, pb, pc;\n\t"
      "mov.b64 pa, {%2, %3};\n\t"
      "mov.b64 pb, {%0, %1};\n\t"
      "mov.b64 pc, {%4, %5};\n\t"
      "add.rn.f32x2 pb, pb, pc;\n\t"
      "mul.rn.f32x2 pb, pa, pb;\n\t"
      "mov.b64 {%0, %1}, pb;\n\t}"
      : "+f"(b0), "+f"(b1)
      : "f"(a0), "f"(a1), "f"(c0), "f"(c1));
}

__device__ __forceinline__ void add2(float& a0, float& a1, float b0, float b1) {
  asm("{\n\t.reg .b64 pa, pb;\n\t"
      "mov.b64 pa, {%0, %1};\n\t"
      "mov.b64 pb, {%2, %3};\n\t"
      "add.rn.f32x2 pa, pa, pb;\n\t"
      "mov.b64 {%0, %1}, pa;\n\t}"
      : "+f"(a0), "+f"(a1)
      : "f"(b0), "f"(b1));
}

// ------------------------------------------------------------------ forward

constexpr int kMhaMaxUnits = 12;
constexpr int kMhaFree = 4;   // a block's release is told on one of so many barriers in turn

struct __align__(16) MhaMisc {
  uint64_t q_full[2], full[kMhaMaxUnits], k_free[kMhaFree], v_free[kMhaFree], s_full[2], p_full[2], o_full[2], o_step, drain;
  uint32_t tmem_base;
  int abort_flag;
  int prior_error;
  int cleared;   // values of V that are not finite were taken out of a block that some rows do not see all of
  MhaWork work;
  float2 part[kMhaTile];   // a row's maximum (in powers of two) and sum over this CTA's keys
};
constexpr int kMhaPartRow = kMhaDv + 4;   // floats of a row that is joined; neighbours in other banks

// Shared memory: Q (NT tiles), then the ring.
template <int DQK, int NT>
struct MhaFwdShape {
  static constexpr int kSub = DQK / 64;                        // 64-column units of a K block or Q tile
  static constexpr uint32_t kQBytes = NT * kSub * kMhaUnit;
  static constexpr int kFree = kMaxSmem - 1024 - static_cast<int>(sizeof(MhaMisc)) - static_cast<int>(kQBytes);
  static constexpr int kFit = kFree / static_cast<int>(kMhaUnit);
  static constexpr int kUnits = kFit < kMhaMaxUnits ? kFit : kMhaMaxUnits;
  static constexpr uint32_t kMiscOff = kQBytes + kUnits * kMhaUnit;
  static constexpr int kBytes = static_cast<int>(kMiscOff) + static_cast<int>(sizeof(MhaMisc)) + 1024;
  static constexpr int kAhead = NT == 1 ? 2 : 1;               // key blocks whose scores are ahead of the weights
  static constexpr int kThreads = NT * 128 + 64;               // two tiles: ptxas leaves 168 registers each, which spills 84 bytes
  static constexpr uint32_t kO = 256;                          // columns of TMEM: two S of 128 each, then O
  static_assert(kUnits >= kSub + 4, "a K block and two V blocks");
  // The barrier that told of block j's release tells of block j + kMhaFree's next, and must not before the first has been
  // waited for.  The loads wait for releases in order, so it is enough that the last unit of K (V) j + kMhaFree has no
  // place in the ring while K (V) j is there: between the two are kMhaFree - 1 blocks of the other kind at least.
  static_assert((kMhaFree + 1) * kSub + (kMhaFree - 1) * 2 > kUnits && (kMhaFree + 1) * 2 + (kMhaFree - 1) * kSub > kUnits,
                "releases told apart");
  static_assert(kBytes <= kMaxSmem, "shared memory");
  static_assert(kUnits * kMhaUnit >= kMhaTile * kMhaPartRow * 4, "rows that are joined");
};

// What one CTA does: keys' blocks of each of its tiles.
template <int NT>
struct MhaSpan {
  int t0[NT];      // first token of the tile, in the sequence
  int blocks[NT];  // blocks of 128 keys that its rows see (of which this CTA takes them)
  int from;        // the first of them
  int most;
  __device__ __forceinline__ MhaSpan(const MhaFwdParams& p, const MhaWork& w, int rank) {
    const int lq = w.q1 - w.q0, lk = w.k1 - w.k0;
    most = 0;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      t0[t] = (w.tile * NT + t) * p.tok_tile;
      const int last = min(t0[t] + p.tok_tile, lq) - 1;
      const int sees = t0[t] < lq ? last + lk - lq + 1 : 0;   // of its last row
      blocks[t] = sees > 0 ? (sees + kMhaTile - 1) / kMhaTile : 0;
      most = max(most, blocks[t]);
    }
    from = 0;
    if (NT == 1 && p.cluster > 1) {
      from = static_cast<int>(static_cast<long long>(most) * rank / p.cluster);
      most = blocks[0] = static_cast<int>(static_cast<long long>(most) * (rank + 1) / p.cluster) - from;
    }
  }
};

__device__ __forceinline__ void mha_raise(MhaMisc& m, int code) {
  *reinterpret_cast<volatile int*>(&m.abort_flag) = 1;
  atomicCAS(&g_device_error, 0, code);
}

// A position in the ring: its unit and the parity of that unit's fill.
template <int UNITS>
struct MhaRing {
  uint32_t at = 0, turn = 0;
  __device__ __forceinline__ void next() { skip(1); }
  __device__ __forceinline__ void skip(uint32_t n) {
    at += n;
    if (at >= UNITS) {
      at -= UNITS;
      turn ^= 1u;
    }
  }
};

// The blocks in the order of their use: K 0, V 0, K 1, V 1, ...; with `ahead` 2: K 0, K 1,
// V 0, K 2, V 1, ...
struct MhaOrder {
  bool value = false;   // of V
  int block = 0;
  __device__ __forceinline__ void next(int ahead, int most) {
    if (!value && ahead == 2 && block == 0 && most > 1) block = 1;
    else if (!value) {
      value = true;
      block = max(0, block + 1 - ahead);
    } else if (block + ahead < most) {
      value = false;
      block += ahead;
    } else ++block;
  }
};

template <int DQK, int NT>
__device__ __forceinline__ bool mha_load(const MhaFwdParams& p, MhaMisc& m, uint32_t sb, const MhaWork& w,
                                         const MhaSpan<NT>& s, int pack0, int kvh, uint32_t& fills) {
  using C = MhaFwdShape<DQK, NT>;
  const volatile int* ab = &m.abort_flag;
  uint64_t deadline = global_timer_ns() + p.timeout_ns;
  auto load_q = [&](int t) {
    const uint32_t bar = smem_u32(&m.q_full[t]);
    const uint32_t bytes = static_cast<uint32_t>(p.pack * p.tok_tile) * 128u;
    mbar_arrive_expect_tx(bar, C::kSub * bytes);
    for (int c = 0; c < C::kSub; ++c)
      tma_load_3d(sb + (t * C::kSub + c) * kMhaUnit, &p.map_q, 64 * c, pack0, w.q0 + s.t0[t], bar);
  };
  if (s.blocks[0] > 0) load_q(0);
  MhaRing<C::kUnits> r;
  MhaOrder now, old;       // the block that is loaded, the one whose units come free next
  int old_left = 0;        // units of `old` that are free and not yet filled
  for (int n = 0; n < 2 * s.most; ++n) {
    deadline = global_timer_ns() + p.timeout_ns;
    for (int c = 0; c < (now.value ? 2 : C::kSub); ++c) {
      if (fills >= static_cast<uint32_t>(C::kUnits)) {
        if (old_left == 0) {
          uint64_t* bar = old.value ? &m.v_free[old.block % kMhaFree] : &m.k_free[old.block % kMhaFree];
          if (!mbar_wait(smem_u32(bar), old.block / kMhaFree & 1, deadline, ab)) return false;
          old_left = old.value ? 2 : C::kSub;
          old.next(C::kAhead, s.most);
        }
        --old_left;
      }
      const uint32_t bar = smem_u32(&m.full[r.at]), dst = sb + C::kQBytes + r.at * kMhaUnit;
      const int row = w.k0 + (s.from + now.block) * kMhaTile;
      mbar_arrive_expect_tx(bar, kMhaUnit);
      if (now.value) {
        tma_load_3d(dst, &p.map_v, 0, kvh, row + 64 * c, bar);
        tma_load_3d(dst + kMhaUnit / 2, &p.map_v, 64, kvh, row + 64 * c, bar);
      } else {
        tma_load_3d(dst, &p.map_k, 64 * c, kvh, row, bar);
      }
      ++fills;
      r.next();
    }
    if (n == 0 && NT > 1 && s.blocks[NT - 1] > 0) load_q(NT - 1);
    now.next(C::kAhead, s.most);
  }
  return true;
}

template <int DQK, int NT>
__device__ __forceinline__ bool mha_mma(const MhaFwdParams& p, MhaMisc& m, uint32_t sb,
                                        const MhaSpan<NT>& s) {
  using C = MhaFwdShape<DQK, NT>;
  constexpr uint32_t kIdescS = idesc_bf16_f32(kMhaTile, kMhaTile, false, false);
  constexpr uint32_t kIdescO = idesc_bf16_f32(kMhaTile, kMhaDv, false, true);
  const volatile int* ab = &m.abort_flag;
  uint64_t deadline = global_timer_ns() + p.timeout_ns;
  const uint32_t chosen = elect_one();
  auto commit = [&](uint64_t* bar) { commit_to(chosen, bar); };
  const uint64_t q_desc = smem_desc(sb, 16, 1024, SWZ_128B), k_desc = smem_desc(sb + C::kQBytes, 16, 1024, SWZ_128B),
                 v_desc = smem_desc(sb + C::kQBytes, kMhaUnit / 2, 1024, SWZ_128B);
  // TMEM is taken whole, so its columns start at 0
  MhaRing<C::kUnits> r;   // the units in the order of their use
  auto wait_unit = [&](const MhaRing<C::kUnits>& u) -> bool {
    return warp_wait(smem_u32(&m.full[u.at]), u.turn, deadline, ab);
  };
  // S (columns `to`, barrier `bar`) = Q_t K^T of block j at `u`; `first`: its units have not been waited for, `last`:
  // they are free behind it
  auto scores = [&](int t, uint32_t to, uint64_t* bar, int j, MhaRing<C::kUnits> u, bool first, bool last) -> bool {
#pragma unroll
    for (int c = 0; c < C::kSub; ++c) {
      if (first && !wait_unit(u)) return false;
      const uint64_t a = desc_plus(q_desc, (t * C::kSub + c) * kMhaUnit), b = desc_plus(k_desc, u.at * kMhaUnit);
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
        mma_ss(chosen, to, desc_plus(a, kk * 32), desc_plus(b, kk * 32), kIdescS, c + kk > 0 ? 1u : 0u);
      u.next();
    }
    commit(bar);
    if (last) commit(&m.k_free[j % kMhaFree]);
    return true;
  };
  // O_t += P (columns `from`) V of block j at `u`
  auto weighted = [&](int t, uint32_t from, int j, MhaRing<C::kUnits> u, bool first, bool last) -> bool {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      if (first && !wait_unit(u)) return false;
      const uint64_t b = desc_plus(v_desc, u.at * kMhaUnit);
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
        mma_ts(chosen, C::kO + t * kMhaDv, from + 8 * (4 * c + kk), desc_plus(b, kk * 2048), kIdescO,
                     j + c + kk > 0 ? 1u : 0u);
      u.next();
    }
    if (last) commit(&m.v_free[j % kMhaFree]);
    return true;
  };
  if constexpr (NT == 1) {
    // two S in turn: block j + 2's scores follow block j's weights, so that a block's are there when the softmax has done
    // the one before
    if (!warp_wait(smem_u32(&m.q_full[0]), 0, deadline, ab)) return false;
    for (int j = 0; j < 2 && j < s.most; ++j) {
      if (!scores(0, kMhaTile * j, &m.s_full[j], j, r, true, true)) return false;
      r.skip(C::kSub);
    }
    for (int j = 0; j < s.most; ++j) {
      deadline = global_timer_ns() + p.timeout_ns;
      const int buf = j & 1;
      if (!warp_wait(smem_u32(&m.p_full[buf]), j >> 1 & 1, deadline, ab)) return false;
      tc_fence_after();
      if (!weighted(0, kMhaTile * buf, j, r, true, true)) return false;
      commit(j + 1 < s.most ? &m.o_step : &m.o_full[0]);
      r.skip(2);
      if (j + 2 < s.most) {
        if (!scores(0, kMhaTile * buf, &m.s_full[buf], j + 2, r, true, true)) return false;
        r.skip(C::kSub);
      }
    }
  } else {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      if (s.blocks[t] == 0) continue;
      if (!warp_wait(smem_u32(&m.q_full[t]), 0, deadline, ab)) return false;
      const bool alone = s.blocks[1 - t] == 0;
      if (!scores(t, kMhaTile * t, &m.s_full[t], 0, r, t == 0 || alone, t == 1 || alone)) return false;
    }
    r.skip(C::kSub);
    for (int j = 0; j < s.most; ++j) {
      deadline = global_timer_ns() + p.timeout_ns;
      MhaRing<C::kUnits> rk = r;                 // block j's V, then block j + 1's K
      rk.skip(2);
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        if (j >= s.blocks[t]) continue;
        const bool alone = j >= s.blocks[1 - t], alone_k = j + 1 >= s.blocks[1 - t];
        if (!warp_wait(smem_u32(&m.p_full[t]), j & 1, deadline, ab)) return false;
        tc_fence_after();
        if (!weighted(t, kMhaTile * t, j, r, t == 0 || alone, t == 1 || alone)) return false;
        if (j + 1 == s.blocks[t]) commit(&m.o_full[t]);
        else if (!scores(t, kMhaTile * t, &m.s_full[t], j + 1, rk, t == 0 || alone_k, t == 1 || alone_k)) return false;
      }
      r = rk;
      if (j + 1 < s.most) r.skip(C::kSub);
    }
  }
  return true;
}

// A hidden key's weight is 0, but 0 times an infinity or a NaN is a NaN: before a product
// with a block that some rows do not see all of, values that are not finite are taken
// out of it.  Each of N threads (the CTA's first, or the N behind them) looks over its share
// of `bytes`, a multiple of 2 KB, and sets `found` where there are some, before it takes them
// out: whoever meets zeros in their place finds it set.
template <int N>
__device__ __forceinline__ void mha_clear(uint32_t tile, uint32_t bytes, int* found = nullptr) {
  uint32_t seen = 0;
  for (uint32_t at = threadIdx.x % N * 16; at < bytes; at += N * 16) {
    uint32_t x[4];
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]) : "r"(tile + at));
    // the sign bit's place is carried into where the exponent is all ones
#pragma unroll
    for (int i = 0; i < 4; ++i) seen |= (x[i] & 0x7fff7fffu) + 0x00800080u;
  }
  if ((seen & 0x80008000u) == 0u) return;
  if (found != nullptr) {
    *reinterpret_cast<volatile int*>(found) = 1;
    __threadfence_block();
  }
  for (uint32_t at = threadIdx.x % N * 16; at < bytes; at += N * 16) {
    uint32_t x[4];
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]) : "r"(tile + at));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if ((x[i] & 0x7f80u) == 0x7f80u) x[i] &= 0xffff0000u;
      if ((x[i] & 0x7f800000u) == 0x7f800000u) x[i] &= 0xffffu;
    }
    st_shared_v4(tile + at, x[0], x[1], x[2], x[3]);
  }
  fence_proxy_async_smem();
}

// A weight is above 0, however small: a value that is not finite makes its column of each row
// that sees its key infinite, and two of them that do not agree, or a NaN, make it NaN.  The
// products have this otherwise where the weight underflows (0 times an infinity), where a sum
// of weights relative to an older maximum does, and where the value was taken out.  So the
// columns of the rows of `asked` become the sums of what is not finite among keys first .. end - 1
// (a lane's end is its row's; it does not fall from lane to lane).  One warp, a row per lane;
// `part`, where it is given, takes the sums in place of `out`.
__device__ __forceinline__ void mha_restore(uint32_t asked, const __nv_bfloat16* values, long long step, int first, int end,
                                            __nv_bfloat16* out, float* part) {
  const int col = static_cast<int>(lane_id()) % 16 * 8;
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  __syncwarp();   // the rows' own threads have written them
  for (; asked != 0u; asked &= asked - 1) {
    const int row = __ffs(asked) - 1, upto = __shfl_sync(0xffffffffu, end, row);
    __nv_bfloat16* o = reinterpret_cast<__nv_bfloat16*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(out), row));
    float* q = reinterpret_cast<float*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(part), row));
    mha_take_odd<16>(values, step, first, upto, acc);
    first = max(first, upto);
    float sum[8];
    mha_sum_odd<16>(acc, sum);
    if (lane_id() < 16) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (sum[k] == 0.f) continue;
        if (q != nullptr) q[col + k] = sum[k];
        else o[col + k] = __float2bfloat16_rn(sum[k]);
      }
    }
  }
}

// One thread per row of tile t.
template <int DQK, int NT>
__device__ __forceinline__ bool mha_softmax(const MhaFwdParams& p, MhaMisc& m, uint8_t* sbase, uint32_t sb, uint32_t tmem,
                                            const MhaWork& w, const MhaSpan<NT>& s, int pack0, int t) {
  using C = MhaFwdShape<DQK, NT>;
  const volatile int* ab = &m.abort_flag;
  uint64_t deadline = global_timer_ns() + p.timeout_ns;
  const int row = static_cast<int>(threadIdx.x) & 127;
  const int lq = w.q1 - w.q0, lk = w.k1 - w.k0;
  const int tok = s.t0[t] + row / p.pack;
  const bool live = row < p.pack * p.tok_tile && tok < lq;
  const int blocks = s.blocks[t];
  const int whole = max(0, s.t0[t] + lk - lq + 1) / kMhaTile - s.from;   // blocks that every row sees all of
  const uint32_t quarter = static_cast<uint32_t>((row >> 5) * 32) << 16;
  const uint32_t to = tmem + quarter + C::kO + t * kMhaDv;
  const float c = p.scale_log2;
  float top = -INFINITY, sum = 0.f;   // the maximum that the weights are relative to, their sum
  for (int j = 0; j < blocks; ++j) {
    deadline = global_timer_ns() + p.timeout_ns;
    const int buf = NT == 1 ? j & 1 : t, par = NT == 1 ? j >> 1 & 1 : j & 1;   // the S that the block's scores are in
    const uint32_t ts = tmem + quarter + buf * kMhaTile;
    if (j >= whole) {
      for (int i = 0; i < 2; ++i) {   // the block's V: units behind those of the K before it and of the V before it
        const uint32_t n = static_cast<uint32_t>(min(j + C::kAhead, s.most) * C::kSub + 2 * j + i);
        if (!warp_wait(smem_u32(&m.full[n % C::kUnits]), n / C::kUnits & 1u, deadline, ab)) return false;
        mha_clear<128>(sb + C::kQBytes + n % C::kUnits * kMhaUnit, kMhaUnit, &m.cleared);
      }
    }
    if (!warp_wait(smem_u32(&m.s_full[buf]), par, deadline, ab)) return false;
    tc_fence_after();
    float v[kMhaTile];
    tmem_load128(ts, v);
    if (j >= whole) {
      const int sees = tok + lk - lq + 1 - (s.from + j) * kMhaTile;
#pragma unroll
      for (int i = 0; i < kMhaTile; ++i) v[i] = i < sees ? v[i] : -INFINITY;
    }
    float mx[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
    for (int i = 4; i < kMhaTile - 4; i += 8) {
#pragma unroll
      for (int k = 0; k < 4; ++k) mx[k] = max3(mx[k], v[i + 2 * k], v[i + 2 * k + 1]);
    }
    const float now = max3(max3(max3(mx[0], mx[1], mx[2]), max3(mx[3], v[124], v[125]), v[126]), v[127], v[127]);
    const bool grown = (now - top) * c > kMhaLazy;
    if (__any_sync(0xffffffffu, grown)) {
      // O is this warp's to change once the product before has ended: with two tiles the block's scores came after it
      if (NT == 1 && j > 0) {
        if (!warp_wait(smem_u32(&m.o_step), (j - 1) & 1, deadline, ab)) return false;
        tc_fence_after();
      }
      const float f = grown ? fast_exp2((top - now) * c) : 1.f;
      if (grown) top = now;
      sum *= f;
      if (j > 0) {
#pragma unroll
        for (int i = 0; i < kMhaDv / 32; ++i) {
          float o[32];
          tmem_load32(to + 32 * i, o);
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] *= f;
          tmem_st16(to + 32 * i, o);
          tmem_st16(to + 32 * i + 16, o + 16);
        }
      }
    }
    const float shift = top == -INFINITY ? 0.f : -top * c;
    float add[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < kMhaTile; i += 32) {
      float pk[16];
#pragma unroll
      for (int k = 0; k < 32; k += 2) {
        float &a = v[i + k], &b = v[i + k + 1];
        scale_shift2(a, b, c, shift, shift);
        a = fast_exp2(a);
        b = fast_exp2(b);
        add2(add[k & 2], add[(k & 2) + 1], a, b);
        pk[k >> 1] = __uint_as_float(pack_bf16x2(a, b));
      }
      tmem_st16(ts + (i >> 1), pk);
    }
    tmem_wait_st();
    tc_fence_before();
    __syncwarp();
    if (lane_id() == 0) mbar_arrive(smem_u32(&m.p_full[buf]));
    add2(add[0], add[1], add[2], add[3]);
    sum += add[0] + add[1];
  }
  const size_t at = live ? static_cast<size_t>(w.q0 + tok) * p.h_q + pack0 + row % p.pack : 0;
  __nv_bfloat16* o = p.out + at * kMhaDv;
  if (blocks > 0) {
    if (!warp_wait(smem_u32(&m.o_full[t]), 0, deadline, ab)) return false;
    tc_fence_after();
  }
  const bool join = NT == 1 && p.cluster > 1;
  if (live && !join) p.lse[at] = sum == 0.f ? -INFINITY : (top * c + log2f(sum)) * 0.6931471805599453f;
  // the products and loads are done: the ring's memory holds the rows that are joined
  float* part = reinterpret_cast<float*>(sbase + C::kQBytes) + row * kMhaPartRow;
  bool odd = false;   // a sum is not finite
  if (join) {
    m.part[row] = make_float2(sum == 0.f ? -INFINITY : top * c, sum);
    float odds[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < kMhaDv / 32; ++i) {
      float x[32];
      if (blocks > 0) {
        tmem_load32(to + 32 * i, x);
        mha_odd32(x, odds);
      }
#pragma unroll
      for (int k = 0; k < 32; k += 4)
        *reinterpret_cast<float4*>(part + 32 * i + k) =
            sum == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(x[k], x[k + 1], x[k + 2], x[k + 3]);
    }
    odd = odds[0] + odds[1] != 0.f;
  } else {
    // the tile's Q is not needed any more: its memory is the stage, at 128 columns for half a row at a time
    constexpr int kPieces = C::kSub * kMhaUnit >= kMhaTile * mha_stage_row<4>() ? 1 : 2, kCols = kMhaDv / kPieces;
    const uint32_t stage = sb + t * C::kSub * kMhaUnit + row * mha_stage_row<kCols / 32>();
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      odd |= mha_store_sums<kCols / 32, true>(o + kCols * i, stage, to + kCols * i, inv, blocks > 0, live);
      bulk_wait();
    }
  }
  if (blocks > 0) {   // long past: the other warps' arrivals with their weights of the last block, and what they have found by then
    const int last = blocks - 1;
    if (!warp_wait(smem_u32(&m.p_full[NT == 1 ? last & 1 : t]), NT == 1 ? last >> 1 & 1 : last & 1, deadline, ab)) return false;
    const bool ask = live && mha_finite(sum) && (odd || *reinterpret_cast<volatile int*>(&m.cleared));
    const uint32_t rows = __ballot_sync(0xffffffffu, ask);
    if (rows != 0u)
      mha_restore(rows, p.v + w.k0 * p.v_tok + pack0 / p.group * p.v_head, p.v_tok, s.from * kMhaTile,
                  min(tok + lk - lq + 1, (s.from + blocks) * kMhaTile), o, join ? part : nullptr);
  }
  return true;
}

// The parts that a cluster's CTAs have left of a tile, joined in the order of their keys:
// W columns a thread.  Reads of another CTA's memory take about a microsecond, so there
// should be few steps of them: many columns a thread for many rows, few for few.
template <int DQK, int W>
__device__ __forceinline__ void mha_join(const MhaFwdParams& p, MhaMisc& m, uint32_t sb, const MhaWork& w, int t0, int rows,
                                         int pack0, int rank) {
  using C = MhaFwdShape<DQK, 1>;
  constexpr int kPerRow = kMhaDv / W, kRows = 128 / kPerRow;
  const int col = static_cast<int>(threadIdx.x) % kPerRow * W;
  for (int row = rank * kRows + static_cast<int>(threadIdx.x) / kPerRow; row < rows; row += kRows * p.cluster) {
    const uint32_t stat = smem_u32(&m.part[row]), at = sb + C::kQBytes + static_cast<uint32_t>(row * kMhaPartRow + col) * 4u;
    float top = -INFINITY, sum = 0.f, acc[W];
#pragma unroll
    for (int i = 0; i < kMhaMaxCluster; ++i)
      if (i < p.cluster) top = fmaxf(top, ld_cluster_f(cluster_addr(stat, i)));
#pragma unroll
    for (int k = 0; k < W; ++k) acc[k] = 0.f;
#pragma unroll W > 4 ? 2 : 8
    for (int i = 0; i < p.cluster; ++i) {
      const uint32_t peer = cluster_addr(stat, i), from = cluster_addr(at, i);
      const float own = ld_cluster_f(peer), own_sum = ld_cluster_f(peer + 4);
      float4 x[W / 4];
#pragma unroll
      for (int k = 0; k < W / 4; ++k) x[k] = ld_cluster_f4(from + 16 * k);
      const float f = own_sum == 0.f ? 0.f : fast_exp2(own - top);   // a sum that is NaN passes it on
      sum += f * own_sum;
      // a part whose weight is 0: what is not finite counts even so
      const bool none = f == 0.f;
      const float g = none ? 1.f : f;
      auto add = [&](float& to, float y) { to += g * (none && mha_finite(y) ? 0.f : y); };
#pragma unroll
      for (int k = 0; k < W / 4; ++k) {
        add(acc[4 * k], x[k].x);
        add(acc[4 * k + 1], x[k].y);
        add(acc[4 * k + 2], x[k].z);
        add(acc[4 * k + 3], x[k].w);
      }
    }
    const float inv = sum == 0.f ? 1.f : 1.f / sum;   // without weights acc has zeros, and what is not finite
    const size_t out = static_cast<size_t>(w.q0 + t0 + row / p.pack) * p.h_q + pack0 + row % p.pack;
    uint2* o = reinterpret_cast<uint2*>(p.out + out * kMhaDv + col);
#pragma unroll
    for (int k = 0; k < W / 4; ++k)
      o[k] = make_uint2(pack_bf16x2(acc[4 * k] * inv, acc[4 * k + 1] * inv),
                        pack_bf16x2(acc[4 * k + 2] * inv, acc[4 * k + 3] * inv));
    if (col == 0)
      p.lse[out] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
  }
}

template <int DQK, int NT>
__global__ void __launch_bounds__(MhaFwdShape<DQK, NT>::kThreads, 1) dense_mha_fwd_kernel(
    const __grid_constant__ MhaFwdParams p) {
  using C = MhaFwdShape<DQK, NT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sbase = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  MhaMisc& m = *reinterpret_cast<MhaMisc*>(sbase + C::kMiscOff);
  const int warp = static_cast<int>(threadIdx.x >> 5);
  const uint32_t sb = smem_u32(sbase);
  // CTAs of a cluster are neighbours
  const unsigned ctas = NT == 1 ? static_cast<unsigned>(p.cluster) : 1u, unit = blockIdx.x / ctas;
  const int rank = static_cast<int>(blockIdx.x % ctas);
  int slot, head;
  mha_unit(unit, p.slots, p.order, slot, head);
  const int pack0 = head * p.pack;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kUnits; ++i) mbar_init(smem_u32(&m.full[i]), 1);
    for (int i = 0; i < kMhaFree; ++i) {
      mbar_init(smem_u32(&m.k_free[i]), 1);
      mbar_init(smem_u32(&m.v_free[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&m.q_full[i]), 1);
      mbar_init(smem_u32(&m.s_full[i]), 1);
      mbar_init(smem_u32(&m.p_full[i]), 4);   // one arrival per softmax warp
      mbar_init(smem_u32(&m.o_full[i]), 1);
    }
    mbar_init(smem_u32(&m.o_step), 1);
    mbar_init(smem_u32(&m.drain), 1);
    m.abort_flag = 0;
    m.cleared = 0;
    m.prior_error = *reinterpret_cast<volatile int*>(&g_device_error);
    fence_mbar_init();
    prefetch_tmap(&p.map_q);
    prefetch_tmap(&p.map_k);
    prefetch_tmap(&p.map_v);
  }
  if (warp == 4 * NT) {
    tmem_alloc(smem_u32(&m.tmem_base), 512);
    tmem_relinquish();
  }
  if (warp == 4 * NT + 1) {
    const MhaWork w = mha_find<false>(p.cu_q, p.cu_kv, p.batch, p.total_q, p.total_kv, slot, p.per);
    if (lane_id() == 0) m.work = w;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = m.tmem_base;
  const MhaWork w = m.work;

  if (warp == 4 * NT + 1 && p.fill != 0 && w.end < p.total_q && m.prior_error == 0) {
    if (p.fill & 1) mha_fill_rows(p.out, static_cast<long long>(p.h_q) * (kMhaDv / 2), w.end, p.total_q, 0u);
    if (p.fill & 2) mha_fill_rows(p.lse, p.h_q, w.end, p.total_q, 0xff800000u);
  }
  if (m.prior_error == 0 && w.q1 > w.q0) {
    const MhaSpan<NT> s(p, w, rank);
    if (warp < 4 * NT) {
      if (!mha_softmax<DQK, NT>(p, m, sbase, sb, tmem, w, s, pack0, warp >> 2)) mha_raise(m, kErrMhaSoftmaxWait);
    } else {
      const int never = 0;
      if (s.most > 0 && warp == 4 * NT) {
        if (!mha_mma<DQK, NT>(p, m, sb, s)) mha_raise(m, kErrMhaMmaWait);
        // every MMA issued completes before TMEM is freed
        commit_to(elect_one(), &m.drain);
        mbar_wait(smem_u32(&m.drain), 0, global_timer_ns() + 100000000ull, &never);
      } else if (s.most > 0 && lane_id() == 0) {
        uint32_t fills = 0;
        if (!mha_load<DQK, NT>(p, m, sb, w, s, pack0, pack0 / p.group, fills)) mha_raise(m, kErrMhaLoadWait);
        // every copy issued has landed before the CTA exits (only a unit's last fill can be in flight)
        const uint64_t dl = global_timer_ns() + 100000000ull;
        for (int t = 0; t < NT; ++t)
          if (s.blocks[t] > 0) mbar_wait(smem_u32(&m.q_full[t]), 0, dl, &never);
        for (uint32_t i = fills > C::kUnits ? fills - C::kUnits : 0; i < fills; ++i)
          mbar_wait(smem_u32(&m.full[i % C::kUnits]), (i / C::kUnits) & 1u, dl, &never);
      }
      __syncwarp();
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 4 * NT) tmem_dealloc(tmem, 512);
  if constexpr (NT == 1) {
    if (p.cluster > 1) {
      cluster_sync();   // every CTA's part is there
      if (warp < 4 && m.prior_error == 0 && m.abort_flag == 0 && w.q1 > w.q0) {
        const int t0 = w.tile * p.tok_tile, rows = min(p.tok_tile, w.q1 - w.q0 - t0) * p.pack;
        if (rows <= 4 * p.cluster) mha_join<DQK, 4>(p, m, sb, w, t0, rows, pack0, rank);
        else mha_join<DQK, 32>(p, m, sb, w, t0, rows, pack0, rank);
      }
      cluster_sync();   // no CTA leaves while another reads its part
    }
  }
}

}  // namespace smla
