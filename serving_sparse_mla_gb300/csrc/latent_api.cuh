// Entry points around the latent cache: norms, rotation and cache write, their
// gradients, and the decode over the 4-bit cache.  It comes behind sparse_mla_api.cu
// in the library's one translation unit (library.cu) and uses that file's checks and set-up.
#pragma once
#include <cmath>

#include "fp4_decode_kernel.cuh"
#include "norm_rope_kernel.cuh"

namespace {

constexpr int kF4ClusterSizes = 4;   // 16, 8, 4 and 2 CTAs
constexpr int kF4ClusterSlack = 192;   // list entries
enum F4ShapeId { kF4Heads8, kF4Heads16, kF4Heads32, kF4Heads8Few, kF4Heads16Few, kF4Shapes };

struct F4State {
  bool set = false;                                // set up with the first call
  int clusters[kF4Shapes][kF4ClusterSizes] = {};   // per shape: clusters held at once
};
F4State g_f4[kMaxDevices];   // under g_mu

template <class C>
void f4_cluster_config(cudaLaunchConfig_t* cfg, cudaLaunchAttribute* attr, int ctas, int cluster) {
  cfg->gridDim = dim3(static_cast<unsigned>(ctas));
  cfg->blockDim = dim3(C::kThreads);
  cfg->dynamicSmemBytes = C::kBytes;
  attr->id = cudaLaunchAttributeClusterDimension;
  attr->val.clusterDim.x = static_cast<unsigned>(cluster);
  attr->val.clusterDim.y = attr->val.clusterDim.z = 1;
  cfg->attrs = attr;
  cfg->numAttrs = 1;
}

// Kernel attributes of a shape, and how many of its clusters of 16, 8, 4 and 2 CTAs
// the device holds at once: none of a size that it refuses (16 is past what every
// device takes, and a part of a device may take less).
template <class C>
bool f4_setup(int* clusters) {
  bool refused = false;
  const bool ok = cudaFuncSetAttribute(smla::fp4_decode_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       C::kBytes) == cudaSuccess;
  if (ok) {
    refused = cudaFuncSetAttribute(smla::fp4_decode_kernel<C>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) !=
              cudaSuccess;
    for (int i = 0; i < kF4ClusterSizes; ++i) {
      const int c = smla::kF4MaxCluster >> i;
      cudaLaunchConfig_t cfg = {};
      cudaLaunchAttribute attr = {};
      f4_cluster_config<C>(&cfg, &attr, c, c);
      if (cudaOccupancyMaxActiveClusters(&clusters[i], smla::fp4_decode_kernel<C>, &cfg) != cudaSuccess) {
        clusters[i] = 0;
        refused = true;
      }
    }
  }
  if (!ok || refused) cudaGetLastError();   // not the next launch's error
  return ok;
}

// The 4-bit decode's kernels, apart from device_setup (which comes first): what a
// device refuses of them stops no other call.
sparse_mla_status_t f4_device_setup() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return SPARSE_MLA_ERR_CUDA;
  std::lock_guard<std::mutex> lock(g_mu);
  F4State& st = g_f4[dev];
  if (!st.set)
    st.set = f4_setup<smla::Fp4Shape8>(st.clusters[kF4Heads8]) &&
             f4_setup<smla::Fp4Shape16>(st.clusters[kF4Heads16]) &&
             f4_setup<smla::Fp4Shape32>(st.clusters[kF4Heads32]) &&
             f4_setup<smla::Fp4Shape8Few>(st.clusters[kF4Heads8Few]) &&
             f4_setup<smla::Fp4Shape16Few>(st.clusters[kF4Heads16Few]);
  return st.set ? SPARSE_MLA_OK : SPARSE_MLA_ERR_CUDA;
}

// A kernel that may be set up while the one before it on the stream still runs
// (and itself waits for that one's end before it reads its results).
template <class... Args>
cudaError_t launch_dependent(void (*kernel)(Args...), dim3 grid, dim3 block, cudaStream_t cs, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.stream = cs;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace

// ------------------------------------------------------------------ 4-bit cache decode

namespace {

// A 4-bit cache's factor: far enough from fp32's ends that a group's step
// (a scale of 2^-9 .. 448 times the factor) and its reciprocal are normal.
bool kv_scale_ok(float f) { return f >= 0x1p-64f && f <= 0x1p64f; }

template <class F>
auto f4_with(int shape, F&& f) {
  switch (shape) {
    case kF4Heads8: return f(smla::Fp4Shape8());
    case kF4Heads16: return f(smla::Fp4Shape16());
    case kF4Heads8Few: return f(smla::Fp4Shape8Few());
    case kF4Heads16Few: return f(smla::Fp4Shape16Few());
    default: return f(smla::Fp4Shape32());
  }
}

// Units, rows and list entries are counted in 32 bits (a list's last block may
// be a block past its end), CTAs times blocks in 64 (3 CTAs per SM are far below 4096).
bool f4_sizes_ok(long long n_tok, int h_q, int topk) {
  if (n_tok > INT_MAX / 2 || static_cast<long long>(h_q) * n_tok > INT_MAX || topk > INT_MAX - 1024) return false;
  const long long blocks = n_tok * ((h_q - 1) / 8 + 1) * ((topk - 1) / 64 + 1);   // at least as many as any shape's
  return blocks <= (1LL << 62) / 4096;
}

struct F4Plan {
  int shape;
  int ctas, groups, rows, nb;
  int cluster;                      // CTAs per unit, merging among themselves (0: ranges)
  size_t lse_at, bytes;   // bytes from the workspace's start; bytes 0: no unit is cut
};

// The grid: as many CTAs as the card holds at once, or fewer where the lists
// are short (a range has at least nb / 62 blocks, so a unit at most 64 pieces).
template <class C>
F4Plan f4_plan_of(long long n_tok, int h_q, int topk, int sms, const int* clusters) {
  F4Plan f;
  constexpr int H = C::kHeads;
  f.groups = (h_q - 1) / H + 1;
  f.rows = h_q < H ? h_q : H;
  f.nb = (topk + C::kRows - 1) / C::kRows;
  const long long most = static_cast<long long>(sms) * C::kPerSm;
  const long long g = n_tok * f.groups * f.nb / ((f.nb + 61) / 62);
  f.ctas = static_cast<int>(g > most ? most : (g < 1 ? 1 : g));
  const size_t slots = 2 * static_cast<size_t>(f.ctas) * static_cast<size_t>(f.rows);
  f.lse_at = slots * smla::kDv * sizeof(float);
  // Few units: the largest cluster of which all fit at once, where that leaves a
  // CTA at most kF4ClusterSlack list entries more than an equal cut of all the work
  // (8 heads, lists of 2048, clusters against ranges: 28 tokens 17.1 and 19.9 us, 96
  // tokens 33.5 and 37.1; at 170 tokens clusters would take 58 us and ranges take 50).
  const long long units = n_tok * f.groups;
  f.cluster = 0;
  for (int i = 0; i < kF4ClusterSizes && f.cluster == 0; ++i) {
    const int c = smla::kF4MaxCluster >> i;
    if (c <= f.nb && units <= clusters[i] && (f.nb + c - 1) / c <= units * f.nb / most + kF4ClusterSlack / C::kRows) f.cluster = c;
  }
  // Short lists: by the same rule a CTA takes a whole list (300 lists of 256, 8
  // heads: 16.2 us, cut into ranges 24.2).
  const bool own = units <= most && f.nb <= units * f.nb / most + kF4ClusterSlack / C::kRows;
  if (f.cluster > 0 || own) {
    f.ctas = static_cast<int>(units) * (f.cluster > 0 ? f.cluster : 1);
    f.lse_at = f.bytes = 0;
    return f;
  }
  const long long total = n_tok * f.groups * f.nb;
  const bool whole = total % f.ctas == 0 && total / f.ctas % f.nb == 0;   // every range is whole units
  f.bytes = whole ? 0 : f.lse_at + slots * sizeof(float);
  return f;
}

// The smallest of 8, 16 and 32 heads that holds h_q (more are several units of
// 32), three CTAs of four warps per SM at 8 and 16 heads.  Few tokens: CTAs of
// eight warps and units of at most 16 heads, where that leaves a CTA at most 256
// list entries (512 at 9 to 16 heads).  Lists of 2048, few against the other; 8
// heads: 1 token 8.9 and 10.5 us, 12 tokens 11.2 and 13.0, 28 tokens 17.7 and 17.1;
// 16 heads: 1 token 11.9 and 14.3, 16 tokens 15.5 and 20.6, 48 tokens 29.8 and
// 29.6; 32 heads: 1 token 12.0 and 17.2, 8 tokens 15.6 and 17.3, 24 tokens 28.1
// and 26.8.
F4Plan f4_plan(long long n_tok, int h_q, int topk, int sms) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) dev = 0;
  auto plan = [&](int shape) {
    F4Plan f = f4_with(shape, [&](auto c) { return f4_plan_of<decltype(c)>(n_tok, h_q, topk, sms, g_f4[dev].clusters[shape]); });
    f.shape = shape;
    return f;
  };
  const F4Plan few = plan(h_q <= 8 ? kF4Heads8Few : kF4Heads16Few);
  const long long entries = few.cluster > 0 ? topk : n_tok * few.groups * topk;   // of a cluster, of the grid
  const long long limit = h_q > 8 && h_q <= 16 ? 512 : 256;
  if (n_tok * few.groups <= few.ctas && entries <= limit * (few.cluster > 0 ? few.cluster : few.ctas)) return few;
  return plan(h_q <= 8 ? kF4Heads8 : (h_q <= 16 ? kF4Heads16 : kF4Heads32));
}

// A CTA counts its blocks, and a few past them, in an int.
bool f4_blocks_ok(const F4Plan& f, long long n_tok) { return n_tok * f.groups * f.nb / f.ctas < INT_MAX - 8; }

template <class C>
cudaError_t f4_launch(const smla::Fp4Params& p, cudaStream_t cs) {
  if (p.cluster > 0) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr = {};
    f4_cluster_config<C>(&cfg, &attr, p.ctas, p.cluster);
    cfg.stream = cs;
    return cudaLaunchKernelEx(&cfg, smla::fp4_decode_kernel<C>, p);
  }
  smla::fp4_decode_kernel<C><<<p.ctas, C::kThreads, C::kBytes, cs>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || p.part_o == nullptr) return e;
  // two warps a row, eight a CTA; set up while the decode runs
  return launch_dependent(smla::fp4_merge_kernel,
                          dim3(static_cast<unsigned>((static_cast<long long>(p.n_tok) * p.h_q + 3) / 4)), dim3(256), cs, p,
                          static_cast<int>(C::kHeads));
}

}  // namespace

extern "C" {

size_t sparse_mla_decode_fp4_workspace_size(int batch, int s_next, int h_q, int d_v, int topk) {
  if (batch < 1 || s_next < 1 || h_q < 1 || topk < 1 || d_v != smla::kDv) return 0;
  int sms = 0;
  const long long n_tok = static_cast<long long>(batch) * s_next;
  if (!f4_sizes_ok(n_tok, h_q, topk) || device_setup(&sms) != SPARSE_MLA_OK || f4_device_setup() != SPARSE_MLA_OK) return 0;
  const F4Plan f = f4_plan(n_tok, h_q, topk, sms);
  return f4_blocks_ok(f, n_tok) ? f.bytes : 0;
}

sparse_mla_status_t sparse_mla_decode_fp4(const void* q, const void* kv_cache, const int32_t* block_table,
                                          const int32_t* cache_seqlens, const int32_t* indices, float sm_scale,
                                          float kv_scale, void* out, float* lse, int batch, int s_next, int h_q,
                                          int d_qk, int d_v, int topk, int page_size, int max_blocks, int num_blocks,
                                          void* workspace, size_t workspace_bytes, void* stream) {
  int sms = 0;
  if (!kv_scale_ok(kv_scale)) return SPARSE_MLA_ERR_INVALID_ARG;
  if (batch > 0 && s_next > 0 && h_q > 0 && topk > 0 &&
      !f4_sizes_ok(static_cast<long long>(batch) * s_next, h_q, topk))
    return SPARSE_MLA_ERR_INVALID_ARG;
  sparse_mla_status_t st = check_decode(q, kv_cache, block_table, cache_seqlens, indices, out, lse, batch, s_next,
                                        h_q, d_qk, d_v, topk, page_size, max_blocks, num_blocks, &sms);
  if (st != SPARSE_MLA_OK) return st;
  const long long n_tok = static_cast<long long>(batch) * s_next;
  if (n_tok == 0) return SPARSE_MLA_OK;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  if (num_blocks == 0 || max_blocks == 0) return launch_fill(out, lse, n_tok * h_q, cs);
  if ((st = f4_device_setup()) != SPARSE_MLA_OK) return st;
  const F4Plan f = f4_plan(n_tok, h_q, topk, sms);
  if (!f4_blocks_ok(f, n_tok)) return SPARSE_MLA_ERR_INVALID_ARG;
  if (f.bytes > 0 && (workspace_bytes < f.bytes || !workspace)) return SPARSE_MLA_ERR_WORKSPACE_TOO_SMALL;
  if (f.bytes > 0 && !aligned(workspace, 16)) return SPARSE_MLA_ERR_INVALID_ARG;
  smla::Fp4Params p;
  std::memset(&p, 0, sizeof(p));
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.cache = static_cast<const uint8_t*>(kv_cache);
  p.indices = indices;
  p.block_table = block_table;
  p.seqlens = cache_seqlens;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  p.n_tok = static_cast<int>(n_tok);
  p.h_q = h_q;
  p.topk = topk;
  p.s_next = s_next;
  p.page_size = page_size;
  p.max_blocks = max_blocks;
  p.num_blocks = num_blocks;
  p.groups = f.groups;
  p.nb = f.nb;
  p.ctas = f.ctas;
  p.part_rows = f.rows;
  p.cluster = f.cluster;
  p.scale_log2 = sm_scale * 1.4426950408889634f;
  p.kv_scale = kv_scale;
  if (f.bytes > 0) {
    unsigned char* ws = static_cast<unsigned char*>(workspace);
    p.part_o = reinterpret_cast<float*>(ws);
    p.part_lse = reinterpret_cast<float*>(ws + f.lse_at);
  }
  const cudaError_t e = f4_with(f.shape, [&](auto c) { return f4_launch<decltype(c)>(p, cs); });
  return e == cudaSuccess ? SPARSE_MLA_OK : SPARSE_MLA_ERR_CUDA;
}

}  // extern "C"

// ------------------------------------------------------------------ norms, rotation, cache write

namespace {

// Row strides: whole 16-byte steps, so that every row starts on one.
bool row_strides_ok(long long a, long long b) { return a % 8 == 0 && b % 8 == 0; }

sparse_mla_status_t check_norm(const void* q, long long q_tok_stride, long long q_head_stride, const void* kv,
                               long long kv_tok_stride, const int32_t* positions, const float* cos_sin, int n_pos,
                               const void* q_weight, const void* kv_weight, float eps, int n_tok, int h_q, int d_qk) {
  if (n_tok < 0 || h_q < 1 || n_pos < 0 || !(eps >= 0.f) || !std::isfinite(eps)) return SPARSE_MLA_ERR_INVALID_ARG;
  if (n_tok > INT_MAX / 2 || static_cast<long long>(h_q) * 64 > INT_MAX) return SPARSE_MLA_ERR_INVALID_ARG;
  if (d_qk != smla::kRowW) return SPARSE_MLA_ERR_UNSUPPORTED_SHAPE;
  if (!row_strides_ok(q_tok_stride, q_head_stride) || !row_strides_ok(kv_tok_stride, 0))
    return SPARSE_MLA_ERR_INVALID_ARG;
  if (!aligned(q_weight, 16) || !aligned(kv_weight, 16)) return SPARSE_MLA_ERR_INVALID_ARG;
  if (n_tok == 0) return SPARSE_MLA_OK;
  if (!q || !kv || !positions || (n_pos > 0 && !cos_sin)) return SPARSE_MLA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(kv, 16) || !aligned(positions, 4) || !aligned(cos_sin, 16))
    return SPARSE_MLA_ERR_INVALID_ARG;
  return SPARSE_MLA_OK;
}

smla::NormParams norm_params(const void* q, long long q_tok_stride, long long q_head_stride, const void* kv,
                             long long kv_tok_stride, const int32_t* positions, const float* cos_sin, int n_pos,
                             const void* q_weight, const void* kv_weight, float eps, int interleaved, int n_tok,
                             int h_q) {
  smla::NormParams p;
  std::memset(&p, 0, sizeof(p));
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.kv = static_cast<const __nv_bfloat16*>(kv);
  p.q_tok = q_tok_stride;
  p.q_head = q_head_stride;
  p.kv_tok = kv_tok_stride;
  p.positions = positions;
  p.cos_sin = cos_sin;
  p.n_pos = n_pos;
  p.q_weight = static_cast<const __nv_bfloat16*>(q_weight);
  p.kv_weight = static_cast<const __nv_bfloat16*>(kv_weight);
  p.eps = eps;
  p.interleaved = interleaved;
  p.n_tok = n_tok;
  p.h_q = h_q;
  return p;
}

// Rows per warp grow with the batch once the card is full (CTAs of 8 warps,
// one row per warp at a time).
int norm_ctas(long long rows, int sms, int per_sm) {
  const long long need = (rows + smla::kNormWarps - 1) / smla::kNormWarps;
  const long long most = static_cast<long long>(sms) * per_sm;
  return static_cast<int>(need < most ? (need < 1 ? 1 : need) : most);
}
// CTAs per SM: as many as are resident at once (8192 tokens x 64 heads: 184.6 us;
// 8, 16 and 32 times the SMs: 186.3, 188.8, 190.6 us).
constexpr int kNormFwdPerSm = 4;
constexpr int kNormBwdPerSm = 2;

}  // namespace

extern "C" {

sparse_mla_status_t mla_norm_rope(const void* q, long long q_tok_stride, long long q_head_stride, const void* kv,
                                  long long kv_tok_stride, const int32_t* positions, const float* cos_sin, int n_pos,
                                  const void* q_weight, const void* kv_weight, float eps, int interleaved,
                                  void* q_out, void* kv_out, void* kv_cache, int cache_format, float kv_scale,
                                  const int32_t* slots, int n_slots, int n_tok, int h_q, int d_qk, void* stream) {
  sparse_mla_status_t st = check_norm(q, q_tok_stride, q_head_stride, kv, kv_tok_stride, positions, cos_sin, n_pos,
                                      q_weight, kv_weight, eps, n_tok, h_q, d_qk);
  if (st != SPARSE_MLA_OK) return st;
  const int format = cache_format & ~(SPARSE_MLA_ZERO_Q_PADDING | SPARSE_MLA_ZERO_KV_PADDING);
  if (n_slots < 0 || format < 0 || format > 2) return SPARSE_MLA_ERR_INVALID_ARG;
  if (!kv_scale_ok(kv_scale) || (format != SPARSE_MLA_CACHE_FP4 && kv_scale != 1.f))
    return SPARSE_MLA_ERR_INVALID_ARG;
  const bool cached = kv_cache != nullptr && n_slots > 0;
  if (cached && n_tok > 0 && (!slots || !aligned(slots, 4) || !aligned(kv_cache, 16))) return SPARSE_MLA_ERR_INVALID_ARG;
  if (n_tok > 0 && (!q_out || !aligned(q_out, 16) || !aligned(kv_out, 16))) return SPARSE_MLA_ERR_INVALID_ARG;
  int sms = 0;
  if ((st = device_setup(&sms)) != SPARSE_MLA_OK) return st;
  if (n_tok == 0) return SPARSE_MLA_OK;
  smla::NormParams p = norm_params(q, q_tok_stride, q_head_stride, kv, kv_tok_stride, positions, cos_sin, n_pos,
                                   q_weight, kv_weight, eps, interleaved, n_tok, h_q);
  p.q_out = static_cast<__nv_bfloat16*>(q_out);
  p.kv_out = static_cast<__nv_bfloat16*>(kv_out);
  p.cache = static_cast<uint8_t*>(kv_cache);
  p.slots = slots;
  // Without a cache the row is still rounded as that format would hold it.
  p.format = format;
  p.zero_q = (cache_format & SPARSE_MLA_ZERO_Q_PADDING) != 0;
  p.zero_kv = (cache_format & SPARSE_MLA_ZERO_KV_PADDING) != 0 && kv_out != nullptr;
  p.n_slots = cached ? n_slots : 0;
  p.kv_scale = kv_scale;
  p.kv_scale6 = static_cast<float>(6.0 * kv_scale);
  const long long rows = static_cast<long long>(n_tok) * (h_q + 1);
  smla::norm_rope_kernel<<<norm_ctas(rows, sms, kNormFwdPerSm), smla::kNormWarps * 32, 0,
                           static_cast<cudaStream_t>(stream)>>>(p);
  return cudaGetLastError() == cudaSuccess ? SPARSE_MLA_OK : SPARSE_MLA_ERR_CUDA;
}

size_t mla_norm_rope_bwd_workspace_size(int n_tok, int h_q) {
  if (n_tok < 1 || h_q < 1) return 0;
  int sms = 0;
  if (device_setup(&sms) != SPARSE_MLA_OK) return 0;
  // one share of 512 sums per CTA for either weight
  return 2 * static_cast<size_t>(norm_ctas(static_cast<long long>(n_tok) * h_q, sms, kNormBwdPerSm)) * smla::kLatW *
         sizeof(float);
}

sparse_mla_status_t mla_norm_rope_bwd(const void* q, long long q_tok_stride, long long q_head_stride, const void* kv,
                                      long long kv_tok_stride, const int32_t* positions, const float* cos_sin,
                                      int n_pos, const void* q_weight, const void* kv_weight, float eps,
                                      int interleaved, const float* dq, const float* dkv, void* dq_in, void* dkv_in,
                                      float* dq_weight, float* dkv_weight, int n_tok, int h_q, int d_qk,
                                      void* workspace, size_t workspace_bytes, void* stream) {
  sparse_mla_status_t st = check_norm(q, q_tok_stride, q_head_stride, kv, kv_tok_stride, positions, cos_sin, n_pos,
                                      q_weight, kv_weight, eps, n_tok, h_q, d_qk);
  if (st != SPARSE_MLA_OK) return st;
  if ((q_weight != nullptr) != (dq_weight != nullptr) || (kv_weight != nullptr) != (dkv_weight != nullptr) ||
      !aligned(dq_weight, 4) || !aligned(dkv_weight, 4))
    return SPARSE_MLA_ERR_INVALID_ARG;
  if (n_tok > 0 && (!dq || !dkv || !dq_in || !dkv_in || !aligned(dq, 16) || !aligned(dkv, 16) || !aligned(dq_in, 16) ||
                    !aligned(dkv_in, 16)))
    return SPARSE_MLA_ERR_INVALID_ARG;
  int sms = 0;
  if ((st = device_setup(&sms)) != SPARSE_MLA_OK) return st;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  if (n_tok == 0) {
    if (dq_weight && cudaMemsetAsync(dq_weight, 0, smla::kLatW * sizeof(float), cs) != cudaSuccess)
      return SPARSE_MLA_ERR_CUDA;
    if (dkv_weight && cudaMemsetAsync(dkv_weight, 0, smla::kLatW * sizeof(float), cs) != cudaSuccess)
      return SPARSE_MLA_ERR_CUDA;
    return SPARSE_MLA_OK;
  }
  const bool sums = dq_weight || dkv_weight;
  const size_t need = sums ? mla_norm_rope_bwd_workspace_size(n_tok, h_q) : 0;
  if (sums && (!workspace || workspace_bytes < need)) return SPARSE_MLA_ERR_WORKSPACE_TOO_SMALL;
  if (sums && !aligned(workspace, 16)) return SPARSE_MLA_ERR_INVALID_ARG;
  smla::NormParams p = norm_params(q, q_tok_stride, q_head_stride, kv, kv_tok_stride, positions, cos_sin, n_pos,
                                   q_weight, kv_weight, eps, interleaved, n_tok, h_q);
  p.dq = dq;
  p.dkv = dkv;
  p.dq_in = static_cast<__nv_bfloat16*>(dq_in);
  p.dkv_in = static_cast<__nv_bfloat16*>(dkv_in);
  const int ctas = norm_ctas(static_cast<long long>(n_tok) * h_q, sms, kNormBwdPerSm);
  p.part_q = static_cast<float*>(workspace);
  p.part_kv = p.part_q + static_cast<size_t>(ctas) * smla::kLatW;
  const dim3 threads(smla::kNormWarps * 32);
  if (q_weight && kv_weight) smla::norm_rope_bwd_kernel<true, true><<<ctas, threads, 0, cs>>>(p);
  else if (q_weight) smla::norm_rope_bwd_kernel<true, false><<<ctas, threads, 0, cs>>>(p);
  else if (kv_weight) smla::norm_rope_bwd_kernel<false, true><<<ctas, threads, 0, cs>>>(p);
  else smla::norm_rope_bwd_kernel<false, false><<<ctas, threads, 0, cs>>>(p);
  if (cudaGetLastError() != cudaSuccess) return SPARSE_MLA_ERR_CUDA;
  if (!sums) return SPARSE_MLA_OK;
  const cudaError_t e = launch_dependent(smla::norm_weight_grad_kernel, dim3(smla::kLatW / 32, 2), dim3(1024), cs,
                                         static_cast<const float*>(p.part_q), static_cast<const float*>(p.part_kv),
                                         dq_weight, dkv_weight, ctas);
  return e == cudaSuccess ? SPARSE_MLA_OK : SPARSE_MLA_ERR_CUDA;
}

}  // extern "C"
