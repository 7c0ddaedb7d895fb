// Entry points of the operators around a layer's dense attention: the residual norm,
// causal attention over whole prompts in the heads' own space, and the gradients of
// both.  It comes behind latent_api.cuh in the library's one translation unit
// (library.cu) and uses that file's launches and sparse_mla_api.cu's checks and set-up.
#pragma once
#include <algorithm>
#include <cmath>

#include "add_norm_kernel.cuh"
#include "dense_mha_bwd_kernel.cuh"
#include "dense_mha_kernel.cuh"

// ------------------------------------------------------------------ residual norm

namespace {

bool step_ok(long long step) { return step % 8 == 0; }

sparse_mla_status_t check_add_norm(const void* x, long long x_stride, const void* weight, float eps, int n, int d) {
  if (n < 0 || d < 1 || !(eps >= 0.f) || !std::isfinite(eps) || !step_ok(x_stride)) return SPARSE_MLA_ERR_INVALID_ARG;
  if (d % 8 != 0 || d > smla::kAddNormMaxWidth) return SPARSE_MLA_ERR_UNSUPPORTED_SHAPE;
  if (!aligned(x, 16) || !aligned(weight, 16)) return SPARSE_MLA_ERR_INVALID_ARG;
  if (n > 0 && (!x || !weight)) return SPARSE_MLA_ERR_INVALID_ARG;
  return SPARSE_MLA_OK;
}

smla::AddNormParams add_norm_params(const void* x, long long x_stride, const void* weight, float eps, int n, int d) {
  smla::AddNormParams p;
  std::memset(&p, 0, sizeof(p));
  p.x = static_cast<const __nv_bfloat16*>(x);
  p.x_step = x_stride;
  p.weight = static_cast<const __nv_bfloat16*>(weight);
  p.eps = eps;
  p.n = n;
  p.d = d;
  auto two = [](double v) {
    const float hi = static_cast<float>(v);
    return smla::Two{hi, static_cast<float>(v - hi)};
  };
  p.sqrt_d = two(std::sqrt(static_cast<double>(d)));
  p.d_eps = two(static_cast<double>(d) * eps);
  return p;
}

// Vectors of 8 values per thread, and threads: whole warps that hold a row.  The forward
// takes two: one takes 0.6 us less for a single row of 1536 but longer for many (16384 x 1536
// in 16 bits, groups: 40 and 47 us against 34 and 40; 8192 x 7168: 87 and 106 against 73 and
// 93), four with 80 registers 38, 45, 76 and 91.  The backward, with twice the values in a
// thread's registers, takes one up to the 1024 threads of a CTA (8192 x 7168: 74 us, with
// two 108); above 8192 values it has to take two, which spill 280 bytes of its 64 registers:
// 7152 x 8200 take 142 us where 7168 x 8192 take 80.  Rows of less than 512 values leave most
// of a warp idle: 65536 x 128 take 38 to 45 us, four times their bytes.
constexpr int kAddNormVectors = 2;
int add_norm_bwd_vectors(int d) { return d <= 8192 ? 1 : 2; }
int add_norm_threads(int d, int v) { return ((d / 8 + v - 1) / v + 31) / 32 * 32; }

// CTAs: as many as are resident at once.
int add_norm_ctas(int n, int threads, int sms, int regs) {
  const int most = sms * (65536 / regs / threads);
  return n < most ? n : most;
}
constexpr int kAddNormBwdRegs = 64;

void add_norm_launch(const smla::AddNormParams& p, int form, int ctas, int threads, cudaStream_t cs) {
  if (form == smla::kAddNormBf16) smla::add_norm_kernel<kAddNormVectors, smla::kAddNormBf16><<<ctas, threads, 0, cs>>>(p);
  else if (form == smla::kAddNormGroups) smla::add_norm_kernel<kAddNormVectors, smla::kAddNormGroups><<<ctas, threads, 0, cs>>>(p);
  else smla::add_norm_kernel<kAddNormVectors, smla::kAddNormRow><<<ctas, threads, 0, cs>>>(p);
}

}  // namespace

extern "C" {

sparse_mla_status_t mla_add_norm(const void* x, long long x_stride, const void* residual, long long residual_stride,
                                 const void* weight, float eps, void* out, float* scales, int out_format,
                                 void* residual_out, int n, int d, void* stream) {
  sparse_mla_status_t st = check_add_norm(x, x_stride, weight, eps, n, d);
  if (st != SPARSE_MLA_OK) return st;
  if (out_format < MLA_ADD_NORM_BF16 || out_format > MLA_ADD_NORM_E4M3_ROW) return SPARSE_MLA_ERR_INVALID_ARG;
  if (!step_ok(residual_stride) || !aligned(residual, 16) || !aligned(residual_out, 16) || !aligned(out, 16) ||
      !aligned(scales, 4))
    return SPARSE_MLA_ERR_INVALID_ARG;
  if (n > 0 && (!out || (residual && !residual_out) || (out_format != MLA_ADD_NORM_BF16 && !scales)))
    return SPARSE_MLA_ERR_INVALID_ARG;
  int sms = 0;
  if ((st = device_setup(&sms)) != SPARSE_MLA_OK) return st;
  if (n == 0) return SPARSE_MLA_OK;
  smla::AddNormParams p = add_norm_params(x, x_stride, weight, eps, n, d);
  p.residual = static_cast<const __nv_bfloat16*>(residual);
  p.residual_step = residual_stride;
  p.z = static_cast<__nv_bfloat16*>(residual_out);
  p.out = out;
  p.scales = scales;
  const int threads = add_norm_threads(d, kAddNormVectors);
  add_norm_launch(p, out_format, add_norm_ctas(n, threads, sms, smla::kAddNormRegs), threads,
                  static_cast<cudaStream_t>(stream));
  return cudaGetLastError() == cudaSuccess ? SPARSE_MLA_OK : SPARSE_MLA_ERR_CUDA;
}

size_t mla_add_norm_bwd_workspace_size(int n, int d) {
  if (n < 1 || d < 8 || d % 8 != 0 || d > smla::kAddNormMaxWidth) return 0;
  int sms = 0;
  if (device_setup(&sms) != SPARSE_MLA_OK) return 0;
  const int ctas = add_norm_ctas(n, add_norm_threads(d, add_norm_bwd_vectors(d)), sms, kAddNormBwdRegs);
  return static_cast<size_t>(ctas) * static_cast<size_t>(d) * sizeof(float);   // one share of the sums per CTA
}

sparse_mla_status_t mla_add_norm_bwd(const void* z, long long z_stride, const void* weight, float eps,
                                     const void* dout, long long dout_stride, const void* dresidual,
                                     long long dresidual_stride, void* dx, float* dweight, int n, int d,
                                     void* workspace, size_t workspace_bytes, void* stream) {
  sparse_mla_status_t st = check_add_norm(z, z_stride, weight, eps, n, d);
  if (st != SPARSE_MLA_OK) return st;
  if (!step_ok(dout_stride) || !step_ok(dresidual_stride) || !aligned(dout, 16) || !aligned(dresidual, 16) ||
      !aligned(dx, 16) || !aligned(dweight, 4) || !dweight)
    return SPARSE_MLA_ERR_INVALID_ARG;
  if (n > 0 && (!dout || !dx)) return SPARSE_MLA_ERR_INVALID_ARG;
  int sms = 0;
  if ((st = device_setup(&sms)) != SPARSE_MLA_OK) return st;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  if (n == 0)
    return cudaMemsetAsync(dweight, 0, static_cast<size_t>(d) * sizeof(float), cs) == cudaSuccess
               ? SPARSE_MLA_OK : SPARSE_MLA_ERR_CUDA;
  if (!workspace || workspace_bytes < mla_add_norm_bwd_workspace_size(n, d)) return SPARSE_MLA_ERR_WORKSPACE_TOO_SMALL;
  if (!aligned(workspace, 16)) return SPARSE_MLA_ERR_INVALID_ARG;
  smla::AddNormParams p = add_norm_params(z, z_stride, weight, eps, n, d);
  p.dout = static_cast<const __nv_bfloat16*>(dout);
  p.dout_step = dout_stride;
  p.dresidual = static_cast<const __nv_bfloat16*>(dresidual);
  p.dresidual_step = dresidual_stride;
  p.dx = static_cast<__nv_bfloat16*>(dx);
  p.part = static_cast<float*>(workspace);
  const int v = add_norm_bwd_vectors(d), threads = add_norm_threads(d, v);
  const int ctas = add_norm_ctas(n, threads, sms, kAddNormBwdRegs);
  if (v == 1) smla::add_norm_bwd_kernel<1><<<ctas, threads, 0, cs>>>(p);
  else smla::add_norm_bwd_kernel<2><<<ctas, threads, 0, cs>>>(p);
  if (cudaGetLastError() != cudaSuccess) return SPARSE_MLA_ERR_CUDA;
  const cudaError_t e = launch_dependent(smla::add_norm_weight_grad_kernel, dim3(static_cast<unsigned>((d + 31) / 32)),
                                         dim3(1024), cs, static_cast<const float*>(p.part), dweight, ctas, d);
  return e == cudaSuccess ? SPARSE_MLA_OK : SPARSE_MLA_ERR_CUDA;
}

}  // extern "C"

// ------------------------------------------------------------------ dense causal attention

namespace {

struct MhaRows {   // an operand as the caller gives it: row (t, h) at p + t tok + h head
  const void* p;
  long long tok, head;
};

bool mha_rows_ok(const MhaRows& r, int total, int heads) {
  return aligned(r.p, 16) && step_ok(r.tok) && step_ok(r.head) && (total < 2 || r.tok > 0) && (heads < 2 || r.head > 0);
}

sparse_mla_status_t check_mha(const MhaRows& q, const MhaRows& k, const MhaRows& v, const int32_t* cu_q,
                              const int32_t* cu_kv, int batch, float sm_scale, int total_q, int total_kv, int h_q,
                              int h_kv, int d_qk, int d_v) {
  if (total_q < 0 || total_kv < 0 || h_q < 1 || h_kv < 1 || h_q % h_kv != 0 || !(sm_scale >= 0.f) ||
      !std::isfinite(sm_scale))
    return SPARSE_MLA_ERR_INVALID_ARG;
  if ((d_qk != 192 && d_qk != 128) || d_v != 128) return SPARSE_MLA_ERR_UNSUPPORTED_SHAPE;
  if (total_q > INT_MAX / 2 || total_kv > INT_MAX / 2 || h_q > 65535) return SPARSE_MLA_ERR_INVALID_ARG;
  if ((cu_q == nullptr) != (cu_kv == nullptr)) return SPARSE_MLA_ERR_INVALID_ARG;
  if (cu_q && (batch < 1 || batch > INT_MAX / 2 || !aligned(cu_q, 4) || !aligned(cu_kv, 4)))
    return SPARSE_MLA_ERR_INVALID_ARG;
  if (!mha_rows_ok(q, total_q, h_q) || !mha_rows_ok(k, total_kv, h_kv) || !mha_rows_ok(v, total_kv, h_kv))
    return SPARSE_MLA_ERR_INVALID_ARG;
  if ((total_q > 0 && !q.p) || (total_kv > 0 && (!k.p || !v.p))) return SPARSE_MLA_ERR_INVALID_ARG;
  return SPARSE_MLA_OK;
}

// Query heads of one group that a tile of `rows` takes side by side: the most that leave
// at most one row in 16 unused.  One head a tile and side by side (us): 15 texts of up to 2000
// tokens, 32 heads on 8, 188 and 149, their gradients 554 and 488; 16 tokens' gradients on 9000
// keys 122 and 97.
int mha_pack(int group, int rows) {
  for (int n = group < rows ? group : rows; n > 1; --n)
    if (group % n == 0 && rows % n <= rows / (64 / smla::kMhaSpare)) return n;
  return 1;
}

smla::MhaDiv mha_div(int d) {
  int log = 0;
  while (1ll << log < d) ++log;
  return {static_cast<unsigned>((1ull << (31 + log)) / static_cast<unsigned>(d) + 1), d, log};
}

// Tiles of `per` rows that any `batch` sequences of `total` rows (> 0) in all have at most
// (0: one dense sequence): one for each that has rows, and one for each `per` rows more.
long long mha_slots(int total, int per, int batch) {
  const long long n = batch < 1 ? 1 : (batch < total ? batch : total);
  return (total - n) / per + n;
}

// exp's scale in powers of two; kept off zero so that a hidden key's -inf stays one.
float mha_scale_log2(float sm_scale) {
  const float c = sm_scale * 1.4426950408889634f;
  return c > 1e-30f ? c : 1e-30f;
}

// bf16 rows [total, heads, d] in boxes of 64 columns x `box_heads` x `box_rows`,
// 128B-swizzled; boxes past the last row read zeros.
sparse_mla_status_t mha_map(CUtensorMap* map, const MhaRows& r, int total, int heads, int d, int box_heads, int box_rows) {
  EncodeTiledFn enc = nullptr;
  const sparse_mla_status_t st = get_encode(&enc);
  if (st != SPARSE_MLA_OK) return st;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(total)};
  // the stride of a dimension of one row is never used
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(heads > 1 ? r.head : d) * 2,
                           static_cast<cuuint64_t>(total > 1 ? r.tok : d) * 2};
  if (strides[0] >= (1ull << 40) || strides[1] >= (1ull << 40)) return SPARSE_MLA_ERR_INVALID_ARG;
  cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_heads), static_cast<cuuint32_t>(box_rows)};
  cuuint32_t estr[3] = {1, 1, 1};
  const CUresult e = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(r.p), dims, strides, box, estr,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return e == CUDA_SUCCESS ? SPARSE_MLA_OK : SPARSE_MLA_ERR_INVALID_ARG;
}


struct MhaState {
  bool set = false;
  int clusters[2][smla::kMhaMaxCluster + 1] = {};   // at 192 and 128 columns: clusters of so many one-tile CTAs held at once
};
MhaState g_mha[kMaxDevices];   // under g_mu

template <class C>
void mha_cluster_config(cudaLaunchConfig_t* cfg, cudaLaunchAttribute* attr, unsigned ctas, int cluster) {
  cfg->gridDim = dim3(ctas);
  cfg->blockDim = dim3(C::kThreads);
  cfg->dynamicSmemBytes = C::kBytes;
  attr->id = cudaLaunchAttributeClusterDimension;
  attr->val.clusterDim.x = static_cast<unsigned>(cluster);
  attr->val.clusterDim.y = attr->val.clusterDim.z = 1;
  cfg->attrs = attr;
  cfg->numAttrs = 1;
}

// Kernel attributes, and how many clusters of each size the device holds at once (none
// of a size that it refuses).
template <int DQK>
bool mha_setup(int* clusters) {
  auto memory = [](const void* kernel, int bytes) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) == cudaSuccess;
  };
  auto address = [](auto* kernel) { return reinterpret_cast<const void*>(kernel); };
  const void* one = address(smla::dense_mha_fwd_kernel<DQK, 1>);
  const bool ok = memory(one, smla::MhaFwdShape<DQK, 1>::kBytes) &&
                  memory(address(smla::dense_mha_fwd_kernel<DQK, 2>), smla::MhaFwdShape<DQK, 2>::kBytes) &&
                  memory(address(smla::dense_mha_dq_kernel<DQK>), smla::MhaDqShape<DQK>::kBytes) &&
                  memory(address(smla::dense_mha_dkv_kernel<DQK>), smla::MhaDkvShape<DQK>::kBytes);
  bool refused = false;
  if (ok) {
    refused = cudaFuncSetAttribute(one, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess;
    for (int c = 2; c <= smla::kMhaMaxCluster; ++c) {
      cudaLaunchConfig_t cfg = {};
      cudaLaunchAttribute attr = {};
      mha_cluster_config<smla::MhaFwdShape<DQK, 1>>(&cfg, &attr, static_cast<unsigned>(c), c);
      if (cudaOccupancyMaxActiveClusters(&clusters[c], smla::dense_mha_fwd_kernel<DQK, 1>, &cfg) != cudaSuccess) {
        clusters[c] = 0;
        refused = true;
      }
    }
  }
  if (!ok || refused) cudaGetLastError();   // not the next launch's error
  return ok;
}

// The dense attention's kernels, apart from device_setup (which comes first): what a
// device refuses of them stops no other call.
sparse_mla_status_t mha_device_setup(const MhaState** state) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return SPARSE_MLA_ERR_CUDA;
  std::lock_guard<std::mutex> lock(g_mu);
  MhaState& st = g_mha[dev];
  if (!st.set) st.set = mha_setup<192>(st.clusters[0]) && mha_setup<128>(st.clusters[1]);
  *state = &st;
  return st.set ? SPARSE_MLA_OK : SPARSE_MLA_ERR_CUDA;
}

// How the forward's work is laid out: tiles per CTA and CTAs that share a tile's keys.
struct MhaPlan {
  int tiles, cluster;
  long long slots;
};

// The layout whose slowest CTA has the least to do, by the sequences' mean lengths: key
// blocks one after the other, of a longest tile and of the card's mean.  A CTA of two
// tiles takes about as long for a block of both as one of a single tile for its own.
// Measured (us; two tiles a CTA / one / one and the keys shared out):
//   1 token on 5001 keys, 8 heads    65.3 / 60.4 / 14.7
//   16 tokens on 9000, 32 heads on 8 103 / 77.5 / 25.6   1024 tokens, 8 heads  21.7 / 17.8 / 17.5
//   15 texts to 2000, 32 heads on 8  149 / 198 (too many tiles for clusters)
// What mean lengths do not show: 16 tokens behind 30000 keys beside 31 short texts, 8 heads, are
// not shared out and take 352.
MhaPlan mha_plan(int total_q, int total_kv, int batch, bool packed, int packs, int tok_tile, int sms,
                 const int* clusters) {
  const double lq = static_cast<double>(total_q) / batch, lk = static_cast<double>(total_kv) / batch;
  const double longest = std::ceil(lk / smla::kMhaTile), mean = (lk - std::min(lq, lk) / 2) / smla::kMhaTile + 0.5;
  auto units = [&](int tiles) { return std::ceil(lq / (tok_tile * tiles)) * batch * packs; };
  MhaPlan best = {2, 1, 0};
  double least = std::max(longest, units(2) * mean / sms);
  for (int c = 1; c <= smla::kMhaMaxCluster; ++c) {
    if (c > 1 && (units(1) > clusters[c] || longest < 2 * c)) continue;
    const double t = std::max(std::ceil(longest / c), units(1) * mean / sms) + (c > 1 ? 1.0 : 0.0);
    if (t < least) {
      least = t;
      best = {1, c, 0};
    }
  }
  best.slots = mha_slots(total_q, tok_tile * best.tiles, packed ? batch : 0);
  return best;
}

template <int DQK, int NT>
cudaError_t mha_fwd_launch(const smla::MhaFwdParams& p, unsigned ctas, cudaStream_t cs) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr = {};
  mha_cluster_config<smla::MhaFwdShape<DQK, NT>>(&cfg, &attr, ctas, p.cluster);
  cfg.stream = cs;
  return cudaLaunchKernelEx(&cfg, smla::dense_mha_fwd_kernel<DQK, NT>, p);
}

// How many heads' tiles run side by side, of which each head's read `bytes`: as many as come
// to `most` (one at least), so that the tiles find each other's reads in the near half of L2;
// the last ones, two tiles an SM, all together, so that the SMs end together.
// Measured (us, 192 columns, 8192 tokens; all heads that 100 MB hold / 24 MB / 11 MB):
//   dk and dv, 32 heads   1363 / 1026 / 961     64 heads   2700 / 2072 / 1959
//   dq, 32 heads           661 /  630 / 636     out, 64 heads   890 / 884 / 876
// The tail (1, 2, 4 tiles an SM): nine texts up to 2119, 40 heads on 8, dk and dv 362, 344,
// 325; 32 heads on 8 of 8192 tokens 826, 917, 912.  No one of them is the best for both.
constexpr double kMhaNearKeys = 2.4e7, kMhaNearRows = 1.1e7;
smla::MhaHeads mha_order(int heads, double bytes, double most, long long slots, int sms) {
  const double near = std::max(1.0, std::min<double>(heads, std::floor(most / (bytes + 1))));
  const double last = std::max(near, std::ceil(2.0 * sms / std::max<double>(slots, 1)));
  const int n = static_cast<int>(near), lead = last < heads ? (heads - static_cast<int>(last)) / n * n : 0;
  return {mha_div(n), mha_div(lead > 0 ? static_cast<int>(slots) * n : 1), mha_div(heads - lead), lead};
}

// dq (and D into the workspace), then dk and dv.
template <int DQK>
sparse_mla_status_t mha_bwd_launch(const MhaRows& q, const MhaRows& k, const MhaRows& v, const MhaRows& g,
                                   const int32_t* cu_q, const int32_t* cu_kv, int batch, float sm_scale, const void* out,
                                   const float* lse, void* dq, void* dk, void* dv, int total_q, int total_kv, int h_q,
                                   int h_kv, void* workspace, int sms, cudaStream_t cs) {
  smla::MhaBwdParams p;
  std::memset(&p, 0, sizeof(p));
  p.cu_q = cu_q;
  p.cu_kv = cu_kv;
  p.batch = cu_q ? batch : 1;
  p.total_q = total_q;
  p.total_kv = total_kv;
  p.h_q = h_q;
  p.h_kv = h_kv;
  p.group = h_q / h_kv;
  p.scale = sm_scale;
  p.scale_log2 = mha_scale_log2(sm_scale);
  p.k = static_cast<const __nv_bfloat16*>(k.p);
  p.k_tok = k.tok;
  p.k_head = k.head;
  p.dout = static_cast<const __nv_bfloat16*>(g.p);
  p.do_tok = g.tok;
  p.do_head = g.head;
  p.lse = lse;
  p.delta = static_cast<float*>(workspace);
  p.dq = static_cast<__nv_bfloat16*>(dq);
  p.dk = static_cast<__nv_bfloat16*>(dk);
  p.dv = static_cast<__nv_bfloat16*>(dv);
  const unsigned long long t = g_timeout_ns.load();
  p.timeout_ns = t ? t : kDefaultTimeoutNs;
  const int seqs = cu_q ? batch : 0;
  sparse_mla_status_t st = SPARSE_MLA_OK;
  // without rows on one side nothing of it is loaded: any map does
  const bool both = total_q > 0 && total_kv > 0;
  const MhaRows &mk = both ? k : (total_q > 0 ? q : k), &mv = both ? v : mk, &mq = both ? q : mk, &mg = both ? g : mk;
  const MhaRows mo = both ? MhaRows{out, static_cast<long long>(h_q) * smla::kMhaDv, smla::kMhaDv} : mk;
  const int tk = both ? total_kv : (total_q > 0 ? total_q : total_kv), hk = both || total_q == 0 ? h_kv : h_q;
  const int tq = both ? total_q : tk, hq = both ? h_q : hk, dv_cols = both ? smla::kMhaDv : DQK;
  auto maps = [&](int rows, int keys) {   // of a query block and a key block
    p.pack = mha_pack(p.group, rows);
    p.tok_tile = rows / p.pack;
    p.per = mha_div(p.tok_tile);
    if ((st = mha_map(&p.map_q, mq, tq, hq, DQK, p.pack, p.tok_tile)) == SPARSE_MLA_OK &&
        (st = mha_map(&p.map_do, mg, tq, hq, dv_cols, p.pack, p.tok_tile)) == SPARSE_MLA_OK &&
        (st = mha_map(&p.map_o, mo, tq, hq, dv_cols, p.pack, p.tok_tile)) == SPARSE_MLA_OK &&
        (st = mha_map(&p.map_k, mk, tk, hk, DQK, 1, keys)) == SPARSE_MLA_OK)
      st = mha_map(&p.map_v, mv, tk, hk, dv_cols, 1, keys);
    return st == SPARSE_MLA_OK;
  };
  if (total_q > 0) {
    using C = smla::MhaDqShape<DQK>;
    if (!maps(smla::kMhaTile, C::kN)) return st;
    const long long slots = mha_slots(total_q, p.tok_tile, seqs), ctas = slots * (h_q / p.pack);
    if (ctas > INT_MAX) return SPARSE_MLA_ERR_INVALID_ARG;
    p.slots = static_cast<int>(slots);
    p.order = mha_order(h_q / p.pack, static_cast<double>(total_kv) * (DQK + smla::kMhaDv) * 2 * p.pack / p.group,
                        kMhaNearKeys, slots, sms);
    smla::dense_mha_dq_kernel<DQK><<<static_cast<unsigned>(ctas), C::kThreads, C::kBytes, cs>>>(p);
    if (cudaGetLastError() != cudaSuccess) return SPARSE_MLA_ERR_CUDA;
  }
  if (total_kv > 0) {
    using C = smla::MhaDkvShape<DQK>;
    if (!maps(C::kN, smla::kMhaTile)) return st;
    const long long slots = mha_slots(total_kv, smla::kMhaTile, seqs), ctas = slots * h_kv;
    if (ctas > INT_MAX) return SPARSE_MLA_ERR_INVALID_ARG;
    p.slots = static_cast<int>(slots);
    p.order = mha_order(h_kv, static_cast<double>(total_q) * (DQK + smla::kMhaDv) * 2 * p.group,
                        kMhaNearRows, slots, sms);
    // its CTAs may take the SMs that the last tiles of dq leave (and themselves wait for D)
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = C::kBytes;
    cfg.stream = cs;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = total_q > 0 ? 1 : 0;
    if (cudaLaunchKernelEx(&cfg, smla::dense_mha_dkv_kernel<DQK>, p) != cudaSuccess) return SPARSE_MLA_ERR_CUDA;
  }
  return SPARSE_MLA_OK;
}

}  // namespace

extern "C" {

sparse_mla_status_t dense_mha_fwd(const void* q, long long q_tok_stride, long long q_head_stride, const void* k,
                                  long long k_tok_stride, long long k_head_stride, const void* v,
                                  long long v_tok_stride, long long v_head_stride, const int32_t* cu_seqlens_q,
                                  const int32_t* cu_seqlens_kv, int batch, float sm_scale, void* out, float* lse,
                                  int fill, int total_q, int total_kv, int h_q, int h_kv, int d_qk, int d_v,
                                  void* stream) {
  const MhaRows rq = {q, q_tok_stride, q_head_stride}, rk = {k, k_tok_stride, k_head_stride},
                rv = {v, v_tok_stride, v_head_stride};
  sparse_mla_status_t st = check_mha(rq, rk, rv, cu_seqlens_q, cu_seqlens_kv, batch, sm_scale, total_q, total_kv, h_q,
                                     h_kv, d_qk, d_v);
  if (st != SPARSE_MLA_OK) return st;
  if (fill < 0 || fill > 3 || !aligned(out, 16) || !aligned(lse, 4) || (total_q > 0 && (!out || !lse)))
    return SPARSE_MLA_ERR_INVALID_ARG;
  int sms = 0;
  if ((st = device_setup(&sms)) != SPARSE_MLA_OK) return st;
  if (total_q == 0) return SPARSE_MLA_OK;
  const MhaState* state = nullptr;
  if ((st = mha_device_setup(&state)) != SPARSE_MLA_OK) return st;
  smla::MhaFwdParams p;
  std::memset(&p, 0, sizeof(p));
  const int group = h_q / h_kv;
  p.pack = mha_pack(group, smla::kMhaTile);
  p.tok_tile = smla::kMhaTile / p.pack;
  if ((st = mha_map(&p.map_q, rq, total_q, h_q, d_qk, p.pack, p.tok_tile)) != SPARSE_MLA_OK) return st;
  p.cu_q = cu_seqlens_q;
  p.cu_kv = cu_seqlens_kv;
  p.batch = cu_seqlens_q ? batch : 1;
  p.total_q = total_q;
  p.total_kv = total_kv;
  p.h_q = h_q;
  p.group = group;
  p.scale_log2 = mha_scale_log2(sm_scale);
  p.v = static_cast<const __nv_bfloat16*>(v);
  p.v_tok = v_tok_stride;
  p.v_head = v_head_stride;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  p.fill = cu_seqlens_q ? fill : 0;
  const unsigned long long t = g_timeout_ns.load();
  p.timeout_ns = t ? t : kDefaultTimeoutNs;
  const MhaPlan plan = mha_plan(total_q, total_kv, p.batch, cu_seqlens_q != nullptr, h_q / p.pack, p.tok_tile,
                                sms, state->clusters[d_qk == 192 ? 0 : 1]);
  // without keys nothing is loaded: any map does
  const bool keys = total_kv > 0;
  if ((st = mha_map(&p.map_k, keys ? rk : rq, keys ? total_kv : total_q, keys ? h_kv : h_q, d_qk, 1, smla::kMhaTile)) !=
          SPARSE_MLA_OK ||
      (st = mha_map(&p.map_v, keys ? rv : rq, keys ? total_kv : total_q, keys ? h_kv : h_q, smla::kMhaDv, 1,
                    smla::kMhaTile / 2)) != SPARSE_MLA_OK)
    return st;
  p.cluster = plan.cluster;
  p.per = mha_div(p.tok_tile * plan.tiles);
  const long long ctas = plan.slots * (h_q / p.pack) * plan.cluster;
  if (ctas > INT_MAX) return SPARSE_MLA_ERR_INVALID_ARG;
  p.order = mha_order(h_q / p.pack, static_cast<double>(total_kv) * (d_qk + d_v) * 2 * p.pack / group, kMhaNearKeys,
                      plan.slots, sms);
  p.slots = static_cast<int>(plan.slots);
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  const unsigned n = static_cast<unsigned>(ctas);
  const cudaError_t e = d_qk == 192 ? (plan.tiles == 2 ? mha_fwd_launch<192, 2>(p, n, cs) : mha_fwd_launch<192, 1>(p, n, cs))
                                    : (plan.tiles == 2 ? mha_fwd_launch<128, 2>(p, n, cs) : mha_fwd_launch<128, 1>(p, n, cs));
  return e == cudaSuccess ? SPARSE_MLA_OK : SPARSE_MLA_ERR_CUDA;
}

size_t dense_mha_bwd_workspace_size(int total_q, int total_kv, int batch, int h_q, int h_kv, int d_qk, int d_v) {
  (void)batch, (void)d_qk, (void)d_v;
  if (total_q < 1 || total_kv < 0 || h_q < 1 || h_kv < 1) return 0;
  return static_cast<size_t>(total_q) * static_cast<size_t>(h_q) * sizeof(float);
}

sparse_mla_status_t dense_mha_bwd(const void* q, long long q_tok_stride, long long q_head_stride, const void* k,
                                  long long k_tok_stride, long long k_head_stride, const void* v,
                                  long long v_tok_stride, long long v_head_stride, const int32_t* cu_seqlens_q,
                                  const int32_t* cu_seqlens_kv, int batch, float sm_scale, const void* out,
                                  const float* lse, const void* dout, long long dout_tok_stride,
                                  long long dout_head_stride, void* dq, void* dk, void* dv, int total_q, int total_kv,
                                  int h_q, int h_kv, int d_qk, int d_v, void* workspace, size_t workspace_bytes,
                                  void* stream) {
  const MhaRows rq = {q, q_tok_stride, q_head_stride}, rk = {k, k_tok_stride, k_head_stride},
                rv = {v, v_tok_stride, v_head_stride}, rg = {dout, dout_tok_stride, dout_head_stride};
  sparse_mla_status_t st = check_mha(rq, rk, rv, cu_seqlens_q, cu_seqlens_kv, batch, sm_scale, total_q, total_kv, h_q,
                                     h_kv, d_qk, d_v);
  if (st != SPARSE_MLA_OK) return st;
  if (!mha_rows_ok(rg, total_q, h_q) || !aligned(out, 16) || !aligned(lse, 4) || !aligned(dq, 16) || !aligned(dk, 16) ||
      !aligned(dv, 16))
    return SPARSE_MLA_ERR_INVALID_ARG;
  if ((total_q > 0 && (!out || !lse || !dout || !dq)) || (total_kv > 0 && (!dk || !dv))) return SPARSE_MLA_ERR_INVALID_ARG;
  int sms = 0;
  if ((st = device_setup(&sms)) != SPARSE_MLA_OK) return st;
  const size_t need = dense_mha_bwd_workspace_size(total_q, total_kv, batch, h_q, h_kv, d_qk, d_v);
  if (need > 0 && (!workspace || workspace_bytes < need)) return SPARSE_MLA_ERR_WORKSPACE_TOO_SMALL;
  if (!aligned(workspace, 16)) return SPARSE_MLA_ERR_INVALID_ARG;
  if (total_q == 0 && total_kv == 0) return SPARSE_MLA_OK;
  const MhaState* state = nullptr;
  if ((st = mha_device_setup(&state)) != SPARSE_MLA_OK) return st;
  return d_qk == 192 ? mha_bwd_launch<192>(rq, rk, rv, rg, cu_seqlens_q, cu_seqlens_kv, batch, sm_scale, out, lse, dq, dk,
                                           dv, total_q, total_kv, h_q, h_kv, workspace, sms,
                                           static_cast<cudaStream_t>(stream))
                     : mha_bwd_launch<128>(rq, rk, rv, rg, cu_seqlens_q, cu_seqlens_kv, batch, sm_scale, out, lse, dq, dk,
                                           dv, total_q, total_kv, h_q, h_kv, workspace, sms,
                                           static_cast<cudaStream_t>(stream));
}

}  // extern "C"
