// mla_token_mass: the attention weight that every cached token received.
//
//   mass[slot(t)] = decay mass[slot(t)] + sum_{i, h} exp(s_{i,h}(t) - lse_{i,h})
// over the step's queries i that see token t and all heads, with the decode's
// scores s and the log-sum-exp that the attention returned.
//
// The simplest form: a block takes 32 tokens, dequantizes them into shared
// memory, and its warps go through the rows, lane = token.
#include <math.h>

#include "mla_internal.cuh"

namespace mla {
namespace {

constexpr int kMassThreads = 256, kMassWarps = kMassThreads / 32;
constexpr int kMassPitch = kDc + kDr + 1;

struct MassParams {
  const uint8_t* pool;
  PageLayout L;
  OutlierSet outl;
  int lf, kf, num_pages;
  const float* q_lat;
  const uint16_t* q_pe;
  const float* lse;
  const int32_t* table;
  int max_pages;
  const int32_t *q_start, *seq_lens, *counted;
  int B, N, H, max_new;
  float scale, decay;
  float* mass;
  int32_t* dev_err;
};

// Channel ch of block token u (0..511 latent, then k_pe), dequantized.
__device__ float value_of(const MassParams& p, const uint8_t* blk, int u, int ch) {
  const bool kpe = ch >= kDc;
  const int c = kpe ? ch - kDc : ch, fmt = kpe ? p.kf : p.lf;
  const uint8_t* row = blk + (kpe ? p.L.kpe_off + u * p.L.kpe_row : p.L.codes_off + u * p.L.codes_row);
  auto at = [&](int chunk) { return row + 16 * (kpe ? kpe_chunk_pos(chunk, u, fmt) : latent_chunk_pos(chunk, u)); };
  if (fmt == MLA_FMT_BF16) return bf16f(reinterpret_cast<const uint16_t*>(at(c / 8))[c % 8]);
  if (!kpe && fmt == MLA_FMT_INT8_OUTLIER && (p.outl.mask[c >> 5] >> (c & 31) & 1u)) {
    for (int k = 0; k < kNOut; ++k)
      if (p.outl.ch[k] == c) return bf16f(reinterpret_cast<const uint16_t*>(blk + p.L.outlier_off)[k * kBlockTokens + u]);
  }
  const int group = kpe ? kKG : latent_group_size(fmt);
  const float s = reinterpret_cast<const float*>(blk + (kpe ? p.L.kpe_scale_off : p.L.scale_off))[c / group * kBlockTokens + u];
  if (fmt == MLA_FMT_INT4_ASYM || fmt == MLA_FMT_INT4_SYM) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(at(c / 32));
    const int idx = c % 16, j = idx / 4, k = ((idx & 2) >> 1) + 4 * (idx & 1) + 2 * (c / 16 % 2);
    const float q = (float)((w[j] >> (4 * k)) & 15u);
    const float z = fmt == MLA_FMT_INT4_SYM ? 8.f : reinterpret_cast<const float*>(blk + p.L.zero_off)[c / group * kBlockTokens + u];
    return (q - z) * s;
  }
  const int8_t* q = reinterpret_cast<const int8_t*>(at(c / 16));
  const int i = c % 16;
  return (float)(fmt == MLA_FMT_INT8_G8 && !kpe ? q[i % 8 / 2 * 4 + i / 8 * 2 + i % 2] : q[i]) * s;
}

__global__ void __launch_bounds__(kMassThreads) mass_kernel(const MassParams p) {
  extern __shared__ float s_x[];
  __shared__ float s_sum[kMassWarps][kBlockTokens];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, b = blockIdx.y;
  pdl_launch_dependents();
  pdl_wait();
  bool bad = false;
  for (int i = tid; i < p.B; i += kMassThreads) {
    const int lo = __ldcg(p.q_start + i), hi = __ldcg(p.q_start + i + 1);
    bad |= lo < 0 || hi < lo || hi > p.N;
  }
  bad = __syncthreads_or(bad);
  const int q0 = __ldcg(p.q_start + b), n = bad ? 0 : __ldcg(p.q_start + b + 1) - q0, len = __ldcg(p.seq_lens + b);
  if (bad || n > p.max_new || len < 0 || len > p.max_pages * kPage || (len > 0 && len < n)) {
    if (tid == 0) set_err(p.dev_err, MLA_DEVERR_SEQLEN);
    return;
  }
  if (n == 0 || len == 0) return;
  const int ctx = len - n;
  int counted = p.counted ? __ldcg(p.counted + b) : ctx;
  if (counted < 0 || counted > len) {
    if (tid == 0) set_err(p.dev_err, MLA_DEVERR_SEQLEN);
    return;
  }
  for (int blk = blockIdx.x; blk * kBlockTokens < len; blk += gridDim.x) {
    const int page = __ldcg(p.table + (int64_t)b * p.max_pages + blk / 2);
    if (page < 0 || page >= p.num_pages) {
      if (tid == 0) set_err(p.dev_err, MLA_DEVERR_PAGE);
      continue;
    }
    const uint8_t* src = p.pool + (int64_t)page * p.L.page_bytes + (blk & 1) * p.L.block_bytes;
    __syncthreads();
    for (int i = tid; i < kBlockTokens * (kDc + kDr); i += kMassThreads)
      s_x[i % kBlockTokens * kMassPitch + i / kBlockTokens] = value_of(p, src, i % kBlockTokens, i / kBlockTokens);
    __syncthreads();
    const int t = blk * kBlockTokens + lane;
    float sum = 0.f;
    for (int r = warp; r < n * p.H; r += kMassWarps) {
      const float lse = __ldg(p.lse + (int64_t)q0 * p.H + r);
      const float* q = p.q_lat + ((int64_t)q0 * p.H + r) * kDc;
      const uint16_t* qp = p.q_pe + ((int64_t)q0 * p.H + r) * kDr;
      float s = 0.f;
      for (int c = 0; c < kDc; ++c) s = fmaf(__ldg(q + c), s_x[lane * kMassPitch + c], s);
      for (int c = 0; c < kDr; ++c) s = fmaf(bf16f(__ldg(qp + c)), s_x[lane * kMassPitch + kDc + c], s);
      if (t <= ctx + r / p.H && isfinite(lse)) sum += expf(fmaf(s, p.scale, -lse));
    }
    s_sum[warp][lane] = sum;
    __syncthreads();
    if (warp == 0 && t < len) {
      sum = 0.f;
      for (int w = 0; w < kMassWarps; ++w) sum += s_sum[w][lane];
      float* m = p.mass + (int64_t)page * kPage + (blk & 1) * kBlockTokens + lane;
      *m = t < counted ? fmaf(*m, p.decay, sum) : sum;
    }
  }
}

bool aligned_to(const void* p, uintptr_t a) { return p && ((uintptr_t)p & (a - 1)) == 0; }

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" size_t mla_mass_workspace_bytes(int32_t batch, int32_t n_tokens, int32_t heads, int32_t max_new) {
  if (batch < 0 || batch > kMaxBatch || n_tokens < 0 || heads < 16 || heads > 128 || heads % 16 || max_new < 0 ||
      max_new > n_tokens || (int64_t)n_tokens * heads > (int64_t)INT32_MAX)
    return 0;
  return 256;
}

extern "C" mla_status mla_token_mass(const mla_cache_layer* cache, const float* q_lat, const uint16_t* q_pe,
                                     const float* lse, const int32_t* block_table, int32_t max_pages,
                                     const int32_t* q_start, const int32_t* seq_lens, const int32_t* counted,
                                     int32_t batch, int32_t n_tokens, int32_t heads, int32_t max_new,
                                     float softmax_scale, float decay, void* workspace, size_t workspace_bytes,
                                     float* mass, int32_t* dev_err, mla_stream_t stream) {
  MassParams p;
  if (!cache_check(cache, &p.L, &p.outl)) return MLA_ERR_INVALID_ARG;
  const size_t need = mla_mass_workspace_bytes(batch, n_tokens, heads, max_new);
  if (need == 0 || max_pages < 1 || (int64_t)max_pages * kPage > (int64_t)INT32_MAX) return MLA_ERR_INVALID_ARG;
  if (!(softmax_scale > 0.f) || !isfinite(softmax_scale) || !(decay >= 0.f) || !isfinite(decay)) return MLA_ERR_INVALID_ARG;
  if (batch == 0 || n_tokens == 0) return MLA_OK;
  if (max_new < 1 || !aligned_to(q_lat, 16) || !aligned_to(q_pe, 16) || !aligned_to(lse, 4) || !aligned_to(block_table, 4) ||
      !aligned_to(q_start, 4) || !aligned_to(seq_lens, 4) || (counted && !aligned_to(counted, 4)) || !aligned_to(mass, 4) ||
      !aligned_to(workspace, 256) || workspace_bytes < need || (dev_err && !aligned_to(dev_err, 4)))
    return MLA_ERR_INVALID_ARG;
  p.pool = (const uint8_t*)cache->pool;
  p.lf = cache->latent_fmt;
  p.kf = cache->kpe_fmt;
  p.num_pages = cache->num_pages;
  p.q_lat = q_lat;
  p.q_pe = q_pe;
  p.lse = lse;
  p.table = block_table;
  p.max_pages = max_pages;
  p.q_start = q_start;
  p.seq_lens = seq_lens;
  p.counted = counted;
  p.B = batch;
  p.N = n_tokens;
  p.H = heads;
  p.max_new = max_new;
  p.scale = softmax_scale;
  p.decay = decay;
  p.mass = mass;
  p.dev_err = dev_err;
  static int configured[64] = {0};
  constexpr int kSmem = kBlockTokens * kMassPitch * 4;
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !configured[dev]) {
    const mla_status st = cuda_status(cudaFuncSetAttribute(mass_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem));
    if (st != MLA_OK) return st;
    if (dev >= 0 && dev < 64) configured[dev] = 1;
  }
  const int64_t blocks = (int64_t)max_pages * 2;
  const dim3 grid((unsigned)(blocks < 1024 ? blocks : 1024), batch);
  return cuda_status(launch_pdl(mass_kernel, grid, dim3(kMassThreads), kSmem, (cudaStream_t)stream, p));
}
