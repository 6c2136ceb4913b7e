// mla_chunk_attention: causal attention of a ragged batch of new tokens over
// the paged latent cache, from the projected queries to the per-head outputs.
//
// The simplest form that is right for every case: one block per (token,
// head), everything in fp32.  The query is absorbed into the latent space
// (q_lat = q_nope W_UK), the keys stream through shared memory 32 tokens at
// a time with an online softmax, and the latent output is projected by W_UV.
#include <math.h>

#include "dequant.cuh"
#include "mla_internal.cuh"

namespace mla {
namespace {

constexpr int kSimpleThreads = 256;
constexpr int kSimpleStride = kDc + kDr + 1;

struct ChunkParams {
  const uint8_t* pool;
  PageLayout L;
  OutlierSet outl;
  int num_pages;
  const uint16_t *qn, *qp;
  int64_t qn_tok, qn_head, qp_tok, qp_head;
  const uint16_t *w_uk, *w_uv;
  const int32_t* block_table;
  int max_pages;
  const int32_t *q_start, *seq_lens;
  int B, N, H, max_new;
  float scale_log2;
  uint16_t* o;
  int32_t* dev_err;
};

template <int LF, int KF>
__global__ void __launch_bounds__(kSimpleThreads) chunk_simple_kernel(const ChunkParams p) {
  extern __shared__ float cs_smem[];
  float* s_q = cs_smem;                      // [576]
  float* s_x = s_q + kDc + kDr;              // [32][577]
  float* s_p = s_x + 32 * kSimpleStride;     // [32]
  float* s_o = s_p + 32;                     // [512]
  pdl_launch_dependents();
  pdl_wait();
  const int tok = blockIdx.x, h = blockIdx.y, tid = threadIdx.x;
  if (tok >= p.q_start[p.B]) return;
  int b = 0;
  while (b < p.B && !(p.q_start[b] <= tok && tok < p.q_start[b + 1])) ++b;
  if (b == p.B) return;
  const int q0 = p.q_start[b], n = p.q_start[b + 1] - q0, len = p.seq_lens[b];
  uint16_t* out = p.o + ((int64_t)tok * p.H + h) * kDv;
  const bool bad = q0 < 0 || p.q_start[b + 1] > p.N || n > p.max_new || len < 0 || (len > 0 && len < n) ||
                   (int64_t)len > (int64_t)p.max_pages * kPage;
  if (bad || len == 0) {
    if (bad && tid == 0) set_err(p.dev_err, MLA_DEVERR_SEQLEN);
    if (tid < kDv) out[tid] = 0;
    return;
  }
  const int pos = len - n + tok - q0;
  const uint16_t* qn = p.qn + tok * p.qn_tok + h * p.qn_head;
  const uint16_t* qp = p.qp + tok * p.qp_tok + h * p.qp_head;
  for (int c = tid; c < kDc; c += kSimpleThreads) {
    float a = 0.f;
    for (int d = 0; d < kDn; ++d) a = fmaf(bf16f(qn[d]), bf16f(p.w_uk[((int64_t)h * kDn + d) * kDc + c]), a);
    s_q[c] = a;
  }
  if (tid < kDr) s_q[kDc + tid] = bf16f(qp[tid]);
  float m = -INFINITY, l = 0.f, acc[2] = {0.f, 0.f};
  for (int t0 = 0; t0 <= pos; t0 += 32) {
    const int page = p.block_table[(int64_t)b * p.max_pages + t0 / kPage];
    if (page < 0 || page >= p.num_pages) {
      if (tid == 0) set_err(p.dev_err, MLA_DEVERR_PAGE);
      continue;
    }
    const uint8_t* blk = p.pool + page * p.L.page_bytes + ((t0 >> 5) & 1) * p.L.block_bytes;
    __syncthreads();
    for (int i = tid; i < 32 * (kLatentUnits + kKpeUnits); i += kSimpleThreads) {
      const int u = i & 31, c = i >> 5;
      if (t0 + u > pos) continue;
      float x[32];
      if (c < kLatentUnits) {
        RawUnit<LF, false> r;
        load_unit<LF, false>(blk, p.L, u, c, r);
        convert_unit<LF, false>(r, x);
        patch_outliers<LF>(blk, p.L, p.outl, u, c, x);
      } else {
        RawUnit<KF, true> r;
        load_unit<KF, true>(blk, p.L, u, c - kLatentUnits, r);
        convert_unit<KF, true>(r, x);
      }
      for (int k = 0; k < 32; ++k) s_x[u * kSimpleStride + 32 * c + k] = x[k];
    }
    __syncthreads();
    for (int u = tid >> 5; u < 32; u += kSimpleThreads / 32) {
      float a = 0.f;
      if (t0 + u <= pos)
        for (int c = tid & 31; c < kDc + kDr; c += 32) a = fmaf(s_q[c], s_x[u * kSimpleStride + c], a);
      for (int o = 16; o; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
      if ((tid & 31) == 0) s_p[u] = t0 + u <= pos ? a * p.scale_log2 : -INFINITY;
    }
    __syncthreads();
    float mx = m;
    for (int u = 0; u < 32; ++u) mx = fmaxf(mx, s_p[u]);
    const float alpha = exp2f(m - mx);
    l *= alpha;
    acc[0] *= alpha;
    acc[1] *= alpha;
    for (int u = 0; u < 32 && t0 + u <= pos; ++u) {
      const float w = exp2f(s_p[u] - mx);
      l += w;
      acc[0] = fmaf(w, s_x[u * kSimpleStride + tid], acc[0]);
      acc[1] = fmaf(w, s_x[u * kSimpleStride + tid + 256], acc[1]);
    }
    m = mx;
  }
  const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
  s_o[tid] = acc[0] * inv;
  s_o[tid + 256] = acc[1] * inv;
  __syncthreads();
  if (tid < kDv) {
    float a = 0.f;
    for (int c = 0; c < kDc; ++c) a = fmaf(s_o[c], bf16f(p.w_uv[((int64_t)h * kDc + c) * kDv + tid]), a);
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;\n" : "=r"(r) : "f"(0.f), "f"(a));
    out[tid] = (uint16_t)r;
  }
}

template <int LF, int KF>
mla_status launch_simple(const ChunkParams& p, cudaStream_t stream) {
  const int smem = (int)sizeof(float) * (kDc + kDr + 32 * kSimpleStride + 32 + kDc);
  const mla_status st =
      cuda_status(cudaFuncSetAttribute(chunk_simple_kernel<LF, KF>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
  if (st != MLA_OK) return st;
  return cuda_status(launch_pdl(chunk_simple_kernel<LF, KF>, dim3(p.N, p.H), dim3(kSimpleThreads), smem, stream, p));
}

bool al(const void* p, uintptr_t a) { return p && ((uintptr_t)p & (a - 1)) == 0; }

bool sizes_ok(int batch, int n_tokens, int heads, int max_new, int64_t kv_tokens) {
  return batch >= 0 && batch <= kMaxBatch && n_tokens >= 0 && heads >= 16 && heads <= 128 && heads % 16 == 0 &&
         (int64_t)n_tokens * heads <= (int64_t)INT32_MAX && max_new >= 0 && max_new <= n_tokens && kv_tokens >= 0 &&
         kv_tokens <= (int64_t)INT32_MAX;
}

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" {

size_t mla_chunk_workspace_bytes(int32_t batch, int32_t n_tokens, int32_t heads, int32_t max_new, int64_t kv_tokens) {
  if (!sizes_ok(batch, n_tokens, heads, max_new, kv_tokens)) return 0;
  return 256;
}

mla_status mla_chunk_attention(const mla_cache_layer* cache, const uint16_t* q_nope, int64_t qn_token_stride,
                               int64_t qn_head_stride, const uint16_t* q_pe, int64_t qp_token_stride,
                               int64_t qp_head_stride, const uint16_t* w_uk, const uint16_t* w_uv,
                               const int32_t* block_table, int32_t max_pages, const int32_t* q_start,
                               const int32_t* seq_lens, int32_t batch, int32_t n_tokens, int32_t heads,
                               int32_t max_new, int64_t kv_tokens, float softmax_scale, void* workspace,
                               size_t workspace_bytes_, uint16_t* o, int32_t* dev_err, mla_stream_t stream) {
  ChunkParams p;
  if (!cache_check(cache, &p.L, &p.outl) || !sizes_ok(batch, n_tokens, heads, max_new, kv_tokens))
    return MLA_ERR_INVALID_ARG;
  if (!(softmax_scale > 0.f) || !isfinite(softmax_scale)) return MLA_ERR_INVALID_ARG;
  if (batch == 0 || n_tokens == 0) return MLA_OK;
  if (max_pages < 1 || (int64_t)max_pages * kPage > (int64_t)INT32_MAX || max_new < 1) return MLA_ERR_INVALID_ARG;
  const int64_t strides[4] = {qn_token_stride, qn_head_stride, qp_token_stride, qp_head_stride};
  for (int i = 0; i < 4; ++i)
    if (strides[i] < 0 || strides[i] % 8) return MLA_ERR_INVALID_ARG;
  if (!al(q_nope, 16) || !al(q_pe, 16) || !al(w_uk, 16) || !al(w_uv, 16) || !al(block_table, 4) || !al(q_start, 4) ||
      !al(seq_lens, 4) || !al(workspace, 256) || !al(o, 16) || (dev_err && !al(dev_err, 4)))
    return MLA_ERR_INVALID_ARG;
  if (workspace_bytes_ < mla_chunk_workspace_bytes(batch, n_tokens, heads, max_new, kv_tokens))
    return MLA_ERR_INVALID_ARG;
  p.pool = (const uint8_t*)cache->pool;
  p.num_pages = cache->num_pages;
  p.qn = q_nope;
  p.qp = q_pe;
  p.qn_tok = qn_token_stride;
  p.qn_head = qn_head_stride;
  p.qp_tok = qp_token_stride;
  p.qp_head = qp_head_stride;
  p.w_uk = w_uk;
  p.w_uv = w_uv;
  p.block_table = block_table;
  p.max_pages = max_pages;
  p.q_start = q_start;
  p.seq_lens = seq_lens;
  p.B = batch;
  p.N = n_tokens;
  p.H = heads;
  p.max_new = max_new;
  p.scale_log2 = softmax_scale * 1.4426950408889634f;
  p.o = o;
  p.dev_err = dev_err;
  const int lf = cache->latent_fmt, kf = cache->kpe_fmt;
#define MLA_CHUNK_CASE(A, K) \
  if (lf == A && kf == K) return launch_simple<A, K>(p, (cudaStream_t)stream);
  MLA_CHUNK_CASE(MLA_FMT_BF16, MLA_FMT_BF16)
  MLA_CHUNK_CASE(MLA_FMT_BF16, MLA_FMT_INT8_SYM)
  MLA_CHUNK_CASE(MLA_FMT_BF16, MLA_FMT_INT4_SYM)
  MLA_CHUNK_CASE(MLA_FMT_INT8_SYM, MLA_FMT_BF16)
  MLA_CHUNK_CASE(MLA_FMT_INT8_SYM, MLA_FMT_INT8_SYM)
  MLA_CHUNK_CASE(MLA_FMT_INT8_SYM, MLA_FMT_INT4_SYM)
  MLA_CHUNK_CASE(MLA_FMT_INT4_ASYM, MLA_FMT_BF16)
  MLA_CHUNK_CASE(MLA_FMT_INT4_ASYM, MLA_FMT_INT8_SYM)
  MLA_CHUNK_CASE(MLA_FMT_INT4_ASYM, MLA_FMT_INT4_SYM)
  MLA_CHUNK_CASE(MLA_FMT_INT4_SYM, MLA_FMT_BF16)
  MLA_CHUNK_CASE(MLA_FMT_INT4_SYM, MLA_FMT_INT8_SYM)
  MLA_CHUNK_CASE(MLA_FMT_INT4_SYM, MLA_FMT_INT4_SYM)
  MLA_CHUNK_CASE(MLA_FMT_INT8_G8, MLA_FMT_INT8_SYM)
  MLA_CHUNK_CASE(MLA_FMT_INT8_G32, MLA_FMT_INT8_SYM)
  MLA_CHUNK_CASE(MLA_FMT_INT8_G64, MLA_FMT_INT8_SYM)
  MLA_CHUNK_CASE(MLA_FMT_INT8_TOKEN, MLA_FMT_INT8_SYM)
  MLA_CHUNK_CASE(MLA_FMT_INT8_OUTLIER, MLA_FMT_BF16)
  MLA_CHUNK_CASE(MLA_FMT_INT8_OUTLIER, MLA_FMT_INT8_SYM)
#undef MLA_CHUNK_CASE
  return MLA_ERR_UNSUPPORTED;
}

}  // extern "C"
