// mla_token_mass: argument checks, the device plan and the queries' halves
// (the kernel itself is in mass.cuh).
#include <cuda_fp16.h>
#include <math.h>

#include "checks.cuh"
#include "mass_params.cuh"
#include "scan.cuh"

namespace mla {
namespace {

constexpr int kPieces = (kDc + kDr) / 8;               // of 8 channels per row
constexpr int kPrepRows = 4, kPrepThreads = kPrepRows * kPieces;     // a thread per piece
static_assert(kPrepThreads % 32 == 0 && kPrepRows <= kPrepThreads / 32, "whole warps, a warp for each row's sequence");

// Block 0: which sequences take part, and where their units begin.
__device__ void plan_mass(const MassParams& p) {
  __shared__ int64_t red[kPrepThreads / 32];
  const int tid = threadIdx.x;
  for (int i = tid; i < p.grid; i += kPrepThreads) p.done[i] = 0;
  bool bad = false;
  for (int i = tid; i < p.B; i += kPrepThreads) {
    const int lo = __ldcg(p.q_start + i), hi = __ldcg(p.q_start + i + 1);
    bad |= lo < 0 || hi < lo || hi > p.N;
  }
  bad = __syncthreads_or(bad);
  const int per = (p.B + kPrepThreads - 1) / kPrepThreads, b0 = tid * per;
  MassSeq s[1];
  int64_t units = 0, passes = 0;
  int count = 0, err = bad ? MLA_DEVERR_SEQLEN : 0;
  // twice: sums first, then the records
  int64_t unit0 = 0, pass0 = 0, at = 0, total_u = 0, total_p = 0, total_c = 0;
  for (int round = 0; round < 2; ++round) {
    for (int k = 0; k < per && b0 + k < p.B && !bad; ++k) {
      const int b = b0 + k;
      MassSeq& r = s[0];
      r.b = b;
      r.q0 = __ldcg(p.q_start + b);
      r.n = __ldcg(p.q_start + b + 1) - r.q0;
      r.len = __ldcg(p.seq_lens + b);
      if (r.n == 0) continue;
      r.counted = p.counted ? __ldcg(p.counted + b) : r.len - r.n;
      if (r.n > p.max_new || r.len < 0 || r.len > p.max_pages * kPage || (r.len > 0 && (r.len < r.n || r.counted < 0 || r.counted > r.len))) {
        err |= MLA_DEVERR_SEQLEN;
        continue;
      }
      if (r.len == 0) continue;
      const int rows = r.n * p.H;
      r.heads = p.H;
      r.tiles = (int)(((int64_t)r.len + p.unit_tokens - 1) / p.unit_tokens);
      r.blocks = (rows + p.R - 1) / p.R;
      r.tile_cost = (r.blocks - 1) * mass_cost(p.R) + mass_cost(rows - (r.blocks - 1) * p.R);
      const int64_t u = (int64_t)r.tiles * r.tile_cost, q = (int64_t)r.tiles * r.blocks;
      if (round == 0) {
        units += u;
        passes += q;
        ++count;
      } else {
        r.unit0 = unit0;
        r.pass0 = pass0;
        r.pad[0] = r.pad[1] = r.pad[2] = 0;
        p.seqs[at++] = r;
        unit0 += u;
        pass0 += q;
      }
    }
    if (round == 0) {
      unit0 = block_scan<kPrepThreads>(units, red, &total_u);
      pass0 = block_scan<kPrepThreads>(passes, red, &total_p);
      at = block_scan<kPrepThreads>((int64_t)count, red, &total_c);
    }
  }
  if (err) set_err(p.dev_err, err);
  if (tid == 0) {
    p.counts->units = total_u;
    p.counts->passes = total_p;
    p.counts->seqs = (int)total_c;
  }
}

// All lanes of a warp: the sequence that row r belongs to, and the rows of its row
// block there.  Any q_start: a batch that does not fit is refused by the plan.
__device__ __forceinline__ int rows_beside(const MassParams& p, int r) {
  const int lane = threadIdx.x & 31, token = (int)((uint32_t)r / (uint32_t)p.H);
  int a = 0, n = p.B;                                  // the answer is in [a, a + n)
  for (;;) {
    const int step = (n + 31) / 32, at = a + lane * step;
    const bool in = at < a + n;
    const int lo = in ? __ldcg(p.q_start + at) : 0, next = in ? __ldcg(p.q_start + at + 1) : 0;
    const int c = max(__popc(__ballot_sync(0xffffffffu, in && lo <= token)), 1);
    if (step == 1) {
      const int r0 = __shfl_sync(0xffffffffu, lo, c - 1), n_q = __shfl_sync(0xffffffffu, next, c - 1) - r0;
      return min(p.R, n_q * p.H - ((r - r0 * p.H) & -p.R));           // R is a power of two
    }
    const int na = a + (c - 1) * step;
    n = min(step, a + n - na);
    a = na;
  }
}

// The queries times the softmax scale, log2 e and kQueryGain, as two halves:
// piece kb of 64 channels, all rows of it side by side, in the 128-byte swizzle.
// A row whose lse is not finite is 0 (it adds nothing).
//
// What the MMAs' accumulations cut off on average (kMassCut) is given back here: a
// channel's part of a score is cut at every accumulation from its own K-step's on, so
// it is multiplied by 1 + kMassCut times their number.  That holds for scores that
// come from any channels: the mean of what is cut off is linear in them.  K-steps where
// the row's query is 0 are not counted.
__global__ void __launch_bounds__(kPrepThreads) mass_prep_kernel(const MassParams p) {
  __shared__ uint32_t s_any[2][kPrepThreads / 32 + 2];               // the pieces that are not 0, bit by bit
  __shared__ bool s_apart[2][kPrepRows];
  pdl_launch_dependents();
  pdl_wait();
  if (blockIdx.x == 0) {
    plan_mass(p);
    return;
  }
  const float gain = p.scale_log2 * kQueryGain;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int mine = threadIdx.x / kPieces, c = threadIdx.x - mine * kPieces;
  int turn = 0;
  for (int64_t row0 = (int64_t)(blockIdx.x - 1) * kPrepRows; row0 < p.rows; row0 += (int64_t)(gridDim.x - 1) * kPrepRows, turn ^= 1) {
    const int64_t r = row0 + mine;
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    bool live = false;
    if (r < p.rows) {
      live = fabsf(__ldcg(p.lse + r)) < INFINITY;
      if (c < kDc / 8) {
        const float4* src = reinterpret_cast<const float4*>(p.q_lat + r * kDc) + 2 * c;
        *reinterpret_cast<float4*>(v) = __ldcg(src);
        *reinterpret_cast<float4*>(v + 4) = __ldcg(src + 1);
      } else {
        const uint4 w = __ldcg(reinterpret_cast<const uint4*>(p.q_pe + r * kDr) + (c - kDc / 8));
        v[0] = bf16lo(w.x), v[1] = bf16hi(w.x), v[2] = bf16lo(w.y), v[3] = bf16hi(w.y);
        v[4] = bf16lo(w.z), v[5] = bf16hi(w.z), v[6] = bf16lo(w.w), v[7] = bf16hi(w.w);
      }
    }
    // whether the low halves' products have columns of their own: always up to 32 rows a pass
    if (warp < kPrepRows && p.R > 32) {
      const bool apart = 2 * rows_beside(p, (int)min(row0 + warp, p.rows - 1)) <= mass_columns(p.R);
      if (lane == 0) s_apart[turn][warp] = apart;
    }
    bool any = false;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      v[k] = live ? v[k] * gain : 0.f;
      any |= v[k] != 0.f;
    }
    const uint32_t some = __ballot_sync(0xffffffffu, any);
    if (lane == 0) s_any[turn][warp] = some;
    __syncthreads();
    if (r >= p.rows) continue;                         // the next turn writes the other arrays: one barrier is enough
    // K-steps of 16 channels that are not 0, 32 of the latent and 4 of the RoPE part; bit
    // 2 s: step s (a row's bits begin at an even one)
    const uint32_t* word = s_any[turn] + mine * kPieces / 32;
    const int shift = mine * kPieces % 32;
    uint32_t steps[3];
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      const uint32_t bits = __funnelshift_r(word[i], word[i + 1], shift);
      steps[i] = (bits | bits >> 1) & 0x55555555u;
    }
    steps[2] &= 0xFFu;
    const bool apart = p.R <= 32 || s_apart[turn][mine];
    const int lat = 1 + !apart + p.split_lat, kpe = 1 + !apart + p.split_kpe;      // MMAs of a K-step on the scores' columns
    // The MMAs of 64 channels (4 K-steps, 8 bits) follow one another by product: high
    // halves first, from the channel's own step on; then the others, all four steps;
    // then the 64-channel pieces behind.
    const int i = c >> 5, at = c & 30, block = c & 24, m = i < 2 ? lat : kpe;
    const uint32_t own = i == 0 ? steps[0] : (i == 1 ? steps[1] : steps[2]);
    const uint32_t here = own & (0xFFu << block), behind = block == 24 ? 0u : own & (0xFFFFFFFFu << (block + 8));
    int cuts = __popc(here & (0xFFFFFFFFu << at)) + (m - 1) * __popc(here) + m * __popc(behind);
    if (i == 0) cuts += lat * __popc(steps[1]);
    if (i < 2) cuts += kpe * __popc(steps[2]);
    const float back = kMassCut * (float)cuts;
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float a = fmaf(v[2 * k], back, v[2 * k]), b = fmaf(v[2 * k + 1], back, v[2 * k + 1]);
      const __half2 h = __floats2half2_rn(a, b), l = __floats2half2_rn(a - __low2float(h), b - __high2float(h));
      hi[k] = *reinterpret_cast<const uint32_t*>(&h);
      lo[k] = *reinterpret_cast<const uint32_t*>(&l);
    }
    uint8_t* dst = p.q_tiles + ((int64_t)(c / 8) * p.rows + r) * 128 + (((c & 7) ^ (int)(r & 7)) << 4);
    *reinterpret_cast<uint4*>(dst) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<uint4*>(dst + (int64_t)9 * p.rows * 128) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  }
}

bool sizes_ok(int32_t batch, int32_t n_tokens, int32_t heads, int32_t max_new) {
  return batch >= 0 && batch <= kMaxBatch && n_tokens >= 0 && heads >= 16 && heads <= 128 && heads % 16 == 0 && max_new >= 0 &&
         max_new <= n_tokens && (int64_t)n_tokens * heads <= (int64_t)INT32_MAX;
}

// Places the workspace's arrays; its size.
int64_t carve(void* base, int B, int64_t rows, MassParams* p) {
  char* c = (char*)base;
  auto take = [&](int64_t bytes) {
    char* at = c;
    c += align256(bytes);
    return at;
  };
  p->counts = (MassCounts*)take(sizeof(MassCounts));
  p->seqs = (MassSeq*)take((int64_t)(B + 1) * sizeof(MassSeq));
  p->done = (int32_t*)take(kMassMaxGrid * 4);
  p->parts = (float*)take((int64_t)2 * kMassMaxGrid * kMassKeys * 4);
  p->q_tiles = (uint8_t*)take(rows * 9 * 256);
  return c - (char*)base;
}

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" size_t mla_mass_workspace_bytes(int32_t batch, int32_t n_tokens, int32_t heads, int32_t max_new) {
  if (!sizes_ok(batch, n_tokens, heads, max_new)) return 0;
  MassParams p;
  return (size_t)carve(nullptr, batch, (int64_t)n_tokens * heads, &p);
}

extern "C" mla_status mla_token_mass(const mla_cache_layer* cache, const float* q_lat, const uint16_t* q_pe,
                                     const float* lse, const int32_t* block_table, int32_t max_pages,
                                     const int32_t* q_start, const int32_t* seq_lens, const int32_t* counted,
                                     int32_t batch, int32_t n_tokens, int32_t heads, int32_t max_new,
                                     float softmax_scale, float decay, void* workspace, size_t workspace_bytes,
                                     float* mass, int32_t* dev_err, mla_stream_t stream) {
  MassParams p;
  if (!cache_check(cache, &p.L, &p.outl) || !sizes_ok(batch, n_tokens, heads, max_new)) return MLA_ERR_INVALID_ARG;
  if (max_pages < 1 || (int64_t)max_pages * kPage > (int64_t)INT32_MAX) return MLA_ERR_INVALID_ARG;
  if (!(softmax_scale > 0.f) || !isfinite(softmax_scale) || !(decay >= 0.f) || !isfinite(decay)) return MLA_ERR_INVALID_ARG;
  if (batch == 0 || n_tokens == 0) return MLA_OK;
  if (max_new < 1 || !aligned_to(q_lat, 16) || !aligned_to(q_pe, 16) || !aligned_to(lse, 4) || !aligned_to(block_table, 4) ||
      !aligned_to(q_start, 4) || !aligned_to(seq_lens, 4) || (counted && !aligned_to(counted, 4)) || !aligned_to(mass, 4) ||
      !aligned_to(workspace, 256) || (dev_err && !aligned_to(dev_err, 4)))
    return MLA_ERR_INVALID_ARG;
  p.rows = (int64_t)n_tokens * heads;
  if ((int64_t)workspace_bytes < carve(workspace, batch, p.rows, &p)) return MLA_ERR_INVALID_ARG;
  p.pool = (const uint8_t*)cache->pool;
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
  p.scale_log2 = softmax_scale * 1.4426950408889634f;
  p.decay = decay;
  p.mass = mass;
  p.dev_err = dev_err;
  p.wait_ns = wait_limit_ns();
  const int64_t most = (int64_t)max_new * heads;
  // Rows of a pass: no more than the longest sequence has (32 x 32768 tokens INT4 at 32
  // rows: 206 us in passes of 32, 259 of 128), and 128 where there are more (24 drafts of
  // 5 tokens at 64 heads: 79 us, 104 in passes of 64; a window of 32 at 16 heads: 94, 124).
  p.R = most <= 16 ? 16 : (most <= 32 ? 32 : (most <= 64 ? 64 : kMassMaxRows));
  const int sms = device_sm_count();
  p.grid = sms < 1 ? 1 : (sms < kMassMaxGrid ? sms : kMassMaxGrid);
  // 16 rows on mma.sync, in the formats that it has: one sequence of 4096 tokens takes 11
  // us there and 14 to 15 on tcgen05 (bf16, INT8), of 32768 16.3 and 18.6 (INT8) or 17.4
  // and 17.6 (bf16), 32 of 500 17 and 20, 32 of 16384 INT8 108 and 109, 32 of 32768 INT4
  // 207 and 203.  Only long batches in bf16 lose (32 of 16384: 136 and 107; three products
  // of bf16 parts where tcgen05 takes two of fp16 ones), and how long they are is known
  // on the device alone.
  p.few = most <= 16 && (cache->latent_fmt == MLA_FMT_BF16 || cache->latent_fmt == MLA_FMT_INT8_SYM ||
                         cache->latent_fmt == MLA_FMT_INT4_ASYM || cache->latent_fmt == MLA_FMT_INT4_SYM);
  // the unit that the kernels copy at a time (FewShape::kBlocks), or a tile of theirs
  p.unit_tokens = p.few ? (p.L.block_bytes < 20000 ? kPage : kBlockTokens) : kMassKeys;
  p.split_lat = cache->latent_fmt != MLA_FMT_BF16;
  p.split_kpe = cache->kpe_fmt != MLA_FMT_BF16;
  // the few rows' kernel makes its queries' fragments itself: the plan alone
  const int64_t want = p.few ? 1 : 1 + (p.rows + kPrepRows - 1) / kPrepRows;
  const mla_status st = cuda_status(launch_pdl(mass_prep_kernel, dim3((unsigned)(want < 4 * p.grid ? want : 4 * p.grid)),
                                               dim3(kPrepThreads), 0, (cudaStream_t)stream, p));
  if (st != MLA_OK) return st;
  switch (cache->latent_fmt) {
    case MLA_FMT_BF16: return launch_mass_bf16(p, cache->latent_fmt, cache->kpe_fmt, (cudaStream_t)stream);
    case MLA_FMT_INT8_SYM: return launch_mass_int8(p, cache->latent_fmt, cache->kpe_fmt, (cudaStream_t)stream);
    case MLA_FMT_INT4_ASYM:
    case MLA_FMT_INT4_SYM: return launch_mass_int4(p, cache->latent_fmt, cache->kpe_fmt, (cudaStream_t)stream);
    default: return launch_mass_int8_blocks(p, cache->latent_fmt, cache->kpe_fmt, (cudaStream_t)stream);
  }
}
