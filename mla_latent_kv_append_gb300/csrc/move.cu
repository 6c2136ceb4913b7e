// mla_move_tokens: the kept tokens of a sequence, from its old pages into its
// new ones: token j of the shorter sequence is token kept[j] of the longer one.
//
// A token's codes, scales, zero-points, bound and protected channels keep their
// bits; its chunks change places (their swizzle goes by the token's place in
// its 32-token block).
//
// What bounds it: reading and writing the kept tokens' bytes.  A block takes a
// 32-token block of the destination and writes it whole; codes are gathered in
// 16-byte chunks, the per-token fields (scales lie side by side for 32 tokens) in
// 4-byte words, a lane per token, of which a read moves a 32-byte sector.
//
// Measured: 2048 tokens of 32768 INT8 3.3 us; 32 sequences cut to a quarter, 104000
// tokens INT4 (122 MB in and out) 41 us: a quarter of a block's tokens touch nine
// tenths of its scales' sectors, so that 195 MB move, 4.8 TB/s or 71% of a plain
// copy's rate.  Four blocks an SM with 64 registers; five (48): 47 us.
#include "checks.cuh"
#include "mla_internal.cuh"

namespace mla {
namespace {

constexpr int kMoveThreads = 256, kMoveWarps = kMoveThreads / 32;
constexpr int kMoveAhead = 4;                          // chunks of codes, scales and zero-points of a thread in flight

struct MoveParams {
  uint8_t* pool;
  PageLayout L;
  int num_pages, kpe_fmt, groups, out_groups;          // scale groups; protected channels (0: none)
  int chunk_shift, kchunk_shift;                       // a row's 16-byte chunks: 1 << shift
  int rounds;                                          // of kMoveAhead chunks and scales a thread
  const int32_t* src_table;
  const int32_t* dst_table;
  int max_pages;
  const int32_t *seq_lens, *kept, *lens;
  int max_keep;
  float* mass;
  int32_t* dev_err;
};

__global__ void __launch_bounds__(kMoveThreads, 4) move_kernel(const MoveParams p) {
  __shared__ const uint8_t* s_src[kBlockTokens];       // the token's old block; null: nothing to move
  __shared__ int s_u[kBlockTokens];                    // and its place in it
  const int b = blockIdx.y, blk = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_launch_dependents();
  pdl_wait();
  // all that the lengths do not decide is read along with them
  const int j0 = blk * kBlockTokens;
  const int len = __ldcg(p.seq_lens + b), n = __ldcg(p.lens + b);
  const int page = __ldcg(p.dst_table + (int64_t)b * p.max_pages + blk / 2);
  const int t = warp == 0 && j0 + lane < p.max_keep ? __ldcg(p.kept + (int64_t)b * p.max_keep + j0 + lane) : -1;
  const bool fits = len >= 0 && len <= p.max_pages * kPage && n >= 0 && n <= len;
  if (fits && n == len) return;                        // stays where it is
  if (!fits || n > p.max_keep) {
    if (blk == 0 && tid == 0) set_err(p.dev_err, MLA_DEVERR_SEQLEN);
    return;
  }
  if (j0 >= n) return;
  if (page < 0 || page >= p.num_pages) {
    if (tid == 0) set_err(p.dev_err, MLA_DEVERR_PAGE);
    return;
  }
  uint8_t* dst = p.pool + (int64_t)page * p.L.page_bytes + (blk & 1) * p.L.block_bytes;
  const int count = min(kBlockTokens, n - j0);
  int from = -1;                                       // warp 0: the token's old page
  if (warp == 0) {
    const uint8_t* src = nullptr;
    int u = 0;
    if (lane < count) {
      if (t < 0 || t >= len) {
        set_err(p.dev_err, MLA_DEVERR_SLOT);
      } else {
        from = __ldcg(p.src_table + (int64_t)b * p.max_pages + t / kPage);
        if (from < 0 || from >= p.num_pages) {
          set_err(p.dev_err, MLA_DEVERR_PAGE);
          from = -1;
        } else {
          src = p.pool + (int64_t)from * p.L.page_bytes + (t / kBlockTokens % 2) * p.L.block_bytes;
          u = t % kBlockTokens;
        }
      }
    }
    s_src[lane] = src;
    s_u[lane] = u;
  }
  __syncthreads();
  // Everything of a thread is loaded before anything is stored: one round of memory
  // latency a block, two where a row has 64 chunks or 64 scales (field by field, six
  // rounds: 4.3 us for the one sequence above).  Codes: 16-byte chunks of the rows; a
  // row has a power of two of them.
  auto load_row = [&](uint4& x, int i, int64_t off, int64_t pitch, int sh, auto pos) {
    if (i >= count << sh) return;
    const uint8_t* src = s_src[i >> sh];
    const int u = s_u[i >> sh];
    if (src) x = __ldcg(reinterpret_cast<const uint4*>(src + off + u * pitch) + pos(i & ((1 << sh) - 1), u));
  };
  auto store_row = [&](const uint4& x, int i, int64_t off, int64_t pitch, int sh, auto pos) {
    if (i >= count << sh || !s_src[i >> sh]) return;
    *(reinterpret_cast<uint4*>(dst + off + (i >> sh) * pitch) + pos(i & ((1 << sh) - 1), i >> sh)) = x;
  };
  const uint8_t* src = s_src[lane];
  const int u = s_u[lane];
  // words of a field [groups][32 tokens], lane = token
  auto load_word = [&](uint32_t& x, int g, int64_t off, int groups) {
    if (src && off >= 0 && g < groups) x = __ldcg(reinterpret_cast<const uint32_t*>(src + off) + g * kBlockTokens + u);
  };
  auto store_word = [&](uint32_t x, int g, int64_t off, int groups) {
    if (src && off >= 0 && g < groups) reinterpret_cast<uint32_t*>(dst + off)[g * kBlockTokens + lane] = x;
  };
  auto latent = [](int c, int v) { return latent_chunk_pos(c, v); };
  auto rope = [&](int c, int v) { return kpe_chunk_pos(c, v, p.kpe_fmt); };
  const PageLayout& L = p.L;
  static_assert(kMoveAhead * kMoveWarps >= kNLG && kMoveWarps >= kNKG, "zero-points and the RoPE part's scales in the first round");
  for (int r = 0; r < p.rounds; ++r) {
    const int i0 = r * kMoveAhead * kMoveThreads + tid, g0 = r * kMoveAhead * kMoveWarps + warp;
    const bool first = r == 0;
    uint4 code[kMoveAhead], kpe;
    uint32_t scale[kMoveAhead], zero[kMoveAhead], kscale, bound;
    float mass;
#pragma unroll
    for (int k = 0; k < kMoveAhead; ++k) load_row(code[k], i0 + k * kMoveThreads, L.codes_off, L.codes_row, p.chunk_shift, latent);
#pragma unroll
    for (int k = 0; k < kMoveAhead; ++k) load_word(scale[k], g0 + k * kMoveWarps, L.scale_off, p.groups);
    if (first) {
#pragma unroll
      for (int k = 0; k < kMoveAhead; ++k) load_word(zero[k], g0 + k * kMoveWarps, L.zero_off, kNLG);
      load_row(kpe, tid, L.kpe_off, L.kpe_row, p.kchunk_shift, rope);
      load_word(kscale, warp, L.kpe_scale_off, kNKG);
      load_word(bound, warp, L.bound_off, 1);
      if (from >= 0 && p.mass) mass = __ldcg(p.mass + (int64_t)from * kPage + t % kPage);
    }
#pragma unroll
    for (int k = 0; k < kMoveAhead; ++k) store_row(code[k], i0 + k * kMoveThreads, L.codes_off, L.codes_row, p.chunk_shift, latent);
#pragma unroll
    for (int k = 0; k < kMoveAhead; ++k) store_word(scale[k], g0 + k * kMoveWarps, L.scale_off, p.groups);
    if (first) {
#pragma unroll
      for (int k = 0; k < kMoveAhead; ++k) store_word(zero[k], g0 + k * kMoveWarps, L.zero_off, kNLG);
      store_row(kpe, tid, L.kpe_off, L.kpe_row, p.kchunk_shift, rope);
      store_word(kscale, warp, L.kpe_scale_off, kNKG);
      store_word(bound, warp, L.bound_off, 1);
      if (from >= 0 && p.mass) p.mass[(int64_t)page * kPage + (blk & 1) * kBlockTokens + lane] = mass;
    }
  }
  if (src) {
    for (int g = warp; g < p.out_groups; g += kMoveWarps)
      reinterpret_cast<uint16_t*>(dst + L.outlier_off)[g * kBlockTokens + lane] =
          __ldcg(reinterpret_cast<const uint16_t*>(src + L.outlier_off) + g * kBlockTokens + u);
  }
}

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" mla_status mla_move_tokens(const mla_cache_layer* cache, const int32_t* src_table, const int32_t* seq_lens,
                                      const int32_t* kept, int32_t max_keep, const int32_t* lens,
                                      const int32_t* dst_table, int32_t max_pages, int32_t batch, float* mass,
                                      int32_t* dev_err, mla_stream_t stream) {
  MoveParams p;
  OutlierSet outl;
  if (!cache_check(cache, &p.L, &outl) || batch < 0 || batch > kMaxBatch || max_keep < 1) return MLA_ERR_INVALID_ARG;
  if (max_pages < 1 || (int64_t)max_pages * kPage > (int64_t)INT32_MAX) return MLA_ERR_INVALID_ARG;
  if (batch == 0) return MLA_OK;
  if (!ok4(src_table) || !ok4(seq_lens) || !ok4(kept) || !ok4(lens) || !ok4(dst_table) || (mass && !ok4(mass)) ||
      (dev_err && !ok4(dev_err)))
    return MLA_ERR_INVALID_ARG;
  p.pool = (uint8_t*)cache->pool;
  p.num_pages = cache->num_pages;
  p.kpe_fmt = cache->kpe_fmt;
  p.groups = kDc / latent_group_size(cache->latent_fmt);
  p.out_groups = cache->latent_fmt == MLA_FMT_INT8_OUTLIER ? kNOut : 0;
  auto log2_chunks = [](int64_t row) {
    int n = 0;
    while ((16 << n) < row) ++n;
    return n;
  };
  p.chunk_shift = log2_chunks(p.L.codes_row);
  p.kchunk_shift = log2_chunks(p.L.kpe_row);
  // the RoPE part's 8 chunks of 32 tokens and everything but codes and scales fit one round
  const int chunks = kBlockTokens << p.chunk_shift, a_round = kMoveAhead * kMoveThreads, words = kMoveAhead * kMoveWarps;
  const int by_codes = (chunks + a_round - 1) / a_round, by_scales = (p.groups + words - 1) / words;
  p.rounds = by_codes > by_scales ? by_codes : by_scales;
  p.src_table = src_table;
  p.dst_table = dst_table;
  p.max_pages = max_pages;
  p.seq_lens = seq_lens;
  p.kept = kept;
  p.lens = lens;
  p.max_keep = max_keep;
  p.mass = mass;
  p.dev_err = dev_err;
  const int64_t cap = (int64_t)max_pages * kPage < max_keep ? (int64_t)max_pages * kPage : max_keep;
  const dim3 grid((unsigned)((cap + kBlockTokens - 1) / kBlockTokens), batch);
  return cuda_status(launch_pdl(move_kernel, grid, dim3(kMoveThreads), 0, (cudaStream_t)stream, p));
}
