// Shared by the translation units of mla_token_mass (mass*.cu).
#pragma once

#include "mla_internal.cuh"

namespace mla {

constexpr int kMassKeys = 128;                         // keys per tile
constexpr int kMassMaxRows = 128;                      // most rows per pass
constexpr int kMassMaxGrid = 512;                      // most blocks
// Cached values are multiplied by kKeyGain, queries (with the softmax scale and
// log2 e) by kQueryGain: halves keep 22 bits of values down to 2^-7 and 2^-8, and stay
// finite up to 4094 and 2047.
constexpr float kKeyGain = 16.f, kQueryGain = 32.f, kMassUngain = 1.f / (kKeyGain * kQueryGain);

// An accumulation in TMEM cuts the sum off to 24 bits, towards 0: half a last place of
// it on average, 2^-24 E[1/m] = 4.3e-8 of the sum for its mantissa m spread as in
// nature; products are cut off one by one before, which takes a fifth of that back where
// they are of both signs, as a query's and a latent's are.  (Scores of 20 nats were off by
// 2.9 to 3.4e-8 for each accumulation from their channels on, 2.6 to 5.2e-8 with products
// of one sign; K-steps of zeros cut nothing off.)  The queries' channels give that mean
// back, each as often as it is cut off: mass_prep_kernel.
constexpr float kMassCut = 3.4e-8f;

// TMEM columns of the scores of a pass of R rows.
__host__ __device__ constexpr int mass_columns(int R) { return R <= 64 ? 64 : kMassMaxRows; }

// One sequence with queries and tokens, in the order of the batch.  Its rows r =
// i H + h are cut into row blocks of R; a pass is a row block of a key tile, the
// passes of a tile lie side by side.  A pass costs mass_cost(its rows) units.
struct __align__(16) MassSeq {
  int64_t unit0;          // units before this sequence's
  int64_t pass0;          // passes before this sequence's
  int32_t b, q0, n, len;  // batch index, first query row (token), queries, cached tokens
  int32_t counted;        // tokens whose mass is up to date
  int32_t tiles, blocks;  // key tiles, row blocks
  int32_t tile_cost;      // units of a key tile
  int32_t heads, pad[3];
};
static_assert(sizeof(MassSeq) == 64, "four 16-byte loads");

struct MassCounts {
  int64_t units, passes;
  int32_t seqs, pad;
};

// Units of a pass with this many rows: an MMA takes about 75 cycles however few
// there are, 92 with 128 (24 drafts of up to 5 tokens at 64 heads: 98 us a call when
// passes were counted by their rows alone, 77 so).
__host__ __device__ constexpr int mass_cost(int rows) { return 4 + (rows + 31) / 32; }

// Run x of G equal runs over U units begins here; the run that holds unit u.
__device__ __forceinline__ int64_t mass_run(int64_t U, int x, int G) {
  if (U <= (int64_t)(0xFFFFFFFFu / 1024u)) return (uint32_t)U * (uint32_t)x / (uint32_t)G;
  return U * x / G;
}
__device__ __forceinline__ int mass_run_of(int64_t U, int64_t u, int G) { return (int)(((u + 1) * G - 1) / U); }

struct MassParams {
  const uint8_t* pool;
  PageLayout L;
  OutlierSet outl;
  int num_pages;
  const float* q_lat;
  const uint16_t* q_pe;
  const float* lse;
  const int32_t* table;
  int max_pages;
  const int32_t *q_start, *seq_lens, *counted;
  int B, N, H, max_new;
  float scale_log2, decay;
  float* mass;
  int32_t* dev_err;
  uint64_t wait_ns;
  int R, grid;
  int split_lat, split_kpe;                            // cached values have low halves (all formats but bf16)
  int few, unit_tokens;                                // 16 rows (mass_few.cuh); cached tokens of a key tile
  int query_pieces, raw_slots;                         // pieces of the queries and raw blocks in shared memory
  int64_t rows;                                        // N H
  // workspace
  MassCounts* counts;
  MassSeq* seqs;
  int32_t* done;          // [kMassMaxGrid] passes finished of the tile that a run ends in
  float* parts;           // [2 kMassMaxGrid][128]
  uint8_t* q_tiles;       // [hi, lo][9][rows][64] fp16, swizzled
};

// The kernel over the key tiles, by latent format (one translation unit each);
// MLA_ERR_UNSUPPORTED for another unit's formats.
mla_status launch_mass_bf16(const MassParams& p, int lf, int kf, cudaStream_t stream);
mla_status launch_mass_int8(const MassParams& p, int lf, int kf, cudaStream_t stream);
mla_status launch_mass_int8_blocks(const MassParams& p, int lf, int kf, cudaStream_t stream);
mla_status launch_mass_int4(const MassParams& p, int lf, int kf, cudaStream_t stream);

}  // namespace mla
