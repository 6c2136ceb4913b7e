// Shared by the translation units of mla_chunk_attention (chunk*.cu).
#pragma once

#include "mla_internal.cuh"

namespace mla {

constexpr int kChunkShort = MLA_CHUNK_SHORT;
constexpr int kKeyTile = kPage;              // short path: keys per tile, one page
constexpr int kItemCost = 4;                 // 38 drafts of 2 and 2 chunks of 1023: 145 us a call with 0, 133 with 2, 129 with 4, 130 with 6;
                                             // 24 drafts of 5 at 64 heads 174, 167, 165, 167; 32 x 32768 201, 200, 202, 203
constexpr int kQBlocks = (kDc + kDr) / 64;   // 9 blocks of 64 channels

// One sequence of the short path (at most kChunkShort new tokens), in the
// order of the batch.  Its rows r = i H + h (new token i, head h) are cut
// into row tiles of R rows; a unit of work is one key tile of one row tile, after
// kItemCost units for what a row tile costs by itself (its queries' way in, its
// output's way out, a pipeline that runs empty in between): without these a run
// of short contexts takes twice as long as one out of the middle of a long one.
struct __align__(16) ShortSeq {
  int64_t unit0;          // units before this sequence's
  int32_t b, q0, n, len;  // batch index, first token row, new tokens, cached tokens (the new ones included)
  int32_t item0;          // row tiles before this sequence's
  int32_t tok0;           // short-path tokens before this sequence's
  int32_t tiles;          // key tiles
  int32_t items;          // row tiles
};
static_assert(sizeof(ShortSeq) == 48, "three 16-byte loads");

// One sequence of the long path.  Its new tokens are cut into pairs of 128-row
// query tiles; a unit is one 128-key tile of one pair of one head, after
// kPairCost units for what a pair costs by itself.
struct __align__(16) LongSeq {
  int64_t unit0;          // units before this sequence's
  int32_t b, q0, n, len;  // batch index, first token row, new tokens, cached tokens (the new ones included)
  int32_t kv0, kvt;       // key tiles before this sequence's, and its own
  int32_t per_head;       // units of one head
  int32_t pad;
};
static_assert(sizeof(LongSeq) == 48, "three 16-byte loads");

// What the device plan writes besides the sequence records.
struct ChunkCounts {
  int32_t s_seqs, s_items, s_toks, l_seqs;
  int64_t s_units, l_units;
  int32_t l_tiles;
  int32_t s_splits, l_splits;      // entries of the split lists: counted by the attention kernels
};

// Run x of G equal runs over U units begins here; 32-bit arithmetic where it
// suffices (a 64-bit division takes a few hundred cycles).
__device__ __forceinline__ int64_t run_begin(int64_t U, int x, int G) {
  if (U <= (int64_t)(0xFFFFFFFFu / 1024u)) return (uint32_t)U * (uint32_t)x / (uint32_t)G;
  return U * x / G;
}
// The run that holds unit u: the last one that begins at or before it.
__device__ __forceinline__ int run_of(int64_t U, int64_t u, int G) { return (int)(((u + 1) * G - 1) / U); }

// The softmax's weights are 2^(s - m + kHead) with the running maximum m, which
// rises only when a score has passed it by kSlack: at most 2^15 in fp16, and the
// largest at least 2^7 once m has risen to it, so that a weight keeps 11 bits
// down to 2^-21 of the largest and steps of 2^-31 of it below (with kHead = 0 a
// key 25 bits under the largest one was lost, and 65536 such keys with it).  Sums
// carry the same factor, so it cancels.
constexpr float kSlack = 8.f, kHead = 7.f;
constexpr int kLongKeys = 128;               // long path: keys per tile
constexpr int64_t kLongMost = 1 << 23;       // most cached tokens of a call's long path: the units of a head fit 31 bits
constexpr int kPairCost = 3;                 // 38 drafts of 2 and 2 chunks of 1023: 128 us a call with 0, 126 with 1, 123.5 with 2 and 3; an
                                             // 8192-token prompt at 64 heads 1138, 1126, 1133, 1091
constexpr int kLongRows = 256;               // query rows (tokens of one head) per item, two tiles of 128
constexpr int kBlkBytes = 16384;             // 128 rows x 64 fp16, swizzled
constexpr int kCTile = 8 * kBlkBytes;        // a key tile's latents
constexpr int kHeadTile = 4 * kBlkBytes;     // a key tile's keys (2 blocks) and values (2 blocks) of one head
constexpr int kWHead = 16 * kBlkBytes;       // a head's W_UK, then W_UV, 64 latent channels per block
__host__ __device__ constexpr int64_t long_partial_floats() { return (int64_t)kLongRows * (kDv + 2); }

// Key tiles up to (not including) which pair `pr` of a sequence's new tokens
// sees any key.
__host__ __device__ inline int pair_tiles(int ctx, int n, int pr) {
  const int last = n < (pr + 1) * kLongRows ? n : (pr + 1) * kLongRows;
  return (ctx + last + kLongKeys - 1) / kLongKeys;
}

// One partial of a row tile whose key tiles two or more blocks share: fp32
// [R][512] unnormalised output, then [R] maxima and [R] sums.
__host__ __device__ constexpr int64_t partial_floats(int R) { return (int64_t)R * (kDc + 2); }

// A row tile that several blocks worked on, listed by the block with its first
// part (in any order: the tiles are merged independently).
struct __align__(16) SplitRec {
  int32_t first, last;    // the blocks with its parts
  int32_t rows;           // rows to write
  int32_t pad;
  int64_t row0;           // first row in the output
};
static_assert(sizeof(SplitRec) == 32, "an aligned 16-byte load and an 8-byte one");

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
  int64_t kv_tokens;
  float scale_log2;       // softmax_scale * log2(e)
  uint16_t* o;
  int32_t* dev_err;
  uint64_t wait_ns;
  int grid;               // blocks of the attention kernels
  int64_t row_tiles;      // most row tiles of the short path
  // workspace
  ChunkCounts* counts;
  ShortSeq* s_seqs;
  int2* s_toks;           // per short-path token: its token row, and its first row in the padded row tiles
  uint8_t* q_tiles;       // [row tile][9][R][64] fp16, swizzled
  uint16_t* o_lat;        // fp16 [rows][512]
  float* parts;           // [2 grid] partials
  SplitRec* splits;       // [grid]
  LongSeq* l_seqs;
  uint8_t* c_tiles;       // [key tile][8][128][64] fp16 latents, swizzled
  uint8_t* k_rope;        // [key tile][128][64] fp16 RoPE keys
  uint32_t* kflags;       // [key tile][8]: a bit per token: 0..3 not finite, 4..7 on no page
  uint8_t* w_tiles;       // [H][8 W_UK blocks 128 x 64, 8 W_UV blocks 64 x 128] fp16
  uint8_t* kv_tiles;      // [key tile][H][K 2 blocks, V 2 blocks] fp16
  float* l_parts;         // [2 grid] partials of the long path
  SplitRec* l_splits;     // [grid]; row0: output row of the first (token row x H + head), rows H apart
};

// Whether a call has a long path at all.
inline bool has_long(int max_new, int64_t kv_tokens) { return max_new > kChunkShort && kv_tokens >= kLongKeys; }

// The row tile's height for calls whose sequences have up to max_new tokens
// of the short path: the smallest that holds all rows of a sequence, so that
// a tile is read (and dequantized) once, up to 64, what shared memory holds.
// A larger tile than the rows need costs MMA and softmax work for nothing (32
// sequences x 32768 tokens INT4 at 16 rows each: 201, 244 and 308 us with 16, 32
// and 64), a smaller one converts the keys again (24 drafts of 5 at 64 heads, bf16:
// 165 us with 64, 233 with 32).
inline int short_rows_per_tile(int max_new, int heads) {
  const int n = max_new < kChunkShort ? max_new : kChunkShort;
  const int64_t rows = (int64_t)n * heads;
  return rows <= 16 ? 16 : (rows <= 32 ? 32 : 64);
}

// The long path's launches, after the plan.
mla_status launch_long(const ChunkParams& p, int lf, int kf, cudaStream_t stream);

// The attention over the short path's sequences, by latent format (one
// translation unit each); MLA_ERR_UNSUPPORTED for another unit's formats.
mla_status launch_short_bf16(const ChunkParams& p, int lf, int kf, int R, cudaStream_t stream);
mla_status launch_short_int8(const ChunkParams& p, int lf, int kf, int R, cudaStream_t stream);
mla_status launch_short_int8_blocks(const ChunkParams& p, int lf, int kf, int R, cudaStream_t stream);
mla_status launch_short_int4(const ChunkParams& p, int lf, int kf, int R, cudaStream_t stream);

}  // namespace mla
