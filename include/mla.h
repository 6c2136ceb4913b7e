/*
 * mla.h - C ABI of the absorbed Multi-head Latent Attention (MLA) decode
 * library for NVIDIA GB300 (sm_103a).
 *
 * What it computes.  A decode step of MLA attention runs directly against a
 * cache that keeps, per token and layer, one 512-dim compressed latent
 * ("compressed_kv") and one 64-dim RoPE key ("k_pe"), and never the per-head
 * K/V.  Sources (page title, section):
 *   [CN] "DeepSeek-V2-Lite MLA 吸收式 KV 缓存优化 — 完整实验报告"
 *        §1.1 (compressed_kv = kv_a_proj(h); K, V = kv_b_proj(compressed)),
 *        §3.1 (cache the 576-dim latent), §3.2 (per-group INT8 in 32 blocks,
 *        asymmetric INT4 in 32 blocks, k_pe INT8 in 8 blocks).
 *   [EN] "Absorbed MLA Cache Optimization on DeepSeek-V2-Lite — Technical
 *        Report" §1.3 (expanded K is nope 128 + rope 64, V is 128), §2.1
 *        (store(layer, compressed_kv, k_pe) quantizes on write; get()
 *        dequantizes and projects at compute time).
 *   [TU] "DeepSeek的MLA技术：极致压缩KV Cache的创新方案" (juejin tutorial),
 *        "步骤2" (K_i = C^KV W_i^upK, V_i = C^KV W_i^upV), "KV Cache的实现"
 *        (append the latent every step), "量化压缩" (scale = absmax / 127).
 * Per sequence b and head h, with c_hat / kpe_hat the dequantized cache:
 *   q_lat[h] = q_nope[h] @ W_UK[h]                         (mla_q_absorb)
 *   s[t]     = (q_lat[h] . c_hat[t] + q_pe[h] . kpe_hat[t]) * softmax_scale
 *   o_lat[h] = sum_t softmax(s)[t] c_hat[t];  lse[h] = log sum_t exp(s[t])
 *                                                          (mla_decode_absorbed)
 *   o[h]     = o_lat[h] @ W_UV[h]                          (mla_out_unabsorb)
 * Moving W_UK onto the query and W_UV onto the output is the algebraic
 * identity q.(W c) = (q W).c; it lets every cached byte be read once for all
 * heads.
 *
 * Conventions for every call.
 *   - Ownership: the caller allocates and frees all memory (memory of the
 *     current device unless stated).  The library never allocates, frees or synchronizes;
 *     it keeps no state between calls apart from a per-device attribute
 *     cache.  Calls are thread-safe and re-entrant.
 *   - Execution: every call enqueues its kernels on `stream` (NULL = the
 *     legacy default stream) and returns without waiting.  The kernels use
 *     programmatic dependent launch: each may start while the previous
 *     kernels of the stream still run, and waits for them (griddepcontrol.wait,
 *     which also makes their stores visible) before touching data a kernel
 *     may have produced.  The few arrays read before that wait are named
 *     below ("read during the launch overlap"): no kernel enqueued on the
 *     stream since its last full ordering point (a host synchronisation, a
 *     cudaStreamWaitEvent, a memory copy) may write them, whether or not
 *     that kernel triggers its dependents early.
 *   - Layout: arrays are row-major and contiguous with the shapes given.
 *     bf16 values are passed as their 16-bit patterns (uint16_t).
 *   - Errors: arguments are checked on the host before any launch; a bad
 *     argument returns MLA_ERR_INVALID_ARG (or MLA_ERR_UNSUPPORTED for a
 *     valid but unimplemented shape) and launches nothing.  A failed launch
 *     returns MLA_ERR_CUDA.  Data-dependent faults found on the device (a
 *     slot, page id or sequence length out of range) never trap: the kernel
 *     skips the affected work and ORs a MLA_DEVERR_* bit into *dev_err when
 *     dev_err is not NULL.  The caller reads dev_err after the stream
 *     completes; a non-zero value means MLA_ERR_DEVICE_BOUNDS.
 *   - Heads: H is a multiple of 16 and at most 128.  Dimensions are fixed at
 *     the DeepSeek-V2 values: kv_lora_rank 512, rope 64, qk_nope 128, v 128.
 */
#ifndef MLA_GB300_H
#define MLA_GB300_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

struct CUstream_st;                       /* cudaStream_t is struct CUstream_st* */
typedef struct CUstream_st* mla_stream_t;

typedef enum {
  MLA_OK = 0,
  MLA_ERR_INVALID_ARG = 1,
  MLA_ERR_UNSUPPORTED = 2,
  MLA_ERR_CUDA = 3,
  MLA_ERR_DEVICE_BOUNDS = 4
} mla_status;

typedef enum {
  MLA_FMT_BF16 = 0,        /* values stored as bf16, no scale */
  MLA_FMT_INT8_SYM = 1,    /* int8 code, fp32 scale per (token, group) */
  MLA_FMT_INT4_ASYM = 2,   /* 4-bit code, fp32 scale and zero per (token, group) */
  MLA_FMT_INT4_SYM = 3,    /* 4-bit code in [-7, 7], fp32 scale per (token, group) */
  /* INT8_SYM latent with another block count ([EN] §5.1 sweep of 8 / 32 /
   * 64 blocks, [CN] §3.2 per-token row); latent only, with INT8 k_pe */
  MLA_FMT_INT8_G8 = 4,     /* 64 blocks of 8 channels */
  MLA_FMT_INT8_G32 = 5,    /* 16 blocks of 32 channels */
  MLA_FMT_INT8_G64 = 6,    /* 8 blocks of 64 channels */
  MLA_FMT_INT8_TOKEN = 7,  /* one block of 512 channels (per-token scale) */
  /* outlier-protected mixed precision ([EN] §4.3 row "C: Mixed precision
   * (outlier-protected)", 18.2 KB per token, 14.8x, 580K tokens in 10 GB;
   * the page gives no mechanism, this is the reading): INT8_SYM latent
   * (32 groups of 16) except MLA_OUTLIER_CHANNELS protected channels per
   * layer, kept as their bf16 input and left out of their group's absmax
   * (their codes are 0).  512 + 2 x 25 code bytes plus bf16 k_pe give the
   * row's 690 B per layer.  k_pe: MLA_FMT_BF16 (the row) or INT8_SYM. */
  MLA_FMT_INT8_OUTLIER = 8
} mla_fmt;

/* Bits ORed into *dev_err. */
#define MLA_DEVERR_SLOT    1  /* append: slot not in [0, num_pages*64) and not -1;
                                 move: a kept position outside the sequence */
#define MLA_DEVERR_PAGE    2  /* decode, chunks, mass, select, move: block_table entry not in
                                 [0, num_pages); plan, release: a page id, a table row or the free range */
#define MLA_DEVERR_SEQLEN  4  /* decode: seq_len < 0 or > max_pages*64; plan, chunks and the
                                 calls behind a step: lengths that do not fit the call's arrays */
#define MLA_DEVERR_TIMEOUT 8  /* a bounded wait inside a kernel gave up           */
#define MLA_DEVERR_NO_PAGES 16 /* plan, release: the free list has too few pages, or
                                 (release) no room for those given back */
#define MLA_DEVERR_TOKEN   32 /* verify: a draft outside the vocabulary, or a row without weight */

#define MLA_KV_LORA_RANK 512
#define MLA_ROPE_DIM 64
#define MLA_QK_NOPE_DIM 128
#define MLA_V_DIM 128
#define MLA_PAGE_TOKENS 64
#define MLA_LATENT_GROUP 16      /* 512 channels = 32 groups ([CN] §3.2 "32块") */
#define MLA_KPE_GROUP 8          /* 64 channels = 8 groups ([CN] §3.2 "8块")   */
#define MLA_OUTLIER_CHANNELS 25  /* protected channels of MLA_FMT_INT8_OUTLIER (5 % of 512) */

/*
 * One layer's paged latent cache.  The pool holds num_pages pages of 64
 * tokens; a token's physical slot is page * 64 + offset.  Which pages belong
 * to which sequence is the caller's business (block tables below).
 *   latent_fmt: any mla_fmt.  kpe_fmt: MLA_FMT_BF16, MLA_FMT_INT8_SYM or
 *   MLA_FMT_INT4_SYM; the INT8_G* / INT8_TOKEN latent formats take
 *   MLA_FMT_INT8_SYM k_pe only, INT8_OUTLIER takes BF16 or INT8_SYM.
 *   pool: device memory of mla_cache_pool_bytes() bytes, 256-byte aligned,
 *         owned by the caller.
 *   outlier_channels: INT8_OUTLIER only (NULL for every other format): HOST
 *         memory holding the layer's MLA_OUTLIER_CHANNELS protected latent
 *         channels, strictly increasing, in [0, 512) (for instance from
 *         mla_select_outlier_channels); read during each call, by value.
 *         Every call on a layer must pass the same set; a violation of
 *         these rules is MLA_ERR_INVALID_ARG.
 */
typedef struct {
  int32_t num_pages;
  int32_t latent_fmt;
  int32_t kpe_fmt;
  int32_t reserved;        /* must be 0 */
  void* pool;
  const int32_t* outlier_channels;
} mla_cache_layer;

/*
 * Byte layout of one page.  A page of 64 tokens is two contiguous blocks of
 * 32 tokens (token t of a page lives in block t / 32 as block token
 * u = t % 32), so that one bulk copy moves a whole 32-token work unit.
 * Inside a block, structure of arrays; offsets are from the block start,
 * every field starts on a 128-byte boundary, -1 marks a field the format
 * does not have:
 *   codes      [32][codes_row_bytes]: bf16 values (1024 B), int8 codes
 *              (512 B) or 4-bit codes (256 B).  The row is a sequence of
 *              16-byte chunks; logical chunk c of block token u is stored at
 *              chunk position (c & ~7) | ((c ^ u) & 7).  An int8 chunk is 16
 *              channels in channel order (INT8_G8: its 32-bit word j holds
 *              channels 2j, 2j+1, 8+2j, 8+2j+1); a bf16 chunk is 8 channels.
 *              A 4-bit chunk c holds groups A = 2c and B = 2c + 1; its 32-bit
 *              word j (j = 0..3) packs, from the least significant nibble,
 *              A[4j], A[4j+2], B[4j], B[4j+2], A[4j+1], A[4j+3], B[4j+1],
 *              B[4j+3] (X[i] = nibble of channel i of group X).  A nibble is
 *              the code (INT4_ASYM, 0..15) or the code + 8 (INT4_SYM, 1..15).
 *   scale      fp32 [G groups][32 block tokens]    (int8 / 4-bit latent; G = 32,
 *              or 64 / 16 / 8 / 1 for INT8_G8 / G32 / G64 / TOKEN)
 *   zero       fp32 [32 groups][32 block tokens]   (INT4_ASYM latent; integer-valued)
 *   outlier    bf16 [25 protected channels][32 block tokens], in the order
 *              of outlier_channels, padded to 1664 bytes (INT8_OUTLIER)
 *   kpe        [32][kpe_row_bytes]: bf16 (128 B = 8 chunks of 8 channels,
 *              chunk c of token u at position c ^ (u & 7)), int8 (64 B =
 *              4 chunks of two 8-channel groups, chunk c at c ^ ((u >> 1) & 3))
 *              or INT4_SYM (32 B = 2 chunks of 32 channels, chunk c at
 *              c ^ ((u >> 2) & 1); chunk c packs its halves A = channels
 *              32c .. 32c+15 and B = 32c+16 .. 32c+31 like a 4-bit latent
 *              chunk, nibble = code + 8)
 *   kpe_scale  fp32 [8 groups][32 block tokens]    (int8 / INT4_SYM k_pe)
 *   bound      fp32 [32 block tokens]              (int8 / 4-bit latent)
 *              M_t, the largest magnitude a code of the token's latent can
 *              dequantize to: 127 max_g s_g (INT8 formats), 7 max_g s_g
 *              (INT4_SYM), max_g s_g (|z_g - 7.5| + 7.5) (INT4_ASYM), in
 *              fp32 with one rounding per product; INT8_OUTLIER also takes
 *              the protected values' magnitudes into the maximum.  For INT8
 *              and INT4_SYM formats it equals max_c |c_hat[c]|.  Written by mla_cache_append;
 *              the decode reads it to find the rows it recomputes exactly
 *              (see mla_decode_absorbed).
 * page_bytes = 2 * block_bytes = 64 x (1152, 740, 612 or 580) bytes for
 * bf16/bf16, int8/int8, int4/int8 and int4/int4-sym (the last is [CN]
 * §4.1's 7.6 KB-per-token scheme: 288 B of codes per layer plus scales,
 * zero-points and the bound).  The swizzles spread the rows of eight consecutive tokens
 * over all shared-memory banks when a block is copied verbatim into shared
 * memory.
 */
typedef struct {
  int64_t page_bytes, block_bytes;
  int64_t codes_off, codes_row_bytes;
  int64_t scale_off, zero_off;
  int64_t kpe_off, kpe_row_bytes;
  int64_t kpe_scale_off;
  int64_t bound_off;
  int64_t outlier_off;
} mla_page_layout;

/* Fills *out for the cache's formats.  MLA_ERR_INVALID_ARG on a bad format. */
mla_status mla_cache_page_layout(const mla_cache_layer* cache, mla_page_layout* out);

/* num_pages * page_bytes, or 0 for an invalid descriptor. */
size_t mla_cache_pool_bytes(const mla_cache_layer* cache);

/*
 * mla_cache_append - quantize-on-write of n new tokens into the paged cache.
 * [EN] §2.1 store(): compressed_kv [seq, 512] is quantized, k_pe [seq, 64]
 * stored; [CN] §3.2 for the formats.  Quantization rules, all IEEE fp32 with
 * round-half-even and no fused multiply-add:
 *   INT8_SYM  (groups of 16 latent channels - 8, 32, 64 or 512 for the
 *             INT8_G8 / G32 / G64 / TOKEN formats - or 8 k_pe channels):
 *       s = max|x| / 127;  q = clamp(rint(x / s), -127, 127);  s = 0 -> q = 0
 *   INT4_ASYM (groups of 16): s = (max - min) / 15;  z = rint(-min / s);
 *       q = clamp(rint(x / s) + z, 0, 15); if s == 0: s = |min|, z = rint(-min/s)
 *       (or s = z = 0 when min == 0) and q = 0.
 *   INT4_SYM  (groups of 16 latent channels, or 8 k_pe channels; [CN] §3.2
 *       "对称 INT4" rows): s = max|x| / 7;  q = clamp(rint(x / s), -7, 7);
 *       s = 0 -> q = 0.
 *   INT8_OUTLIER: the protected channels' input bits are stored, their
 *       codes are 0, and the INT8_SYM rule runs on the other channels with
 *       the protected ones counted as 0 in their group's max|x|.
 *   BF16: the input bits are copied.
 *   A quantized latent also gets its bound M_t (see mla_page_layout).
 *   c_new   bf16 [n][512]     kpe_new bf16 [n][64]
 *   slot    int32 [n]: physical slot (page * 64 + offset) of each token;
 *           -1 skips the token silently; any other value outside
 *           [0, num_pages * 64) skips it and sets MLA_DEVERR_SLOT.
 *   Two tokens with the same slot in one call race; the result is one of them.
 *   n == 0 is a no-op.  dev_err may be NULL.
 */
mla_status mla_cache_append(const mla_cache_layer* cache, const uint16_t* c_new,
                            const uint16_t* kpe_new, const int32_t* slot, int32_t n,
                            int32_t* dev_err, mla_stream_t stream);

/*
 * mla_select_outlier_channels - calibration of MLA_FMT_INT8_OUTLIER's
 * protected set ([EN] §4.3 row C, read as in mla_fmt): the
 * MLA_OUTLIER_CHANNELS latent channels with the largest max |x| over n
 * sample rows, ties to the lower channel index, written in increasing
 * order.  NaN inputs are skipped by the maximum.
 *   c_sample     device bf16 [n][512], 16-byte aligned; n >= 1
 *   channels_out device int32 [MLA_OUTLIER_CHANNELS], 4-byte aligned
 */
mla_status mla_select_outlier_channels(const uint16_t* c_sample, int32_t n, int32_t* channels_out,
                                       mla_stream_t stream);

/*
 * mla_q_absorb - q_lat[b][h] = q_nope[b][h] @ W_UK[h]   (the query side of
 * weight absorption; [TU] "步骤2" K_i = C^KV W_i^upK with W_UK[h] = (W_i^upK)^T).
 *   q_nope bf16 [B][H][128]   W_UK bf16 [H][128][512]   q_lat fp32 [B][H][512]
 *   fp32 accumulation of exact bf16 products.  B == 0 is a no-op.
 *   W_UK is read during the launch overlap (see Execution above).
 */
mla_status mla_q_absorb(const uint16_t* q_nope, const uint16_t* w_uk, float* q_lat,
                        int32_t batch, int32_t heads, mla_stream_t stream);

/*
 * mla_decode_workspace_bytes - bytes of device workspace mla_decode_absorbed
 * needs for this batch, head count and num_splits (0 = automatic).  The
 * workspace holds the split-K partials (per split and head, fp32: running
 * max, running sum, the weight of the fp16 P V products and the
 * unnormalised 512-wide latent output).
 */
size_t mla_decode_workspace_bytes(int32_t batch, int32_t heads, int32_t num_splits);

/*
 * mla_decode_absorbed - absorbed attention of one decode query per sequence
 * against its cached latents ([EN] §2.1 get(): attention computed from the
 * latent; flash-decode split over context chunks with a log-sum-exp
 * combine).  Dequantization is fused into the tile loads: x_hat = q * s for
 * INT8 and INT4_SYM, (q - z) * s for INT4_ASYM.
 *   q_lat       fp32 [B][H][512]   (from mla_q_absorb)
 *   q_pe        bf16 [B][H][64]
 *   block_table int32 [B][max_pages]: page id of each sequence's logical page
 *   seq_lens    int32 [B]: tokens attended (positions 0..len-1, the newly
 *               appended token included).  0 gives o_lat = 0 and lse = -inf.
 *   softmax_scale: typically 1 / sqrt(128 + 64).
 *   num_splits: ranges the context work is divided into, 1 .. 65535
 *               (0 = automatic: SMs / (H / 16), so that the H / 16 head
 *               tiles of every range run side by side, one CTA per SM, and
 *               read the range's pages once between them).  Work is split
 *               evenly over all sequences' 32-token chunks.
 *   workspace:  device, >= mla_decode_workspace_bytes(B, H, num_splits)
 *               bytes, 256-byte aligned; contents are scratch.
 *   o_lat fp32 [B][H][512]      lse fp32 [B][H] (natural log; may be NULL)
 *   Precision, against attention in fp64 over the same dequantized values:
 *   the scores use exact products (q_lat split into two fp16 parts against
 *   the exact codes); P enters the P V products as fp16 times the fp16
 *   group scale, which costs ~2-6e-4 relative error over long contexts.
 *   Two kinds of rows are recomputed in fp32 from the cache instead:
 *   sequences shorter than 256 tokens, and rows whose output is a small
 *   residual of heavily weighted tokens (latents that cancel), detected
 *   from the partials as sqrt(sum_t (w_t M_t)^2) > 4 |o_lat row|_inf, with
 *   w_t the softmax weights and M_t a bound on token t's |c_hat| from its
 *   scales (and zero-points).
 *   Every row is tested to a max relative error below 2e-3 (o_lat) and
 *   2e-3 absolute (lse).
 *   A page id outside [0, num_pages) contributes nothing and sets
 *   MLA_DEVERR_PAGE; seq_len outside [0, max_pages*64] is treated as 0 and
 *   sets MLA_DEVERR_SEQLEN.  B == 0 is a no-op.  B <= 4096, and
 *   B * max_pages * 2 (the batch's 32-token chunk capacity) < 2^31, else
 *   MLA_ERR_INVALID_ARG.
 *   seq_lens is read during the launch overlap (see Execution above).
 */
mla_status mla_decode_absorbed(const mla_cache_layer* cache, const float* q_lat,
                               const uint16_t* q_pe, const int32_t* block_table,
                               int32_t max_pages, const int32_t* seq_lens, int32_t batch,
                               int32_t heads, float softmax_scale, int32_t num_splits,
                               void* workspace, size_t workspace_bytes, float* o_lat,
                               float* lse, int32_t* dev_err, mla_stream_t stream);

/*
 * mla_decode_absorbed_unabsorb - mla_decode_absorbed followed by
 * mla_out_unabsorb on its o_lat, in one call: o[b][h] = o_lat[b][h] @ W_UV[h]
 * ([TU] "步骤2", V_i = C^KV W_i^upV, the output side of the absorption).
 * The arguments are mla_decode_absorbed's plus
 *   w_uv  device bf16 [H][512][128], 16-byte aligned (as mla_out_unabsorb)
 *   o     device fp32 [B][H][128], 16-byte aligned
 * Both must be non-NULL (MLA_ERR_INVALID_ARG otherwise).  o_lat and lse are
 * written as by mla_decode_absorbed.  When the batch takes the combine's
 * one-block-per-(sequence, head) grid (about 8 to 32 context splits per
 * sequence, e.g. a few sequences of a few thousand tokens), that block
 * projects its row right after merging it (fp32 multiply-adds over bf16
 * W_UV), which removes a kernel from the decode step's critical path;
 * otherwise the call launches the unabsorb kernel after the combine.  The
 * two ways differ only in the order of the fp32 sums.
 */
/*
 * mla_decode_kernel_count - how many kernels one mla_decode_absorbed call
 * (with_unabsorb = 0) or mla_decode_absorbed_unabsorb call (1) launches for
 * this batch shape: the split kernel and the combine, plus the unabsorb
 * kernel when the combine's grid does not project the rows itself.  0 for
 * batch 0, -1 for arguments the calls would reject.  Host only.
 */
int32_t mla_decode_kernel_count(const mla_cache_layer* cache, int32_t batch, int32_t heads, int32_t num_splits,
                                int32_t with_unabsorb);

mla_status mla_decode_absorbed_unabsorb(const mla_cache_layer* cache, const float* q_lat,
                                        const uint16_t* q_pe, const int32_t* block_table,
                                        int32_t max_pages, const int32_t* seq_lens, int32_t batch,
                                        int32_t heads, float softmax_scale, int32_t num_splits,
                                        void* workspace, size_t workspace_bytes, float* o_lat,
                                        float* lse, const uint16_t* w_uv, float* o, int32_t* dev_err,
                                        mla_stream_t stream);

/*
 * mla_decode_absorbed_noalloc - the same decode as mla_decode_absorbed for
 * callers that cannot allocate device memory: a plugin handed only its input
 * and output buffers, code running during CUDA-graph capture (cudaMalloc is
 * not capturable there), or a serving loop that forbids allocation after
 * start-up.  The source pages have no counterpart; this is a deployment
 * variant of the call above.
 *   Arguments and results are those of mla_decode_absorbed, without the
 *   workspace: the split-K partials go to a scratch array of
 *   MLA_NOALLOC_SCRATCH_BYTES compiled into the library, which every device
 *   that loads the library holds until the process exits.  It calls no
 *   allocator (no cudaMalloc, cudaFree or allocating library routine).
 *   Returns MLA_ERR_INVALID_ARG when mla_decode_workspace_bytes(batch, heads,
 *   num_splits) exceeds MLA_NOALLOC_SCRATCH_BYTES (e.g. 64 heads at batch 64
 *   with the automatic split count fits; pass a smaller num_splits
 *   otherwise).
 *   The first call on a device looks up the array's device address (with
 *   that device current) and caches it; make that first call before any
 *   stream capture.  All calls share the array and it keeps the last call's
 *   contents (nothing in it needs to start at zero), so calls that overlap
 *   on the GPU - on different streams or from different host threads - race.
 */
#define MLA_NOALLOC_SCRATCH_BYTES (32u << 20)
mla_status mla_decode_absorbed_noalloc(const mla_cache_layer* cache, const float* q_lat,
                                       const uint16_t* q_pe, const int32_t* block_table,
                                       int32_t max_pages, const int32_t* seq_lens, int32_t batch,
                                       int32_t heads, float softmax_scale, int32_t num_splits,
                                       float* o_lat, float* lse, int32_t* dev_err, mla_stream_t stream);

/*
 * mla_prefill_workspace_bytes - bytes of device workspace mla_prefill_absorbed
 * needs for a chunk of n query tokens and this head count under the current
 * prefill path setting (0 for invalid arguments).  Bounded in n: queries are
 * processed in slices of 2048 (decode kernels) or 4096 (tensor cores: 288 KB
 * of query tiles per 128 rows, ~600 MB at 64 heads); the tensor-core path
 * adds the key tiles of up to 65536 positions (~151 MB).
 */
size_t mla_prefill_workspace_bytes(int32_t n, int32_t heads);

/*
 * Prefill implementations (mla_set_prefill_path):
 *   MLA_PREFILL_AUTO           tensor cores when 256 < ctx_before + n <=
 *                              65536 and either n * heads >= 8192, or
 *                              n * heads >= 2048 and ctx_before + n >= 4096;
 *                              else the decode kernels (the default)
 *   MLA_PREFILL_DECODE_KERNELS always the split-K decode kernels
 *   MLA_PREFILL_TENSOR_CORES   always tensor cores; a call with
 *                              ctx_before + n > 65536 returns
 *                              MLA_ERR_UNSUPPORTED
 * Both compute the same attention within the same bound (§ prefill below).
 */
#define MLA_PREFILL_AUTO 0
#define MLA_PREFILL_DECODE_KERNELS 1
#define MLA_PREFILL_TENSOR_CORES 2

/*
 * mla_set_prefill_path - selects the implementation of the prefill calls this
 * process makes afterwards (and the size mla_prefill_workspace_bytes
 * returns); returns the previous setting, or -1 (nothing changed) for an
 * unknown value.
 */
int32_t mla_set_prefill_path(int32_t path);

/*
 * mla_prefill_path_taken - the implementation (MLA_PREFILL_DECODE_KERNELS or
 * MLA_PREFILL_TENSOR_CORES) a prefill call with these sizes takes under the
 * current setting; -1 for invalid sizes.
 */
int32_t mla_prefill_path_taken(int32_t ctx_before, int32_t n, int32_t heads);

/*
 * mla_prefill_absorbed - causal absorbed attention of a prefill chunk: the
 * queries of n tokens of one sequence that were just appended to the cache
 * (chunked prefill when ctx_before > 0).  Query i sits at position
 * ctx_before + i and attends to the cached positions 0 .. ctx_before + i,
 * its own token included; per query this is the decode of [EN] §2.1 over
 * that prefix.  Tensor-core path: the cached tokens are dequantized once
 * into fp16 (hi, lo) key tiles and a tcgen05 kernel runs 128 query rows
 * against 128 keys at a time (scores from three fp16 products, P and V in
 * fp16, fp32 accumulation); decode-kernel path: the split-K decode kernels
 * with the queries as the batch.  On both, rows that see fewer than 256
 * tokens, and rows whose softmax weight sits on tokens whose latents cancel
 * (the decode's precision check), are recomputed exactly in fp32.
 *   q_lat       fp32 [n][H][512]  (mla_q_absorb with batch = n)
 *   q_pe        bf16 [n][H][64]
 *   block_table int32 [max_pages]: the sequence's page ids; positions up to
 *               ctx_before + n - 1 must have been appended.
 *   workspace:  device, >= mla_prefill_workspace_bytes(n, H) bytes,
 *               256-byte aligned; contents are scratch.
 *   o_lat fp32 [n][H][512]      lse fp32 [n][H] (natural log; may be NULL)
 *   n == 0 is a no-op.  ctx_before >= 0 and ctx_before + n <= max_pages * 64,
 *   else MLA_ERR_INVALID_ARG.  A page id outside [0, num_pages) contributes
 *   nothing and sets MLA_DEVERR_PAGE.
 */
mla_status mla_prefill_absorbed(const mla_cache_layer* cache, const float* q_lat, const uint16_t* q_pe,
                                const int32_t* block_table, int32_t max_pages, int32_t ctx_before, int32_t n,
                                int32_t heads, float softmax_scale, void* workspace, size_t workspace_bytes,
                                float* o_lat, float* lse, int32_t* dev_err, mla_stream_t stream);

/*
 * mla_out_unabsorb - o[b][h] = o_lat[b][h] @ W_UV[h]   (the output side of
 * weight absorption; [TU] "步骤2" V_i = C^KV W_i^upV with W_UV[h] = W_i^upV).
 *   o_lat fp32 [B][H][512]   W_UV bf16 [H][512][128]   o fp32 [B][H][128]
 *   B == 0 is a no-op.  W_UV is read during the launch overlap (see
 *   Execution above).
 */
mla_status mla_out_unabsorb(const float* o_lat, const uint16_t* w_uv, float* o,
                            int32_t batch, int32_t heads, mla_stream_t stream);

/*
 * mla_lse_merge - attention over the union of disjoint context parts of the
 * same sequences, from the parts' own results: the exchange step of a
 * context-sharded decode (each GPU runs mla_decode_absorbed over its own
 * pages of a sequence; the (o_lat, lse) pairs are gathered and merged here).
 * With M = max_r lse_r and w_r = exp(lse_r - M):
 *   o_lat = sum_r w_r o_r / sum_r w_r,   lse = M + ln sum_r w_r
 * which is exactly the softmax attention of [EN] §2.1 over the union.
 *   o_parts  fp32 [R][B][H][512]   lse_parts fp32 [R][B][H]  (natural log;
 *            -inf marks an empty part, weight 0)
 *   o_lat    fp32 [B][H][512]      lse fp32 [B][H] (may be NULL)
 *   All parts empty gives o_lat = 0 and lse = -inf.  1 <= R <= 4096,
 *   B <= 4096, H as for the decode; B == 0 is a no-op.  Arrays 16-byte
 *   aligned; o_lat must not overlap o_parts.
 */
mla_status mla_lse_merge(const float* o_parts, const float* lse_parts, int32_t parts, int32_t batch,
                         int32_t heads, float* o_lat, float* lse, mla_stream_t stream);

/*
 * ---------------------------------------------------------------------------
 * A serving step over a ragged batch: mla_plan_chunks, mla_rope,
 * mla_cache_append, mla_chunk_attention, in this order.
 *
 * The sequences of a step have any numbers of new tokens - 1 for a decode, a
 * few for a speculative draft, thousands for a prefill chunk - stored one
 * sequence behind the other: sequence b's are rows q_start[b] ..
 * q_start[b + 1] - 1 of every per-token array.  Lengths live on the device,
 * so that a captured step can be replayed with other lengths.
 * ---------------------------------------------------------------------------
 */

/*
 * mla_plan_chunks - block tables, slot map, positions and lengths of a step,
 * built on the GPU from the requests' lengths.
 *   Inputs, all device int32:
 *   ctx_lens    [B]: tokens of the request already in the cache
 *   new_lens    [B]: its new tokens in this step (0 is allowed)
 *   req         [B]: its row of page_table
 *   page_table  [rows][max_pages]: the requests' page ids, kept from step to
 *               step.  The step's new pages are written into it; every other
 *               entry stays as it was.
 *   free_pages  [free_len]: ids of unused pages; free_range {head, tail}:
 *               entries head .. tail - 1 are available.  New pages are taken
 *               from free_pages[head] on, in the order of the batch.
 *   num_pages   pages in the pool (ids are checked against it)
 *   n_tokens    length of the per-token outputs
 *   Outputs, all device int32, no two of them (nor an input) overlapping:
 *   block_table [B][max_pages]: the row of each request, -1 behind its last
 *               page: what the attention calls take
 *   q_start     [B + 1]: first token row of each request, then the total
 *   seq_lens    [B]: ctx + new
 *   positions, token_req, slot [n_tokens]: each token's position (its place
 *               in the cache; see mla_move_tokens for a cache that was cut),
 *               batch index and cache slot (mla_cache_append's); 0, -1 and -1
 *               behind the last token, which the append skips
 *   free_head   [1]: the next step's head (not free_range itself)
 *   A request is refused, and the others go on, when its lengths are
 *   negative or exceed max_pages * 64, or its tokens do not fit n_tokens
 *   (MLA_DEVERR_SEQLEN); its req is out of range or named twice in the call
 *   (MLA_DEVERR_PAGE); or the free list has too few pages
 *   (MLA_DEVERR_NO_PAGES: nobody behind it gets pages either).  A refused
 *   request takes no page; its seq_lens entry is 0, its block_table row -1,
 *   its tokens' slots -1 and their positions 0.  Its new tokens (none where
 *   new is negative) keep their rows, so that a count far too large leaves the
 *   requests behind it no room.  A page id outside the pool
 *   sets MLA_DEVERR_PAGE and is written as -1; a bad free_range counts as
 *   empty and sets MLA_DEVERR_PAGE.
 *   rows <= 65536; batch <= 4096; batch == 0 is a no-op.  The same inputs
 *   give the same outputs, also when the call is repeated: it does not move
 *   free_range.
 *   seq_lens feeds mla_chunk_attention directly; mla_decode_absorbed reads
 *   its lengths during the launch overlap and needs an ordering point in
 *   between (see Execution above).
 */
mla_status mla_plan_chunks(const int32_t* ctx_lens, const int32_t* new_lens, const int32_t* req, int32_t batch,
                           int32_t* page_table, int32_t rows, int32_t max_pages, const int32_t* free_pages,
                           int32_t free_len, const int32_t* free_range, int32_t num_pages, int32_t n_tokens,
                           int32_t* block_table, int32_t* q_start, int32_t* seq_lens, int32_t* positions,
                           int32_t* token_req, int32_t* slot, int32_t* free_head, int32_t* dev_err,
                           mla_stream_t stream);

/*
 * mla_rope - rotary positions on 64-channel rows of queries and keys, with
 * one to four position axes (text; time, height and width of images and
 * video).  Pair i (i = 0..31) of a row turns by
 *   t = positions[pair_axis[i]][token] * inv_freq[i]:
 *   y1 = amplitude (x1 cos t - x2 sin t),  y2 = amplitude (x1 sin t + x2 cos t)
 * Angles are off by at most 1e-7 + 2^-52 |position * inv_freq| radians (6e-7
 * at every 32-bit position for |inv_freq| <= 1), the products are fp32,
 * rounded once to bf16.
 *   q_pe     bf16 [n][heads][64] at the given strides (elements, multiples of
 *            8), 16-byte aligned; heads 0..128 (0: keys only)
 *   k_pe     bf16 [n][64] at k_token_stride, or NULL (then k_out is NULL too)
 *   positions int32 [axes][n], negative ones allowed; inv_freq fp32 [32],
 *            finite: the caller's frequency table, with any long-context
 *            interpolation already in it
 *   pair_axis HOST uint8 [32], each < axes, read during the call; NULL: axis 0
 *   interleaved 1: pairs are channels (2i, 2i + 1); 0: (i, i + 32)
 *   inverse  1: turns by -t (the gradient of the forward call; with amplitude
 *            1 or -1 it also takes a rotation back)
 *   q_out, k_out: bf16 at their own strides; a call may write over its
 *            inputs (same pointer and strides), any other overlap is
 *            undefined.  Rows of an output must not overlap each other.
 *   n == 0 is a no-op.
 */
mla_status mla_rope(const uint16_t* q_pe, int64_t q_token_stride, int64_t q_head_stride, const uint16_t* k_pe,
                    int64_t k_token_stride, const int32_t* positions, int32_t axes, const uint8_t* pair_axis,
                    const float* inv_freq, int32_t n, int32_t heads, int32_t interleaved, int32_t inverse,
                    float amplitude, uint16_t* q_out, int64_t qo_token_stride, int64_t qo_head_stride,
                    uint16_t* k_out, int64_t ko_token_stride, mla_stream_t stream);

/*
 * mla_chunk_attention - causal attention of a ragged batch of new tokens over
 * the paged cache, from the projected queries to the per-head outputs.  The
 * new tokens were appended before.  With c = seq_lens[b] - n_b (n_b = q_start
 * [b + 1] - q_start[b]), new token i of sequence b attends to positions t <=
 * c + i:
 *   s[h][t] = (q_nope[h] . (W_UK[h] c_hat[t]) + q_pe[h] . kpe_hat[t]) * scale
 *   o[h]    = sum_t softmax(s[h])[t] c_hat[t] @ W_UV[h]
 *   q_nope  bf16 [n_tokens][H][128], q_pe bf16 [n_tokens][H][64], both at the
 *           given token and head strides (elements, multiples of 8; they may
 *           be slices of one [n][H][192] array), 16-byte aligned
 *   w_uk    bf16 [H][128][512], w_uv bf16 [H][512][128]; both are read during
 *           the launch overlap (see Execution above)
 *   block_table int32 [B][max_pages]; q_start int32 [B + 1], increasing;
 *           seq_lens int32 [B], the new tokens included (0: the sequence's
 *           rows are 0)
 *   max_new bound on every n_b (host; at most n_tokens): what the launch and
 *           the workspace are sized for
 *   kv_tokens bound on the sum of seq_lens, each rounded up to 128, over the
 *           sequences with more than MLA_CHUNK_SHORT new tokens (0 when
 *           there is none); at most 2^23.  Those sequences' latents are
 *           expanded into the workspace, 512 bytes per token and head
 *   workspace: device, >= mla_chunk_workspace_bytes(...) bytes, 256-byte
 *           aligned; contents are scratch, so calls that may overlap (other
 *           streams, two graphs replayed at once) need their own
 *   o       bf16 [n_tokens][H][128], 16-byte aligned.  Rows behind
 *           q_start[B] are left as they were.
 *   A page id outside the pool contributes nothing and sets MLA_DEVERR_PAGE.
 *   A sequence whose figures do not fit (n_b > max_new, 0 < seq_lens[b] <
 *   n_b, seq_lens[b] < 0 or > max_pages * 64, kv_tokens exceeded: then every
 *   later one that counts toward kv_tokens too) sets MLA_DEVERR_SEQLEN; its
 *   rows are 0.  A q_start that decreases or leaves [0, n_tokens] anywhere
 *   refuses all sequences, since their rows could overlap.
 *   Precision: fp16 operands, fp32 accumulation and softmax, one rounding of
 *   o to bf16.  A softmax weight keeps 11 bits down to 2^-21 of the row's
 *   largest one; below it is off by at most 2^-32 of that (so 2^23 keys by
 *   2^-9 together).  Queries (after the absorption and the scale), cached values,
 *   weights, keys and values beyond 65504 in magnitude count as non-finite.
 *   A non-finite token makes the rows that attend to it NaN and leaves the
 *   others alone.  A wait that runs out (mla_set_wait_limit_ns) sets
 *   MLA_DEVERR_TIMEOUT and leaves the rows of o undefined.
 *   batch <= 4096, n_tokens * H < 2^31; n_tokens == 0 or batch == 0 is a
 *   no-op.
 */
#define MLA_CHUNK_SHORT 64
mla_status mla_chunk_attention(const mla_cache_layer* cache, const uint16_t* q_nope, int64_t qn_token_stride,
                               int64_t qn_head_stride, const uint16_t* q_pe, int64_t qp_token_stride,
                               int64_t qp_head_stride, const uint16_t* w_uk, const uint16_t* w_uv,
                               const int32_t* block_table, int32_t max_pages, const int32_t* q_start,
                               const int32_t* seq_lens, int32_t batch, int32_t n_tokens, int32_t heads,
                               int32_t max_new, int64_t kv_tokens, float softmax_scale, void* workspace,
                               size_t workspace_bytes, uint16_t* o, int32_t* dev_err, mla_stream_t stream);

/* Bytes of device workspace mla_chunk_attention needs; 0 for invalid
 * arguments. */
size_t mla_chunk_workspace_bytes(int32_t batch, int32_t n_tokens, int32_t heads, int32_t max_new, int64_t kv_tokens);

/*
 * ---------------------------------------------------------------------------
 * Behind a step's attention: which of the cached tokens stay.
 *
 * Speculative decoding: mla_verify_drafts says how many drafts of each
 * sequence were accepted, mla_release_pages (trim) gives back the pages of
 * the rejected ones.  A cache with a budget: mla_token_mass adds up the
 * attention weight that every token received, mla_select_tokens picks those
 * that stay, mla_release_pages (move) gives the sequences fresh pages for
 * them, mla_move_tokens moves them.  Pages are the same for all layers, so
 * the release runs once a step, the others once a layer.  Lengths live on the
 * device, so that a captured step can be replayed with other ones.  The calls
 * of this section, the plan, the append and mla_chunk_attention take lengths
 * from the call before them; mla_decode_absorbed, whose lse the attention
 * weight needs, reads its seq_lens during the launch overlap: between a call
 * that writes them (the plan, kept_lens, lens_out) and the decode a full
 * ordering point is needed (see Execution above), for instance a device-to-
 * device copy of the lengths, which a graph captures as well.  No output may
 * overlap an input or another output, but where a call says so.
 * ---------------------------------------------------------------------------
 */

/*
 * mla_verify_drafts - drafted tokens against the target model's
 * probabilities, from given random numbers, and the token sampled behind the
 * accepted ones.  Sequence b has rows row_start[b] .. row_start[b + 1] - 1,
 * one more than its drafts (one row: it only samples; none: it takes no part).
 * Row r holds the target's and the draft model's distribution of the same
 * token.  With c(x) = x where 0 < x < inf and 0 elsewhere:
 *   drafts pass in order while u_accept[r] * c(q_r(d_r)) < c(p_r(d_r));
 *   behind the last that passed, at row j, the next token is drawn from
 *   w(v) = max(c(p_j(v)) - c(q_j(v)), 0), or from w = c(p_j) behind the
 *   last draft or where nothing else is left: the smallest v for which the
 *   sum of w up to v is larger than u_sample[b] * sum w
 *   target_probs [rows][vocab] of type prob_type, rows target_row_stride
 *           elements apart (>= vocab; any alignment of the type).  Rows need
 *           not add up to 1
 *   draft_probs the same (the last row of a sequence is not read), or NULL:
 *           drafts that were certain, as from a lookup: q_r is 1 at d_r
 *   drafts  int32 [rows]: d_r; a sequence's last entry is not used
 *   u_accept fp32 [rows], u_sample fp32 [B], in [0, 1): u_sample is clamped
 *           to [0, 1] (1: the last v with weight; NaN counts as 0), a NaN in
 *           u_accept rejects
 *   seq_lens int32 [B]: cached tokens with all drafts; with kept_lens, or both NULL
 *   accepted int32 [B]: drafts that passed
 *   tokens  int32 [B][max_out]: the accepted drafts, the drawn token, -1 behind
 *   kept_lens int32 [B]: seq_lens less the rejected drafts (may be seq_lens,
 *           else must not overlap it): the next step's context
 *   A draft outside [0, vocab) is rejected, with the draft's row as it is, and
 *   sets MLA_DEVERR_TOKEN.  A row without weight draws -1 and sets it too.  A
 *   sequence with more than max_out rows is refused (MLA_DEVERR_SEQLEN): it
 *   accepts nothing, its tokens are -1, its length stays.  So are all
 *   sequences when row_start decreases or leaves [0, rows] anywhere.
 *   Sums are good to 2^-40 of the row's, the comparison is exact.
 *   vocab <= 2^22, batch <= 4096; batch == 0 is a no-op.
 */
#define MLA_PROB_FP32 0
#define MLA_PROB_BF16 1
#define MLA_PROB_FP16 2
mla_status mla_verify_drafts(const void* target_probs, int64_t target_row_stride, const void* draft_probs,
                             int64_t draft_row_stride, int32_t prob_type, int32_t vocab, const int32_t* drafts,
                             const int32_t* row_start, int32_t batch, int32_t rows, const float* u_accept,
                             const float* u_sample, const int32_t* seq_lens, int32_t* accepted, int32_t* tokens,
                             int32_t max_out, int32_t* kept_lens, int32_t* dev_err, mla_stream_t stream);

/*
 * mla_token_mass - adds up the attention weight that every cached token
 * received from a step's queries, all heads together:
 *   mass[slot(t)] = m + sum_{i, h} exp(s_{i,h}(t) - lse_{i,h})
 * over the queries i that see t, with the scores s of mla_decode_absorbed and
 * the lse that it (or mla_prefill_absorbed) returned; m = decay * mass
 * [slot(t)] for t < counted[b], else 0 (tokens that are new in their slot).
 * Sequence b's queries are rows q_start[b] .. q_start[b + 1] - 1, the last of
 * its seq_lens[b] tokens: query i (of n) sees positions t <= seq_lens[b] - n +
 * i.  They may be fewer than the step's new tokens (an observation window).
 *   q_lat   fp32 [n_tokens][H][512], q_pe bf16 [n_tokens][H][64], lse fp32
 *           [n_tokens][H] (natural log; a row whose lse is not finite adds nothing).
 *           mla_chunk_attention returns neither q_lat nor lse.  For queries of
 *           a ragged batch they come from mla_q_absorb and a second attention:
 *           one mla_decode_absorbed whose sequences are the queries (each its
 *           sequence's block_table row, and as many tokens as it sees: the
 *           cache is read once a query), or one mla_prefill_absorbed a
 *           sequence, whose context length lives on the host
 *   block_table int32 [B][max_pages], q_start int32 [B + 1], seq_lens int32 [B]
 *   counted int32 [B]: tokens whose mass is up to date; NULL: seq_lens[b] - n
 *   max_new bound on every n (host; at most n_tokens)
 *   mass    fp32 [num_pages * 64], by cache slot
 *   workspace: device, >= mla_mass_workspace_bytes(...) bytes, 256-byte
 *           aligned; contents are scratch, so calls that may overlap need
 *           their own
 *   A page id outside the pool is passed over and sets MLA_DEVERR_PAGE.  A
 *   sequence whose figures do not fit (n > max_new, 0 < seq_lens[b] < n,
 *   seq_lens[b] < 0 or > max_pages * 64, counted[b] not in [0, seq_lens[b]])
 *   is left alone and sets MLA_DEVERR_SEQLEN; so are all when q_start
 *   decreases or leaves [0, n_tokens].  Sequences without queries are left
 *   alone.  Sequences of a call must not share pages.
 *   Precision: queries and cached values as two fp16 halves (22 bits), products
 *   summed by the tensor cores, which cut a running sum off at 24 bits (what that
 *   takes on average is given back), exponentials and masses in fp32.  A weight
 *   is off by its score's error: 1e-6 of it for scores of a nat or so, and in
 *   proportion to larger ones, on average within 5e-7 of the score (1.2e-6 of it for
 *   one query of 16 heads over bf16), single weights within 2^-16 of the sum of
 *   the score's |products|.  A cached value beyond 4094 in magnitude, or a query
 *   beyond 2047 after the scale and log2 e, may count as non-finite: its token's
 *   mass, or that of all tokens the query sees, is then not finite.  A cached
 *   value below 2^-7 is off by up to 2^-29.
 *   A wait that runs out (mla_set_wait_limit_ns) sets MLA_DEVERR_TIMEOUT and
 *   leaves the call's masses undefined.
 *   The same call gives the same bits.  batch <= 4096, n_tokens * H < 2^31;
 *   n_tokens == 0 or batch == 0 is a no-op.
 */
mla_status mla_token_mass(const mla_cache_layer* cache, const float* q_lat, const uint16_t* q_pe, const float* lse,
                          const int32_t* block_table, int32_t max_pages, const int32_t* q_start,
                          const int32_t* seq_lens, const int32_t* counted, int32_t batch, int32_t n_tokens,
                          int32_t heads, int32_t max_new, float softmax_scale, float decay, void* workspace,
                          size_t workspace_bytes, float* mass, int32_t* dev_err, mla_stream_t stream);

/* Bytes of device workspace mla_token_mass needs; 0 for invalid arguments. */
size_t mla_mass_workspace_bytes(int32_t batch, int32_t n_tokens, int32_t heads, int32_t max_new);

/*
 * mla_select_tokens - the tokens of each sequence that stay when it is cut to
 * keep_lens[b]: the first `sinks`, the last `recent` and, of those in
 * between, the ones with the largest mass (ties: the lower position; a NaN,
 * and a token on a page outside the pool, which sets MLA_DEVERR_PAGE, counts
 * as the smallest).  Where keep_lens is small, sinks come first, then recent.
 *   mass    fp32 [num_pages * 64], by cache slot
 *   keep_lens int32 [B], 0 and more; not below seq_lens: nothing is cut
 *   kept    int32 [B][max_keep]: the positions that stay, increasing, -1
 *           behind (all positions, as far as they fit, where nothing is cut)
 *   kept_lens int32 [B]: min(keep_lens, seq_lens); must not overlap seq_lens or
 *           keep_lens
 *   A sequence with keep_lens < 0, or with max_keep < keep_lens < seq_lens,
 *   is not cut and sets MLA_DEVERR_SEQLEN; a seq_lens outside [0, max_pages *
 *   64] counts as 0 and sets it.
 *   max_pages <= 2^24, batch <= 4096; batch == 0 is a no-op.
 */
mla_status mla_select_tokens(const float* mass, int32_t num_pages, const int32_t* block_table, int32_t max_pages,
                             const int32_t* seq_lens, const int32_t* keep_lens, int32_t batch, int32_t sinks,
                             int32_t recent, int32_t* kept, int32_t max_keep, int32_t* kept_lens, int32_t* dev_err,
                             mla_stream_t stream);

/*
 * mla_release_pages - page tables and the free list after requests got
 * shorter, from old_lens[b] to new_lens[b] tokens.
 *   move 0  the last tokens go (rejected drafts): the pages behind the new
 *           length are given back
 *   move 1  a request with new_lens < old_lens gets fresh pages for its new
 *           length and gives all its old ones back; one with new_lens ==
 *           old_lens keeps its pages
 *   block_table int32 [B][max_pages]: the requests' pages (mla_plan_chunks's
 *           output), read only
 *   req     int32 [B]: each request's row of page_table (move 1; else may be NULL)
 *   page_table int32 [rows][max_pages]: move 1: the fresh pages are written
 *           into it, other entries stay (may be NULL for move 0)
 *   free_pages int32 [free_len], free_range {head, tail}: as for the plan,
 *           entries head .. tail - 1 are available.  Fresh pages are taken
 *           from free_pages[head] on, pages given back are then written in
 *           front of the first entry left, both in the order of the batch
 *   new_table int32 [B][max_pages]: the requests' pages, -1 behind the last
 *   lens_out int32 [B]: new_lens, or old_lens for a refused request
 *   free_range_out int32 [2]: the next call's free_range (not free_range
 *           itself): {head + pages taken - pages given back, tail}
 *   No output may overlap an input or another output (MLA_ERR_INVALID_ARG),
 *   apart from page_table and free_pages being changed in place.
 *   A request is refused and stays as it was, while the others go on, when
 *   its lengths do not fit (MLA_DEVERR_SEQLEN; an old length outside [0,
 *   max_pages * 64] counts as 0), when its req is out of range or named twice
 *   (move 1; MLA_DEVERR_PAGE), or when the list has too few pages left or too
 *   few places in front (MLA_DEVERR_NO_PAGES: nobody behind it gets any
 *   either).  A page id outside the pool is written as -1 and sets
 *   MLA_DEVERR_PAGE; a bad free_range counts as empty, without places, and
 *   sets it too.  A move writes over list entries that it took, so it is made
 *   once; a trim made again writes the same.
 *   rows <= 65536; batch <= 4096; batch == 0 is a no-op.
 */
mla_status mla_release_pages(const int32_t* old_lens, const int32_t* new_lens, const int32_t* req, int32_t batch,
                             const int32_t* block_table, int32_t* page_table, int32_t rows, int32_t max_pages,
                             int32_t* free_pages, int32_t free_len, const int32_t* free_range, int32_t num_pages,
                             int32_t move, int32_t* new_table, int32_t* lens_out, int32_t* free_range_out,
                             int32_t* dev_err, mla_stream_t stream);

/*
 * mla_move_tokens - moves the tokens that stay: token j < lens[b] of sequence
 * b's pages in dst_table becomes token kept[b][j] of its pages in src_table,
 * in the stored form, bit for bit; with mass, their mass too.  A sequence with
 * lens[b] == seq_lens[b] stays where it is.
 *   src_table, dst_table int32 [B][max_pages]: the old pages and the fresh
 *           ones (no page of one may be a page of the other that the call
 *           touches, or be named twice in dst_table)
 *   seq_lens int32 [B]: tokens in the old pages
 *   kept    int32 [B][max_keep] of mla_select_tokens; lens int32 [B]:
 *           mla_release_pages's lens_out
 *   mass    fp32 [num_pages * 64], by cache slot, or NULL
 *   The kept tokens' k_pe keep the rotation of their old positions, while the
 *   next mla_plan_chunks counts positions on from the shortened cache: so that
 *   new tokens keep their distances to those kept, add to its positions,
 *   before mla_rope, the tokens that the request lost so far (seq_lens - lens,
 *   summed over its moves).
 *   Slots behind a sequence's last token are left as they were.  A kept
 *   position outside the sequence (MLA_DEVERR_SLOT) or a page id outside the
 *   pool (MLA_DEVERR_PAGE) leaves the new token's slot as it was; a sequence
 *   whose lens do not fit (negative, above seq_lens or max_keep; seq_lens
 *   outside [0, max_pages * 64]) is left alone and sets MLA_DEVERR_SEQLEN.
 *   batch <= 4096; batch == 0 is a no-op.
 */
mla_status mla_move_tokens(const mla_cache_layer* cache, const int32_t* src_table, const int32_t* seq_lens,
                           const int32_t* kept, int32_t max_keep, const int32_t* lens, const int32_t* dst_table,
                           int32_t max_pages, int32_t batch, float* mass, int32_t* dev_err, mla_stream_t stream);

/* Static string for a status code. */
const char* mla_status_string(mla_status status);

/* Text of the CUDA error behind the calling thread's most recent
 * MLA_ERR_CUDA ("no error" if none); a static string, not to be freed. */
const char* mla_last_cuda_error(void);

/*
 * mla_set_wait_limit_ns - bound, in nanoseconds, on every wait inside the
 * decode kernels (stage arrivals, the hand-offs between the block's warp
 * roles) of the decode, prefill, chunk and mass calls this process launches afterwards;
 * returns the previous bound, or -1 (nothing changed) for ns < 0.  The
 * default is 10 s.  A test and diagnostic hook, not part of the pages'
 * method: a wait that runs out sets MLA_DEVERR_TIMEOUT in *dev_err, and its
 * block writes empty partials (weight 0) for the rest of its share of the
 * context and leaves once its own bulk copies have landed.  Nothing traps
 * and the outputs stay finite, but they miss that share of the context.
 * With ns = 0 a wait polls without suspending and gives up once the GPU's
 * global timer has advanced (within about a microsecond) without completion.
 */
int64_t mla_set_wait_limit_ns(int64_t ns);

/* ABI version (major * 100 + minor). */
int32_t mla_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* MLA_GB300_H */
