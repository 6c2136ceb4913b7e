// Chunk attention of sequences with many new tokens (long path): the cached
// latents are expanded once per head into keys and values,
//   K[h][t] = [W_UK[h] c_hat[t]; kpe_hat[t]]  (192),   V[h][t] = c_hat[t] W_UV[h]  (128),
// and attention runs on those: 2 x 320 operations per (query, head, key)
// against the absorbed form's 2 x 1088, for 2 x 512 x 256 per (key, head).
//
// Three kernels over fp16 tiles in the workspace, all tiles stored as 128-row
// x 64-channel blocks of 16 KB in the swizzled order that the MMAs read, so
// that a tile moves as plain bulk copies:
//   long_prep_kernel    dequantizes the latents (and converts the weights)
//   long_expand_kernel  K and V tiles: a tcgen05 GEMM, one key tile's latents
//                       resident, the heads' weights streaming
//   long_attention_kernel  two 128-row query tiles of one head against the
//                       head's key tiles, online softmax
// Work is split as on the short path: all units in order, cut into equal
// runs, one per SM; query tiles that fall into several runs leave fp32
// partials that long_combine_kernel merges in block order.
//
// What bounds it: the MMAs.  Measured, call after call: 8192 tokens on their own, 64
// heads, INT8: 1.21 to 1.25 ms, 1.25 to 1.21 PFLOP/s of the formula's operations (64 to
// 66% of a library matrix product's rate in a short burst, 71 to 74% of its rate
// under the power limit); 2048 tokens after 32768, 16 heads: 0.63 ms (72 and 80%); in a
// burst of 20 ms, before the power limit acts, 1.13 and 0.58 ms; 54.9 and 5.9 ms for
// the absorbed form's kernel.
//
// Rounding: latents, weights, keys, values, queries and P are fp16 (2^-11
// relative each; bf16 queries and weights convert exactly within fp16's normal
// range), all sums, scores, maxima and outputs fp32 until o is written.
#include <math.h>

#include "chunk.cuh"
#include "dequant.cuh"
#include "tc.cuh"

namespace mla {
namespace {

using namespace tc;

// ---------------------------------------------------------------------------
// long_prep_kernel: block x < 4 tiles: a 32-token block of a key tile, lane =
// token, warp w dequantizes units w and w + 8, warps 0 and 1 the RoPE units;
// the rows leave as 4 KB bulk stores (a lane's own 16-byte stores to its row
// would touch 32 lines each).  Bound by latency: the cache's block, its
// conversion and the store follow one another, up to seven blocks per SM overlap;
// 34816 tokens of INT8 and the weights of 16 heads: 19 us.
// The blocks behind convert 64 latent channels of a head's weights each.
// ---------------------------------------------------------------------------
constexpr int kPrepThreads = 256;
constexpr int kPrepRows = 32 * 128;        // a block's 32 rows of one 64-channel block: 4 KB

// 32 channels of a row into a 128-byte row of a swizzled block.
__device__ __forceinline__ void put_rows(uint8_t* blk, int row, int c16, const uint32_t* h) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    *reinterpret_cast<uint4*>(blk + row * 128 + (((c16 + i) ^ (row & 7)) << 4)) =
        make_uint4(h[4 * i], h[4 * i + 1], h[4 * i + 2], h[4 * i + 3]);
}

__device__ void convert_weights(const ChunkParams& p, int h, int st) {
  uint8_t* out = p.w_tiles + (int64_t)h * kWHead + st * kBlkBytes;
  for (int i = threadIdx.x; i < 2 * 128 * 8; i += kPrepThreads) {
    // W_UK: rows d, 64 channels (K-major); W_UV: rows c, 128 values as two blocks of 64 (MN-major)
    const bool uk = i < 1024;
    const int row = (i & 1023) >> (uk ? 3 : 4), c = i & (uk ? 7 : 15);
    const uint16_t* src = uk ? p.w_uk + ((int64_t)h * kDn + row) * kDc + 64 * st + 8 * c
                             : p.w_uv + ((int64_t)h * kDc + 64 * st + row) * kDv + 8 * c;
    const uint4 v = __ldcg(reinterpret_cast<const uint4*>(src));
    uint8_t* blk = uk ? out : out + 8 * kBlkBytes + (c >> 3) * 8192;
    *reinterpret_cast<uint4*>(blk + row * 128 + (((c & 7) ^ (row & 7)) << 4)) =
        make_uint4(half2_bits(bf16lo(v.x), bf16hi(v.x)), half2_bits(bf16lo(v.y), bf16hi(v.y)),
                   half2_bits(bf16lo(v.z), bf16hi(v.z)), half2_bits(bf16lo(v.w), bf16hi(v.w)));
  }
}

template <int LF, int KF>
__global__ void __launch_bounds__(kPrepThreads) long_prep_kernel(const ChunkParams p, int key_blocks) {
  constexpr int kBlock = block_bytes<LF, KF>();
  extern __shared__ __align__(1024) uint8_t prep_smem[];
  uint8_t* out = prep_smem;                // 8 latent blocks' rows and the RoPE keys'
  uint8_t* raw = prep_smem + kQBlocks * kPrepRows;
  __shared__ uint64_t bar;
  __shared__ uint32_t s_bad;
  pdl_launch_dependents();
  pdl_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if ((int)blockIdx.x >= key_blocks) {
    const int w = blockIdx.x - key_blocks;
    if (__ldcg(&p.counts->l_seqs) > 0) convert_weights(p, w >> 3, w & 7);
    return;
  }
  const int tile = blockIdx.x >> 2, sub = blockIdx.x & 3;
  if (tile >= __ldcg(&p.counts->l_tiles)) return;
  int k = 0, n = __ldcg(&p.counts->l_seqs);          // the sequence: last with kv0 <= tile
  while (n - k > 1) {
    const int mid = (k + n) >> 1;
    if (__ldcg(&p.l_seqs[mid].kv0) <= tile) k = mid;
    else n = mid;
  }
  const int kv0 = __ldcg(&p.l_seqs[k].kv0), len = __ldcg(&p.l_seqs[k].len), b = __ldcg(&p.l_seqs[k].b);
  const int t0 = (tile - kv0) * kLongKeys + 32 * sub;
  const int n_tok = min(32, max(0, len - t0));
  const int page = n_tok > 0 ? __ldcg(p.block_table + (int64_t)b * p.max_pages + t0 / kPage) : 0;
  const bool page_ok = page >= 0 && page < p.num_pages;
  const bool read = page_ok && n_tok > 0;
  if (tid == 0) {
    bar_init(smem_u32(&bar), 1);
    bar_init_fence();
    s_bad = 0;
    if (!page_ok) set_err(p.dev_err, MLA_DEVERR_PAGE);
  }
  __syncthreads();
  if (tid == 0 && read) {
    bar_expect(smem_u32(&bar), kBlock);
    bulk_copy(smem_u32(raw), p.pool + (int64_t)page * p.L.page_bytes + ((t0 >> 5) & 1) * p.L.block_bytes, kBlock, smem_u32(&bar));
  }
  bool arrived = true;
  if (read) {
    volatile int never = 0;
    arrived = bar_wait(smem_u32(&bar), 0, p.wait_ns, &never);
    if (!arrived) {                        // any thread's: the limit may end between two of them
      set_err(p.dev_err, MLA_DEVERR_TIMEOUT);
      drain_wait(smem_u32(&bar), 0);
    }
  }
  const bool live = read && arrived && lane < n_tok;
  bool fine = true;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int unit = warp + 8 * i;
    RawUnit<LF, false> r;
    uint32_t h[16];
    if (live) load_unit<LF, false>(raw, p.L, lane, unit, r);
    else zero_unit(r);
    fine &= convert_unit<LF, false>(r, h);
    if (live) fine &= patch_outliers<LF>(raw, p.L, p.outl, lane, unit, h);
    put_rows(out + (unit >> 1) * kPrepRows, lane, 4 * (unit & 1), h);
  }
  if (warp < 2) {
    RawUnit<KF, true> r;
    uint32_t h[16];
    if (live) load_unit<KF, true>(raw, p.L, lane, warp, r);
    else zero_unit(r);
    fine &= convert_unit<KF, true>(r, h);
    put_rows(out + 8 * kPrepRows, lane, 4 * warp, h);
  }
  if (!fine) atomicOr(&s_bad, 1u << lane);
  fence_async_smem();
  __syncthreads();
  if (tid == 0) {
    for (int c = 0; c < kQBlocks; ++c)
      bulk_store((c < 8 ? p.c_tiles + (int64_t)tile * kCTile + c * kBlkBytes : p.k_rope + (int64_t)tile * kBlkBytes) + sub * kPrepRows,
                 smem_u32(out + c * kPrepRows), kPrepRows);
    bulk_store_commit();
    p.kflags[8 * tile + sub] = s_bad;
    p.kflags[8 * tile + 4 + sub] = page_ok ? 0u : 0xFFFFFFFFu;
    bulk_store_done();
  }
}

// ---------------------------------------------------------------------------
// long_expand_kernel: a unit is (key tile, head), tile-major.  The tile's latents
// stay in TMEM (128 lanes x 256 columns of fp16 pairs) as the A operand while
// the heads' weights stream through shared memory, 16 KB (64 latent channels
// of W_UK or of W_UV) per item, four M = 128, N = 128 MMAs each.  A head's keys
// and values are 128 TMEM columns each; while one half is computed the other
// leaves, through 32 KB of shared memory as bulk stores.
// What bounds it: 4100 cycles of MMAs per unit, and the weights' 64 bytes per
// cycle and SM from L2, whose latency wants 100 KB and more under way: that is
// why the latents are not in shared memory (64 KB under way: 10000 cycles per
// unit).  Every block fetches its own items with plain copies.
// Measured: 34816 tokens, 16 heads: 106 us, 5100 cycles per unit (81% of the MMAs'
// rate); with the latents in shared memory and 64 KB of weights under way 136 us.
// Warps: 0 copies, 1 MMAs, 4..7 epilogue (and the latents' way into TMEM).
// ---------------------------------------------------------------------------
constexpr int kExThreads = 256;
constexpr int kExItems = 11;
constexpr int kExOut = kExItems * kBlkBytes;
constexpr int kExBars = kExOut + 2 * kBlkBytes;
constexpr int kExSmem = kExBars + 512 + 1024;
static_assert(kExSmem <= 232448, "a block's shared memory");
enum { xFull = 0, xEmpty = xFull + kExItems, xA = xEmpty + kExItems, xD, xDFree = xD + 2, xFin = xDFree + 2, xCount };

__global__ void __launch_bounds__(kExThreads, 1) long_expand_kernel(const ChunkParams p) {
  extern __shared__ uint8_t ex_smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(ex_smem_raw) + 1023) & ~(uintptr_t)1023);
  const uint32_t sb = smem_u32(sm), bars = sb + kExBars;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + kExBars + 8 * xCount);
  volatile int* abort = reinterpret_cast<volatile int*>(sm + kExBars + 8 * xCount + 4);
  volatile int* quit = reinterpret_cast<volatile int*>(sm + kExBars + 8 * xCount + 8);       // [2, by unit parity]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    quit[0] = quit[1] = 0;
    for (int i = 0; i < xCount; ++i)
      bar_init(bars + 8 * i, i == xA || i == xDFree || i == xDFree + 1 ? 128 : 1);
    *abort = 0;
    bar_init_fence();
  }
  if (warp == 1) tmem_alloc(smem_u32(tmem_slot), 512);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tbase = *tmem_slot, t_d = tbase + 256;
  pdl_launch_dependents();
  pdl_wait();
  const int64_t U = (int64_t)__ldcg(&p.counts->l_tiles) * p.H;
  const int64_t lo = U * blockIdx.x / gridDim.x, hi = U * (blockIdx.x + 1) / gridDim.x;
  bool ok = true;
  if (warp == 0) {
    if (elect_one() && hi > lo) {
      uint32_t it = 0;
      for (int64_t u = lo; u < hi && ok; ++u) {
        const uint8_t* src = p.w_tiles + (u % p.H) * kWHead;
        for (int st = 0; st < 16; ++st, ++it) {
          const uint32_t s = it % kExItems;
          if (it >= kExItems && !bar_wait(bars + 8 * (xEmpty + s), (it / kExItems - 1) & 1, p.wait_ns, abort)) {
            ok = false;
            break;
          }
          bar_expect(bars + 8 * (xFull + s), kBlkBytes);
          bulk_copy(sb + s * kBlkBytes, src + st * kBlkBytes, kBlkBytes, bars + 8 * (xFull + s));
        }
      }
      if (!ok) {
        set_err(p.dev_err, MLA_DEVERR_TIMEOUT);
        *abort = 1;
      }
      for (uint32_t s = 0; s < kExItems; ++s)
        if (it > s) drain_wait(bars + 8 * (xFull + s), ((it - 1 - s) / kExItems) & 1);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (elect_one() && hi > lo) {
      constexpr uint32_t kIdK = f16_idesc(128, 128, false, false), kIdV = f16_idesc(128, 128, false, true);
      const uint64_t d_uk = sw128_desc(sb, 16, 1024), d_uv = sw128_desc(sb, 8192, 1024);
      uint32_t it = 0, na = 0, nd = 0;
      for (int64_t u = lo; u < hi && ok; ++u, ++nd) {
        if (u == lo || u % p.H == 0) {
          if (!bar_wait(bars + 8 * xA, na & 1, p.wait_ns, abort)) {
            ok = false;
            break;
          }
          ++na;
        }
        for (int half = 0; half < 2 && ok; ++half) {
          if (nd >= 1 && !bar_wait(bars + 8 * (xDFree + half), (nd - 1) & 1, p.wait_ns, abort)) {
            ok = false;
            break;
          }
          for (int st = 0; st < 8; ++st, ++it) {
            const uint32_t s = it % kExItems;
            if (!bar_wait(bars + 8 * (xFull + s), (it / kExItems) & 1, p.wait_ns, abort)) {
              ok = false;
              break;
            }
            fence_after();
            const uint64_t w = (uint64_t)(s * (kBlkBytes >> 4));
            if (half == 0) umma4_ta<2>(t_d, tbase + 32 * st, d_uk + w, kIdK, st != 0);
            else umma4_ta<(2048 >> 4)>(t_d + 128, tbase + 32 * st, d_uv + w, kIdV, st != 0);
            umma_commit(bars + 8 * (xEmpty + s));
          }
          if (ok) umma_commit(bars + 8 * (xD + half));
        }
      }
      if (!ok) {
        set_err(p.dev_err, MLA_DEVERR_TIMEOUT);
        *abort = 1;
      }
      umma_commit(bars + 8 * xFin);
      drain_wait(bars + 8 * xFin, 0);
    }
    __syncwarp();
  } else if (warp >= 4) {
    // The four warps meet twice per half: when the staging blocks are free, and
    // when they are filled; one that gave up a wait says so before the meeting.
    const int w = warp & 3, row = 32 * w + lane;
    const uint32_t tl = (uint32_t)(32 * w) << 16;
    uint8_t* stage = sm + kExOut;
    uint32_t nd = 0;
    for (int64_t u = lo; u < hi && ok; ++u, ++nd) {
      const uint32_t g = nd & 1;
      const int tile = (int)(u / p.H);
      if (u == lo || u % p.H == 0) {
        // The latents into TMEM, a row per lane (the last tile's MMAs are done,
        // their results have been read).  A warp reads its 32 rows of four
        // blocks at a time, side by side, and turns them through its quarter of
        // the staging blocks.
        if (threadIdx.x == 128) bulk_store_read_done();
        asm volatile("bar.sync 1, 128;\n" ::: "memory");
        const uint8_t* src = p.c_tiles + (int64_t)tile * kCTile + w * 4096 + lane * 16;
        uint8_t* mine = stage + w * 8192;
#pragma unroll 1
        for (int c0 = 0; c0 < 8; c0 += 4) {
          uint4 v[4][8];
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int e = 0; e < 8; ++e) v[c][e] = __ldcg(reinterpret_cast<const uint4*>(src + (c0 + c) * kBlkBytes + 512 * e));
#pragma unroll
          for (int c2 = 0; c2 < 4; c2 += 2) {
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
              for (int e = 0; e < 8; ++e) *reinterpret_cast<uint4*>(mine + 4096 * c + 512 * e + lane * 16) = v[c2 + c][e];
            __syncwarp();
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              uint32_t r[32];
#pragma unroll
              for (int e = 0; e < 8; ++e)
                *reinterpret_cast<uint4*>(r + 4 * e) =
                    *reinterpret_cast<const uint4*>(mine + 4096 * c + lane * 128 + ((e ^ (lane & 7)) << 4));
              tmem_store32(tbase + 32 * (c0 + c2 + c) + tl, r);
            }
            __syncwarp();
          }
        }
        fence_before();
        bar_arrive(bars + 8 * xA);
      }
      uint8_t* out = p.kv_tiles + ((int64_t)tile * p.H + u % p.H) * kHeadTile;
      bool fine = true;
      for (int half = 0; half < 2; ++half) {               // keys, values
        if (!warp_wait(bars + 8 * (xD + half), nd & 1, p.wait_ns, abort)) quit[g] = 1;
        if (threadIdx.x == 128) bulk_store_read_done();
        asm volatile("bar.sync 1, 128;\n" ::: "memory");
        if (quit[g]) {
          ok = false;
          break;
        }
        fence_after();
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {      // 32 columns: half a block
          uint32_t r[32], hw[16];
          tmem_load32(t_d + 128 * half + 32 * c + tl, r);
          __half2 acc = __float2half2_rn(0.f);
          const __half2 zero = acc;
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            hw[i] = half2_bits(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
            acc = __hfma2(*reinterpret_cast<const __half2*>(&hw[i]), zero, acc);
          }
          if (__hisnan(__low2half(acc)) || __hisnan(__high2half(acc))) {
            fine = false;
#pragma unroll
            for (int i = 0; i < 16; ++i) hw[i] = 0u;
          }
          put_rows(stage + (c >> 1) * kBlkBytes, row, 4 * (c & 1), hw);
          __syncwarp();
        }
        fence_before();
        bar_arrive(bars + 8 * (xDFree + half));            // TMEM has been read
        fence_async_smem();
        asm volatile("bar.sync 1, 128;\n" ::: "memory");
        if (threadIdx.x == 128) {
          bulk_store(out + half * 2 * kBlkBytes, sb + kExOut, 2 * kBlkBytes);
          bulk_store_commit();
        }
      }
      if (ok && !fine) atomicOr(p.kflags + 8 * tile + w, 1u << lane);
    }
    if (threadIdx.x == 128) bulk_store_done();
    if (!ok) {
      set_err(p.dev_err, MLA_DEVERR_TIMEOUT);
      *abort = 1;
    }
  }
  fence_before();
  __syncthreads();
  if (warp == 1) {
    fence_after();
    tmem_free(tbase, 512);
  }
}

// ---------------------------------------------------------------------------
// long_attention_kernel.  An item is 256 query tokens of one head: two tiles
// of 128 rows that share the head's key tiles.  While the softmax warps of
// one tile work, the MMAs of the other run:
//   S_0(j+1) = Q_0 K(j+1)^T after O_0 += P_0(j) V(j), then the same for tile 1.
// P replaces its S in TMEM (fp16, half the columns) and is the A operand from
// there.  Per key tile 2 x (12 + 8) MMAs of M = N = 128, 65 cycles each: 2600
// cycles bound it; the softmax's 2 x 128 x 128 exponentials take less.
// TMEM: S_0, S_1, O_0, O_1, 128 columns each.  Shared memory: the two query
// tiles (96 KB) and a ring of eight 16 KB blocks that carries, per key tile,
// two K blocks, the RoPE keys, two V blocks.
// Measured (profiler): 2048 tokens after 32768, 16 heads: 412 us, tensor pipe 77%
// active, 0.34 GB from DRAM (460 us and 2.3 GB while runs began with their first
// item).  8192 tokens on their own, 64 heads: tensor pipe 71% active, 3.8 GB from
// DRAM, since the keys and values (268 MB) exceed L2: with all heads on four
// heads' tiles, so that L2 holds them, a call takes 10% less.  Cutting the runs in
// two or four, to work on fewer heads at a time, costs more in split items than
// it saves (2% and 4% slower).
// Warps: 0..3 and 4..7 softmax (thread = row), 8 copies, 9 MMAs, 10 fetches the
// next item's query rows to L2.
// ---------------------------------------------------------------------------
constexpr int kLaThreads = 384;
constexpr int kRing = 8;
constexpr int kLaRing = 6 * kBlkBytes;
constexpr int kLaBars = kLaRing + kRing * kBlkBytes;
constexpr int kLaSmem = kLaBars + 256 + 1024;
static_assert(kLaSmem <= 232448, "a block's shared memory");
// Registers: 384 threads launch with 168 each (64,512): then 216 for the
// softmax warps, 72 for the others.
constexpr int kLaRegsSoftmax = 216, kLaRegsIssue = 72;
static_assert(256 * kLaRegsSoftmax + 128 * kLaRegsIssue <= kLaThreads * 168 && kLaThreads * 168 <= 65536 &&
                  kLaThreads * 176 > 65536,
              "the warpgroups' shares come out of the launch's registers");
enum { aFull = 0, aEmpty = aFull + kRing, aQ = aEmpty + kRing, aS = aQ + 2, aP = aS + 2, aO = aP + 2, aFin = aO + 2, aCount };

// A run's segments (a pair of query tiles of one head, key tiles t0 .. t1), the
// last one first: the runs that share a head then read its tiles nearly in
// step.  A run shorter than an item has its end in the middle of one: the
// beginnings of items, read first, start together, and what is left of the
// items before follows at the same distance behind in every run, so a tile
// is still in L2 when its other readers come by.
struct LongWalk {
  const LongSeq* seqs;
  int k;
  int64_t lo, u;                   // the run's first unit, and the first one behind what is left
  LongSeq s;
  int h, pair, t0, t1, tiles0;     // tiles0: key tiles the pair's first query tile sees
  bool started, first, last, two;  // two: the pair has a second query tile

  __device__ __forceinline__ void load() {
    const int4* r = reinterpret_cast<const int4*>(seqs + k);
    int4* d = reinterpret_cast<int4*>(&s);
    d[0] = __ldcg(r);
    d[1] = __ldcg(r + 1);
    d[2] = __ldcg(r + 2);
  }
  __device__ __forceinline__ void start(const ChunkParams& p, int64_t lo_, int64_t hi) {
    seqs = p.l_seqs;
    lo = lo_;
    u = hi;
    started = false;
    int n = __ldcg(&p.counts->l_seqs);
    k = 0;
    while (n - k > 1) {
      const int mid = (k + n) >> 1;
      if (__ldcg(&seqs[mid].unit0) < u) k = mid;
      else n = mid;
    }
    load();
  }
  __device__ __forceinline__ bool next(int H) {
    if (u <= lo) return false;
    if (!started) {                  // the run's first segment: the one of unit u - 1
      started = true;
      const int64_t d = u - 1 - s.unit0;
      h = (int)(d / s.per_head);
      int r = (int)(d % s.per_head);
      for (pair = 0; r >= pair_tiles(s.len - s.n, s.n, pair) + kPairCost; ++pair) r -= pair_tiles(s.len - s.n, s.n, pair) + kPairCost;
      if (r >= kPairCost) return begin(r + 1 - kPairCost);
      u -= r + 1;                    // the run ends before the pair's first key tile: its next one has the pair
      if (u <= lo) return false;
    }
    if (--pair < 0) {                // after it, item by item
      if (--h < 0) {
        --k;
        load();
        h = H - 1;
      }
      pair = (s.n - 1) / kLongRows;
    }
    return begin(pair_tiles(s.len - s.n, s.n, pair));
  }
  __device__ __forceinline__ bool begin(int end) {
    const int ctx = s.len - s.n, J = pair_tiles(ctx, s.n, pair);
    t1 = end;
    t0 = (int)max((int64_t)0, end - (u - lo));
    first = t0 == 0;
    last = t1 == J;
    two = s.n > pair * kLongRows + 128;
    tiles0 = two ? (ctx + pair * kLongRows + 128 + kLongKeys - 1) / kLongKeys : J;
    u -= t1 - t0 + (first ? kPairCost : 0);
    return true;
  }
};

__global__ void __launch_bounds__(kLaThreads, 1) long_attention_kernel(const ChunkParams p) {
  extern __shared__ uint8_t la_smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(la_smem_raw) + 1023) & ~(uintptr_t)1023);
  const uint32_t sb = smem_u32(sm), bars = sb + kLaBars;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + kLaBars + 8 * aCount);
  volatile int* abort = reinterpret_cast<volatile int*>(sm + kLaBars + 8 * aCount + 4);
  volatile uint32_t* begun = reinterpret_cast<volatile uint32_t*>(sm + kLaBars + 8 * aCount + 8);    // segments whose MMAs have begun
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < aCount; ++i) bar_init(bars + 8 * i, (i >= aQ && i < aS) || (i >= aP && i < aO) ? 128 : 1);
    *abort = 0;
    *begun = 0;
    bar_init_fence();
  }
  if (warp == 9) tmem_alloc(smem_u32(tmem_slot), 512);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tbase = *tmem_slot;
  pdl_launch_dependents();
  pdl_wait();
  const int64_t U = __ldcg(&p.counts->l_units);
  const int G = (int)(U < gridDim.x ? U : gridDim.x), x = blockIdx.x;
  const bool work = x < G;
  const int64_t lo = work ? run_begin(U, x, G) : 0, hi = work ? run_begin(U, x + 1, G) : 0;
  bool ok = true;
  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kLaRegsSoftmax));
    // ---- softmax of query tile i, thread = row
    const int i = warp >> 2, row = threadIdx.x & 127;
    const uint32_t tl = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t t_s = tbase + 128 * i + tl, t_o = tbase + 256 + 128 * i + tl;
    const float sc = p.scale_log2;
    LongWalk wk;
    if (work) wk.start(p, lo, hi);
    uint32_t it = 0;                       // this tile's key tiles so far
    // Moves to the next segment that this query tile takes part in and hands
    // over its query rows as fp16, swizzled (padding rows are 0); false at the
    // run's end.  A warp loads its own 32 rows, eight lanes to a row.
    auto enter = [&]() -> bool {
      for (;;) {
        if (!wk.next(p.H)) return false;
        if (i == 1 && !wk.two) continue;
        if (i == 0 && wk.t0 >= wk.tiles0) {            // the run begins behind the first tile's last key: an empty partial
          float* part = p.l_parts + (int64_t)(2 * x + (wk.first ? 1 : 0)) * long_partial_floats();
#pragma unroll 4
          for (int c = 0; c < kDv / 4; ++c) reinterpret_cast<float4*>(part + row * kDv)[c] = make_float4(0.f, 0.f, 0.f, 0.f);
          part[kLongRows * kDv + row] = -INFINITY;
          part[kLongRows * kDv + kLongRows + row] = 0.f;
          continue;
        }
        break;
      }
      const int tok0 = wk.pair * kLongRows + 128 * i, piece = lane & 7;
      const uint16_t* qn = p.qn + wk.h * p.qn_head + 8 * piece;
      const uint16_t* qp = p.qp + wk.h * p.qp_head + 8 * piece;
      uint8_t* q = sm + i * 3 * kBlkBytes;
#pragma unroll
      for (int e0 = 0; e0 < 8; e0 += 4) {              // twelve loads in flight, then their stores
        uint4 v[4][3];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = 32 * (warp & 3) + 4 * (e0 + e) + (lane >> 3);
          const int64_t tok = wk.s.q0 + min(tok0 + r, wk.s.n - 1);
          v[e][0] = __ldcg(reinterpret_cast<const uint4*>(qn + tok * p.qn_tok));
          v[e][1] = __ldcg(reinterpret_cast<const uint4*>(qn + tok * p.qn_tok + 64));
          v[e][2] = __ldcg(reinterpret_cast<const uint4*>(qp + tok * p.qp_tok));
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = 32 * (warp & 3) + 4 * (e0 + e) + (lane >> 3);
#pragma unroll
          for (int c = 0; c < 3; ++c) {
            uint4 x = v[e][c];
            if (tok0 + r >= wk.s.n) x = make_uint4(0u, 0u, 0u, 0u);
            *reinterpret_cast<uint4*>(q + c * kBlkBytes + r * 128 + ((piece ^ (r & 7)) << 4)) =
                make_uint4(half2_bits(bf16lo(x.x), bf16hi(x.x)), half2_bits(bf16lo(x.y), bf16hi(x.y)),
                           half2_bits(bf16lo(x.z), bf16hi(x.z)), half2_bits(bf16lo(x.w), bf16hi(x.w)));
          }
        }
      }
      fence_async_smem();
      bar_arrive(bars + 8 * (aQ + i));
      return true;
    };
    bool more = work && enter();
    while (more) {
      const int t0 = wk.t0, t1 = i == 0 ? min(wk.t1, wk.tiles0) : wk.t1;
      const int tok0 = wk.pair * kLongRows + 128 * i, ctx = wk.s.len - wk.s.n;
      const bool live = tok0 + row < wk.s.n;
      const int qpos = ctx + tok0 + (live ? row : 0);
      const uint4* flags = reinterpret_cast<const uint4*>(p.kflags) + 2 * (int64_t)wk.s.kv0;
      float m = -INFINITY, l = 0.f;
      uint4 f_bad = __ldcg(flags + 2 * t0), f_out = __ldcg(flags + 2 * t0 + 1);
      for (int t = t0; t < t1; ++t, ++it) {
        const uint4 bad4 = f_bad, out4 = f_out;
        if (t + 1 < t1) {                  // fetched a tile ahead
          f_bad = __ldcg(flags + 2 * t + 2);
          f_out = __ldcg(flags + 2 * t + 3);
        }
        // S_i is complete, and the O_i of the tile before (its MMAs were issued first)
        if (!warp_wait(bars + 8 * (aS + i), it & 1, p.wait_ns, abort) ||
            (t > t0 && !warp_wait(bars + 8 * (aO + i), (it - 1) & 1, p.wait_ns, abort))) {
          ok = false;
          break;
        }
        fence_after();
        uint32_t s[128];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_load32(t_s + 32 * c, s + 32 * c);
        const uint32_t any_flag = bad4.x | bad4.y | bad4.z | bad4.w | out4.x | out4.y | out4.z | out4.w;
        const int seen = qpos - t * kLongKeys;         // keys 0 .. seen of the tile are visible
        if (any_flag) {
          const uint32_t fb[4] = {bad4.x, bad4.y, bad4.z, bad4.w}, fo[4] = {out4.x, out4.y, out4.z, out4.w};
#pragma unroll
          for (int c = 0; c < 128; ++c) {
            const bool hid = c > seen || ((fo[c >> 5] >> (c & 31)) & 1u);
            const bool nan = (fb[c >> 5] >> (c & 31)) & 1u;
            s[c] = hid ? 0xFF800000u : (nan ? 0x7FC00000u : s[c]);
          }
        } else if ((t + 1) * kLongKeys - 1 > ctx + tok0) {
#pragma unroll
          for (int c = 0; c < 128; ++c) s[c] = c > seen ? 0xFF800000u : s[c];
        }
        float mx = -INFINITY, my = -INFINITY;
#pragma unroll
        for (int c = 0; c < 128; c += 4) {
          mx = max3(mx, __uint_as_float(s[c]), __uint_as_float(s[c + 1]));
          my = max3(my, __uint_as_float(s[c + 2]), __uint_as_float(s[c + 3]));
        }
        mx = fmaxf(mx, my);
        const bool raise = (mx - m) * sc > kSlack;     // from -inf: the first key seen
        if (__any_sync(0xffffffffu, raise)) {
          const float alpha = raise ? ex2((m - mx) * sc) : 1.f;
          if (raise) m = mx;
          l *= alpha;
          if (t > t0) {
#pragma unroll 1
            for (int c = 0; c < 8; ++c) {
              uint32_t o[16];
              tmem_load16(t_o + 16 * c, o);
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
              tmem_store16(t_o + 16 * c, o);
            }
          }
        }
        const float ms = m == -INFINITY ? 0.f : kHead - m * sc;
        const uint64_t sc2 = pack2(sc, sc), ms2 = pack2(ms, ms);
        uint64_t la = pack2(0.f, 0.f), lb = la;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t pw[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            float a, b;
            unpack2(fma2(pack2(__uint_as_float(s[64 * c + 2 * e]), __uint_as_float(s[64 * c + 2 * e + 1])), sc2, ms2), a, b);
            a = ex2(a);
            b = ex2(b);
            uint64_t& acc = (e & 1) ? lb : la;
            acc = add2(acc, pack2(a, b));
            pw[e] = half2_bits(a, b);
          }
          tmem_store32(t_s + 32 * c, pw);
        }
        float l0, l1;
        unpack2(add2(la, lb), l0, l1);
        l += l0 + l1;
        fence_before();
        bar_arrive(bars + 8 * (aP + i));
      }
      if (!ok) break;
      // this segment's epilogue needs its place; the next one's query rows go
      // out first (the last S_i has read the old ones), so that its scores are
      // computed meanwhile
      const bool whole = wk.first && wk.last, opens = wk.first && !wk.last;       // whole: this block saw every key
      const int64_t out_row = (int64_t)(wk.s.q0 + tok0 + row) * p.H + wk.h;
      float* part = p.l_parts + (int64_t)(2 * x + (wk.first ? 1 : 0)) * long_partial_floats();
      const int64_t end = wk.u + kPairCost + pair_tiles(ctx, wk.s.n, wk.pair);       // of the item, if it begins here
      SplitRec rec;
      rec.rows = min(kLongRows, wk.s.n - wk.pair * kLongRows);
      rec.row0 = (int64_t)(wk.s.q0 + wk.pair * kLongRows) * p.H + wk.h;
      more = enter();
      if (!warp_wait(bars + 8 * (aO + i), (it - 1) & 1, p.wait_ns, abort)) {
        ok = false;
        break;
      }
      fence_after();
      const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        uint32_t o[32];
        tmem_load32(t_o + 32 * c, o);
        if (live) {
          if (whole) {
            uint4* dst = reinterpret_cast<uint4*>(p.o + out_row * kDv + 32 * c);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint32_t w[4];
#pragma unroll
              for (int q = 0; q < 4; ++q)
                asm("cvt.rn.bf16x2.f32 %0, %1, %2;\n"
                    : "=r"(w[q])
                    : "f"(__uint_as_float(o[8 * e + 2 * q + 1]) * inv), "f"(__uint_as_float(o[8 * e + 2 * q]) * inv));
              dst[e] = make_uint4(w[0], w[1], w[2], w[3]);
            }
          } else {
            uint4* dst = reinterpret_cast<uint4*>(part + (128 * i + row) * kDv + 32 * c);
#pragma unroll
            for (int e = 0; e < 8; ++e) dst[e] = make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
          }
        }
        __syncwarp();
      }
      if (!whole && live) {
        part[kLongRows * kDv + 128 * i + row] = m * sc;
        part[kLongRows * kDv + kLongRows + 128 * i + row] = l;
      }
      fence_before();
      if (opens && i == 0 && row == 0) {
        rec.first = x;
        rec.last = run_of(U, end - 1, G);
        rec.pad = 0;
        p.l_splits[atomicAdd(&p.counts->l_splits, 1)] = rec;
      }
    }
    if (!ok) {
      set_err(p.dev_err, MLA_DEVERR_TIMEOUT);
      *abort = 1;
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kLaRegsIssue));
    if (work && warp == 8 && elect_one()) {
      // ---- copies: K0 K1 RoPE V0 V1 of every key tile
      LongWalk wk;
      wk.start(p, lo, hi);
      uint32_t n = 0;
      while (ok && wk.next(p.H)) {
        for (int t = wk.t0; t < wk.t1 && ok; ++t) {
          const int64_t tile = wk.s.kv0 + t;
          const uint8_t* kv = p.kv_tiles + (tile * p.H + wk.h) * kHeadTile;
          if (t + 2 < wk.t1) {             // the ring reaches one tile ahead: L2 should have the next
            bulk_prefetch(kv + 2 * (int64_t)p.H * kHeadTile, kHeadTile);
            bulk_prefetch(p.k_rope + (tile + 2) * kBlkBytes, kBlkBytes);
          }
#pragma unroll 1
          for (int c = 0; c < 5; ++c, ++n) {
            const uint32_t s = n % kRing;
            if (n >= kRing && !bar_wait(bars + 8 * (aEmpty + s), (n / kRing - 1) & 1, p.wait_ns, abort)) {
              ok = false;
              break;
            }
            const uint8_t* src = c < 2 ? kv + c * kBlkBytes : (c == 2 ? p.k_rope + tile * kBlkBytes : kv + (c - 1) * kBlkBytes);
            bar_expect(bars + 8 * (aFull + s), kBlkBytes);
            bulk_copy(sb + kLaRing + s * kBlkBytes, src, kBlkBytes, bars + 8 * (aFull + s));
          }
        }
      }
      if (!ok) {
        set_err(p.dev_err, MLA_DEVERR_TIMEOUT);
        *abort = 1;
      }
      for (uint32_t s = 0; s < kRing; ++s)
        if (n > s) drain_wait(bars + 8 * (aFull + s), ((n - 1 - s) / kRing) & 1);
    } else if (work && warp == 10) {
      // ---- the next segment's query rows to L2 while this one runs.  No other
      // warp waits for this one, so it may be any number of segments late: it is
      // paced by a count that only grows (a barrier's parity could pass it twice
      // and leave it waiting for a phase that never comes).
      LongWalk wk;
      wk.start(p, lo, hi);
      const bool any = wk.next(p.H);
      for (uint32_t seg = 1; any && wk.next(p.H); ++seg) {
        for (int r = lane; r < kLongRows; r += 32) {
          const int tok = wk.pair * kLongRows + r;
          if (tok >= wk.s.n) break;
          const uint16_t* qn = p.qn + (int64_t)(wk.s.q0 + tok) * p.qn_tok + wk.h * p.qn_head;
          prefetch_line(qn);
          prefetch_line(qn + 64);
          prefetch_line(p.qp + (int64_t)(wk.s.q0 + tok) * p.qp_tok + wk.h * p.qp_head);
        }
        // one segment ahead, not more
        const uint64_t t0 = now_ns();
        while (*begun < seg && !*abort && now_ns() - t0 < p.wait_ns) __nanosleep(500);
      }
    } else if (work && warp == 9 && elect_one()) {
      // ---- MMAs
      LongWalk wk;
      wk.start(p, lo, hi);
      constexpr uint32_t kIdS = f16_idesc(128, 128, false, false), kIdO = f16_idesc(128, 128, false, true),
                         kIdO64 = f16_idesc(128, 64, false, true);
      const uint64_t d_q = sw128_desc(sb, 16, 1024), d_k = sw128_desc(sb + kLaRing, 16, 1024),
                     d_v = sw128_desc(sb + kLaRing, kBlkBytes, 1024);
      uint32_t n = 0;                      // ring blocks of the tiles before this one
      uint32_t nq[2] = {0, 0}, np[2] = {0, 0}, segs = 0;
      auto wait_slots = [&](uint32_t first, int count) -> bool {
        for (int c = 0; c < count; ++c)
          if (!bar_wait(bars + 8 * (aFull + (first + c) % kRing), ((first + c) / kRing) & 1, p.wait_ns, abort)) return false;
        return true;
      };
      auto scores = [&](int i, uint32_t at) -> bool {      // S_i = Q_i K^T, K in blocks at, at + 1, at + 2
#pragma unroll
        for (int c = 0; c < 3; ++c) {
          if (!wait_slots(at + c, 1)) return false;        // the second tile finds them there
          fence_after();
          umma4<2, 2>(tbase + 128 * i, d_q + (uint64_t)((i * 3 + c) * (kBlkBytes >> 4)),
                      d_k + (uint64_t)(((at + c) % kRing) * (kBlkBytes >> 4)), kIdS, c != 0);
        }
        umma_commit(bars + 8 * (aS + i));
        return true;
      };
      auto outputs = [&](int i, uint32_t at, uint32_t acc) {   // O_i += P_i V, V in blocks at, at + 1
        fence_after();
        const uint32_t s0 = at % kRing, d = tbase + 256 + 128 * i, a = tbase + 128 * i;
        const uint64_t v0 = d_v + (uint64_t)(s0 * (kBlkBytes >> 4));
        if (s0 + 1 < kRing) {
          umma4_ta<(2048 >> 4)>(d, a, v0, kIdO, acc);
          umma4_ta<(2048 >> 4)>(d, a + 32, v0 + 4 * (2048 >> 4), kIdO, 1u);
        } else {                           // the second block wrapped around: 64 columns at a time
          umma4_ta<(2048 >> 4)>(d, a, v0, kIdO64, acc);
          umma4_ta<(2048 >> 4)>(d, a + 32, v0 + 4 * (2048 >> 4), kIdO64, 1u);
          umma4_ta<(2048 >> 4)>(d + 64, a, d_v, kIdO64, acc);
          umma4_ta<(2048 >> 4)>(d + 64, a + 32, d_v + 4 * (2048 >> 4), kIdO64, 1u);
        }
        umma_commit(bars + 8 * (aO + i));
      };
      auto release = [&](uint32_t first, int count) {
        for (int c = 0; c < count; ++c) umma_commit(bars + 8 * (aEmpty + (first + c) % kRing));
      };
      while (ok && wk.next(p.H)) {
        const int end0 = min(wk.t1, wk.tiles0), tiles = wk.t1 - wk.t0;
        const bool zero = wk.t0 < end0;    // the first query tile takes part
        if (zero) {
          if (!bar_wait(bars + 8 * aQ, nq[0] & 1, p.wait_ns, abort)) { ok = false; break; }
          ++nq[0];
        }
        if (wk.two) {
          if (!bar_wait(bars + 8 * (aQ + 1), nq[1] & 1, p.wait_ns, abort)) { ok = false; break; }
          ++nq[1];
        }
        *begun = ++segs;
        if ((zero && !scores(0, n)) || (wk.two && !scores(1, n))) { ok = false; break; }
        release(n, 3);
        for (int j = 0; j < tiles; ++j, n += 5) {
          const int t = wk.t0 + j;
          const bool more = j + 1 < tiles;
          if (!wait_slots(n + 3, 2)) { ok = false; break; }
          if (t < end0) {
            if (!bar_wait(bars + 8 * aP, np[0] & 1, p.wait_ns, abort)) { ok = false; break; }
            ++np[0];
            outputs(0, n + 3, j > 0);
          }
          if (more && t + 1 < end0 && !scores(0, n + 5)) { ok = false; break; }
          if (wk.two) {
            if (!bar_wait(bars + 8 * (aP + 1), np[1] & 1, p.wait_ns, abort)) { ok = false; break; }
            ++np[1];
            outputs(1, n + 3, j > 0);
          }
          release(n + 3, 2);
          if (more) {
            if (wk.two && !scores(1, n + 5)) { ok = false; break; }
            release(n + 5, 3);
          }
        }
      }
      if (!ok) {
        set_err(p.dev_err, MLA_DEVERR_TIMEOUT);
        *abort = 1;
      }
      *begun = 0xFFFFFFFFu;
      umma_commit(bars + 8 * aFin);
      drain_wait(bars + 8 * aFin, 0);
    }
    __syncwarp();
  }
  fence_before();
  __syncthreads();
  if (warp == 9) {
    fence_after();
    tmem_free(tbase, 512);
  }
}

// long_combine_kernel: block 128, grid (splits, 16): a warp merges four rows of
// a split item, their parts in block order with the running maximum's weights
// (few parts per item, so one pass with all four rows' loads in flight).  Bound by
// reading the partials, 132 KB each, from L2: 12 us for 151 split items.
__global__ void __launch_bounds__(128) long_combine_kernel(const ChunkParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, r0 = 16 * blockIdx.y + 4 * (threadIdx.x >> 5);
  if ((int)blockIdx.x >= __ldcg(&p.counts->l_splits)) return;
  const SplitRec* sr = p.l_splits + blockIdx.x;
  const int4 rec = __ldcg(reinterpret_cast<const int4*>(sr));
  const int64_t row0 = __ldcg(&sr->row0);
  if (r0 >= rec.z) return;
  // part 0 is slot 2 first + 1, part i > 0 slot 2 (first + i)
  const float* part = p.l_parts + (int64_t)(2 * rec.x + 1) * long_partial_floats();
  float m[4], l[4] = {0.f, 0.f, 0.f, 0.f};
  float4 acc[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    m[e] = -INFINITY;
    acc[e] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  for (int y = rec.x; y <= rec.y; ++y) {
    float mi[4], li[4];
    float4 v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {          // rows of the padding are read (they lie in the slot) and not written
      mi[e] = __ldcg(part + kLongRows * kDv + r0 + e);
      li[e] = __ldcg(part + kLongRows * kDv + kLongRows + r0 + e);
      v[e] = __ldcg(reinterpret_cast<const float4*>(part + (r0 + e) * kDv) + lane);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float top = fmaxf(m[e], mi[e]), base = top == -INFINITY ? 0.f : top;
      const float a = ex2(m[e] - base), b = ex2(mi[e] - base);
      m[e] = top;
      l[e] = l[e] * a + li[e] * b;
      acc[e].x = acc[e].x * a + v[e].x * b;
      acc[e].y = acc[e].y * a + v[e].y * b;
      acc[e].z = acc[e].z * a + v[e].z * b;
      acc[e].w = acc[e].w * a + v[e].w * b;
    }
    part += (y == rec.x ? 1 : 2) * long_partial_floats();
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (r0 + e >= rec.z) break;
    const float inv = l[e] == 0.f ? 0.f : 1.f / l[e];
    uint32_t a, b;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;\n" : "=r"(a) : "f"(acc[e].y * inv), "f"(acc[e].x * inv));
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;\n" : "=r"(b) : "f"(acc[e].w * inv), "f"(acc[e].z * inv));
    reinterpret_cast<uint2*>(p.o + (row0 + (int64_t)(r0 + e) * p.H) * kDv)[lane] = make_uint2(a, b);
  }
}

template <int LF, int KF>
mla_status launch_prep(const ChunkParams& p, cudaStream_t stream) {
  const int smem = kQBlocks * kPrepRows + block_bytes<LF, KF>();
  static int configured[64] = {0};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !configured[dev]) {
    const mla_status st =
        cuda_status(cudaFuncSetAttribute(long_prep_kernel<LF, KF>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
    if (st != MLA_OK) return st;
    if (dev >= 0 && dev < 64) configured[dev] = 1;
  }
  const int key_blocks = 4 * (int)(p.kv_tokens / kLongKeys);
  return cuda_status(launch_pdl(long_prep_kernel<LF, KF>, dim3(key_blocks + 8 * p.H), dim3(kPrepThreads), smem, stream, p, key_blocks));
}

}  // namespace

mla_status launch_long(const ChunkParams& p, int lf, int kf, cudaStream_t stream) {
  static int configured[64] = {0};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !configured[dev]) {
    mla_status st = cuda_status(cudaFuncSetAttribute(long_expand_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kExSmem));
    if (st == MLA_OK) st = cuda_status(cudaFuncSetAttribute(long_attention_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kLaSmem));
    if (st != MLA_OK) return st;
    if (dev >= 0 && dev < 64) configured[dev] = 1;
  }
  mla_status st = MLA_ERR_UNSUPPORTED;
#define MLA_CHUNK_CASE(A, K) \
  if (lf == A && kf == K) st = launch_prep<A, K>(p, stream);
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
  if (st != MLA_OK) return st;
  st = cuda_status(launch_pdl(long_expand_kernel, dim3(p.grid), dim3(kExThreads), kExSmem, stream, p));
  if (st != MLA_OK) return st;
  st = cuda_status(launch_pdl(long_attention_kernel, dim3(p.grid), dim3(kLaThreads), kLaSmem, stream, p));
  if (st != MLA_OK) return st;
  return cuda_status(launch_pdl(long_combine_kernel, dim3(p.grid, kLongRows / 16), dim3(128), 0, stream, p));
}

}  // namespace mla
