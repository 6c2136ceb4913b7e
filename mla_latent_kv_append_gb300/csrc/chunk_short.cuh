// Chunk attention of sequences with few new tokens (short path): absorbed
// queries against the cached latents, so that every cached byte is read and
// dequantized once for all heads and new tokens of a row tile.
//
//   S^T = C Q^T          [64 keys] x [R rows], contraction over 576 channels
//   P^T = exp2(S^T - m)  (the softmax scale and log2 e are folded into Q; m is
//                        the running maximum less kHead)
//   O^T = C^T P^T        [512 channels] x [R rows], contraction over 64 keys
//
// with C the key tile (one 64-token page, dequantized to fp16) and Q a tile
// of R = 16, 32 or 64 query rows (any mix of new tokens and heads of one
// sequence).  Keys and channels, not rows, are the MMAs' M side: a decode has
// 16 rows per sequence, which as M would waste most of the tensor core, and
// the 512-channel output of 128 rows would fill TMEM alone.  As N, 64 rows
// need 4 x 64 TMEM columns for O^T and 2 x 64 for a double-buffered S^T.  C
// is both operands, as it lies: K-major for S^T, MN-major for O^T.
//
// What bounds it: reading the cache (740 bytes per token for INT8), and for
// 64-row tiles the shared-memory traffic of the MMAs' operands.  Cached bytes
// come as bulk copies of whole 32-token blocks into a ring of shared-memory
// slots (loads through L1 could not keep enough lines in flight next to 200
// KB of shared memory: 4.7 bytes per cycle and SM); sixteen warps dequantize
// them, lane = token, into fp16.  The key tile is handed on in four pieces of
// 128 channels, from a ring of 4 to 8 pieces, and the RoPE block: the S^T MMAs
// of a piece start when it is written, and the O^T MMAs release it.  The
// shared memory beside the queries is shared out by format: three raw blocks
// where they fit (the memory's latency wants 40 KB and more under way), the
// rest pieces, so that the next tile is converted while this one is used.
//
// Measured (whole call, absorption and projection included): 32 sequences x
// 32768 tokens, 16 heads, one new token each, INT4: 200 us, 3.0 TB/s of cache
// (45% of a plain copy's rate).  24 ragged drafts at 64 heads, bf16 cache: 160
// us.  One sequence of 4096 tokens, 16 heads, INT8: 19 us of a captured graph, of
// which this kernel 9, all latency (called from Python 25 to 30, the host's part).  With R = 16 a key tile takes 3100 to 3400 cycles per SM,
// 2400 of them shared-memory traffic that the split cannot avoid: 72 KB written
// by the dequantization, 72 + 18 KB read by the S^T MMAs, 64 + 8 KB by the O^T
// MMAs, the raw bytes in and out.  With R = 64 and a bf16 cache (5000 cycles) the
// queries and the raw blocks leave room for one key tile, so its steps and the
// next tile's follow one another; 1950 of the cycles are MMAs.
//
// Warps: 16 dequantize, 4 or 8 softmax (one group per 32 rows), then one each
// issues the S^T MMAs, the O^T MMAs (apart, so that neither waits for the
// other's operands) and the copies.
//
// Work split: all (row tile, key tile) units of the call, in order, are cut
// into equal runs, one per SM, so ragged lengths need no care.  A row tile
// that falls into several runs leaves fp32 partials, merged by
// short_combine_kernel in block order (no atomics: results repeat bit for
// bit).
//
// Rounding: keys, queries and P enter the MMAs as fp16 (2^-11 relative);
// scores, sums, maxima and O stay fp32 until o_lat is written as fp16.
#pragma once

#include <math.h>

#include "chunk.cuh"
#include "dequant.cuh"
#include "tc.cuh"

namespace mla {
namespace {

using namespace tc;

// Warps: 16 convert, 4 per softmax group (32 rows each), 4 issue.  Registers:
// the block launches with kLaunch a thread, then the roles take their shares.
template <int R>
struct Roles {
  static constexpr int kGroups = R == 64 ? 2 : 1, kGroupRows = R / kGroups;
  static constexpr int kSoftmax = 16, kIssue = 16 + 4 * kGroups, kWarps = kIssue + 4, kThreads = 32 * kWarps;
  static constexpr int kLaunch = R == 64 ? 72 : 80;
  static constexpr int kRegsConvert = R == 64 ? 64 : 72, kRegsSoftmax = R == 64 ? 96 : 104, kRegsIssue = R == 64 ? 56 : 88;
  static_assert(512 * kRegsConvert + 128 * kGroups * kRegsSoftmax + 128 * kRegsIssue <= kThreads * kLaunch &&
                    kThreads * kLaunch <= 65536 && kThreads * (kLaunch + 8) > 65536,
                "the warpgroups' shares come out of the launch's registers");
};
constexpr int kKeyBlk = kKeyTile * 128;              // one 64-key x 64-channel fp16 block: 8 KB
constexpr int kMaxSmem = 232448 - 1024;              // a block's shared memory, less the alignment slack
constexpr int kMaxSlots = 3;

constexpr int kPiece = 2 * kKeyBlk;                  // 128 channels of a key tile: 16 KB
constexpr int kMaxPieces = 8;

template <int LF, int KF, int R>
struct Shape {
  static constexpr int kBlock = block_bytes<LF, KF>();
  static constexpr int kRoom = kMaxSmem - (kQBlocks * R * 128 + R * 128 + 4 * R * 4 + 512);      // beside Q, P, reduction, barriers
  static constexpr int kRopes = kRoom - 4 * kPiece - 2 * kKeyBlk >= 2 * kBlock ? 2 : 1;
  static constexpr int kKeys = kRoom - kRopes * kKeyBlk;                                        // for pieces and raw blocks
  static constexpr int kSlots = kKeys - 4 * kPiece >= 3 * kBlock ? 3 : 2;
  static constexpr int kFit = (kKeys - kSlots * kBlock) / kPiece;
  static constexpr int kPieces = kFit < kMaxPieces ? kFit : kMaxPieces;
  static_assert(kPieces >= 4, "a whole key tile");
  static constexpr int kRope = kPieces * kPiece;
  static constexpr int kQ = kRope + kRopes * kKeyBlk;
  static constexpr int kP = kQ + kQBlocks * R * 128;
  static constexpr int kRed = kP + R * 128;          // [4 warps][R] maxima, then sums
  static constexpr int kRaw = kRed + 4 * R * 4;      // 256-byte aligned for R >= 16
  static constexpr int kBars = kRaw + kSlots * kBlock;
  static constexpr int kBytes = kBars + 512 + 1024;  // barriers and words; alignment slack
};

// Barriers: per piece of the ring, and per RoPE block, "written" and "free";
// S^T and P per score buffer; O^T of a tile done; raw slots.
enum { bWritten = 0, bFree = bWritten + kMaxPieces, bRopeW = bFree + kMaxPieces, bRopeF = bRopeW + 2, bS = bRopeF + 2,
       bP = bS + 2, bO = bP + 2, bRaw, bRawFree = bRaw + kMaxSlots, bQ = bRawFree + kMaxSlots, bFinS, bFinO, bTiles, bCount };
static_assert(8 * bCount + 76 + 4 * kMaxSlots <= 512, "barriers and words");

// One run's walk over the units: segments (a row tile, key tiles t0 .. t1).
struct Walk {
  const ShortSeq* seqs;
  int n_seqs, k;
  int64_t u, hi;
  ShortSeq s;
  int item, t0, t1, skip;   // skip: key tiles of the first segment's row tile before the run
  bool first, last;         // the segment holds the row tile's first / last key tile

  __device__ __forceinline__ void load() {
    const int4* r = reinterpret_cast<const int4*>(seqs + k);
    int4* d = reinterpret_cast<int4*>(&s);
    d[0] = __ldcg(r);
    d[1] = __ldcg(r + 1);
    d[2] = __ldcg(r + 2);
  }
  // The first sequence's record comes along with their number (it lies in the
  // workspace whether or not there is one).
  __device__ __forceinline__ void open(const ChunkParams& p) {
    seqs = p.s_seqs;
    k = 0;
    load();
    n_seqs = __ldcg(&p.counts->s_seqs);
  }
  // All lanes of a warp: the sequence of unit u, 32 probes per round.
  __device__ __forceinline__ void find(int64_t u) {
    const int lane = threadIdx.x & 31;
    int a = 0, n = n_seqs;                   // the answer is in [a, a + n)
    while (n > 1) {
      const int step = (n + 31) / 32;
      const int at = a + lane * step;
      const bool le = at < a + n && __ldcg(&seqs[at].unit0) <= u;
      const int c = __popc(__ballot_sync(0xffffffffu, le));      // at least 1: lane 0's is <= u
      const int na = a + (c - 1) * step;
      n = min(step, a + n - na);
      a = na;
    }
    if (a != k) {
      k = a;
      load();
    }
  }
  // All lanes of a warp: key tiles before unit v.
  __device__ __forceinline__ int64_t tiles_before(int64_t v) {
    find(v);
    const int cost = s.tiles + kItemCost;
    const int64_t d = v - s.unit0, at = d / cost;
    return s.unit0 - (int64_t)kItemCost * s.item0 + at * s.tiles + max((int)(d - at * cost) - kItemCost, 0);
  }
  __device__ __forceinline__ void start(int64_t lo, int64_t hi_) {
    u = lo;
    hi = hi_;
    find(u);
    const int64_t d = u - s.unit0;
    const int cost = s.tiles + kItemCost, r = (int)(d % cost);
    item = (int)(d / cost) - 1;
    skip = max(r - kItemCost, 0);
    u += max(kItemCost - r, 0);
  }
  // The next segment; false behind the run's end.  u: the unit of the next key tile.
  __device__ __forceinline__ bool next() {
    if (u >= hi) return false;
    if (++item == s.items) {
      item = 0;
      ++k;
      load();
    }
    t0 = skip;
    skip = 0;
    t1 = (int)min((int64_t)s.tiles, t0 + (hi - u));
    first = t0 == 0;
    last = t1 == s.tiles;
    u += t1 - t0 + kItemCost;
    return true;
  }
};

// A unit's 32 fp16 channels into a 64-channel block (half: its first or second
// 32 channels), swizzled.
__device__ __forceinline__ void put_unit(const uint32_t* h, uint32_t blk, int tok, int half) {
  const uint32_t row = blk + tok * 128, flip = (4 * half ^ (tok & 7)) << 4;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};\n" ::"r"(row + (flip ^ (i << 4))), "r"(h[4 * i]),
                 "r"(h[4 * i + 1]), "r"(h[4 * i + 2]), "r"(h[4 * i + 3])
                 : "memory");
}

template <int LF, int KF, int R>
__global__ void __launch_bounds__(Roles<R>::kThreads, 1) short_attention_kernel(const ChunkParams p) {
  using SH = Shape<LF, KF, R>;
  using RO = Roles<R>;
  constexpr int NP = SH::kPieces, NR = SH::kRopes, NS = SH::kSlots;
  extern __shared__ uint8_t short_smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(short_smem_raw) + 1023) & ~(uintptr_t)1023);
  const uint32_t sb = smem_u32(sm), bars = sb + SH::kBars;
  uint8_t* words = sm + SH::kBars + 8 * bCount;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(words);
  volatile int* abort = reinterpret_cast<volatile int*>(words + 4);
  volatile int* quit = reinterpret_cast<volatile int*>(words + 8);           // [groups][2, by tile parity]
  volatile int* tile_ok = reinterpret_cast<volatile int*>(words + 24);       // [4, by tile]
  uint32_t* bad = reinterpret_cast<uint32_t*>(words + 40);                   // [4, by tile][2]: a bit per token
  volatile uint32_t* run_tiles = reinterpret_cast<volatile uint32_t*>(words + 72 + 4 * kMaxSlots);
  volatile int* slot_len = reinterpret_cast<volatile int*>(words + 72);      // [slots] tokens of the block, -1: no page
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kCols = R == 64 ? 512 : 8 * R;       // 6 R columns used, a power of two allocated

  if (threadIdx.x == 0) {
    for (int i = 0; i < kMaxPieces; ++i) {
      bar_init(bars + 8 * (bWritten + i), 128);        // four warps write a piece
      bar_init(bars + 8 * (bFree + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(bars + 8 * (bRopeW + i), 128);          // and four the RoPE block
      bar_init(bars + 8 * (bRopeF + i), 1);
      bar_init(bars + 8 * (bS + i), 1);
      bar_init(bars + 8 * (bP + i), 128 * RO::kGroups);
    }
    bar_init(bars + 8 * bO, 1);
    for (int i = 0; i < kMaxSlots; ++i) {
      bar_init(bars + 8 * (bRaw + i), 1);
      bar_init(bars + 8 * (bRawFree + i), 512);
    }
    bar_init(bars + 8 * bQ, 1);
    bar_init(bars + 8 * bFinS, 1);
    bar_init(bars + 8 * bFinO, 1);
    bar_init(bars + 8 * bTiles, 1);
    *abort = 0;
    for (int i = 0; i < 4; ++i) quit[i] = 0;
    for (int i = 0; i < 8; ++i) bad[i] = 0;
    bar_init_fence();
  }
  if (warp == RO::kIssue) tmem_alloc(smem_u32(tmem_slot), kCols);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tbase = *tmem_slot;
  const uint32_t t_s = tbase + 4 * R;                // S^T: two buffers of R columns
  pdl_launch_dependents();
  pdl_wait();

  const int64_t U = __ldcg(&p.counts->s_units);
  const int G = (int)(U < gridDim.x ? U : gridDim.x);
  const int x = blockIdx.x;
  const bool work = x < G;
  const int64_t lo = work ? run_begin(U, x, G) : 0, hi = work ? run_begin(U, x + 1, G) : 0;
  bool ok = true;
  if (warp < 16) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(RO::kRegsConvert));
    // ---- dequantize.  Warp w takes unit w (32 channels, half a block of piece
    // w / 4) of both 32-token blocks of a tile; every fourth tile also the RoPE
    // block's unit w % 2 of block w / 2 % 2 (the four warps of a piece in turn:
    // always the same ones were a third slower than the rest); lane = token.
    const int s = warp >> 2, rope_half = (warp >> 1) & 1;
    uint32_t piece = s, round = 0;                     // the ring's piece for this tile, and how often it went round
    uint32_t n_tiles = 0;                              // of the run: the last warp counts them
    if (work) {
      if (warp_wait(bars + 8 * bTiles, 0, p.wait_ns, abort)) n_tiles = *run_tiles;
      else ok = false;
    }
    for (uint32_t it = 0; it < n_tiles; ++it) {
      const uint32_t f = it & 3;                       // the tile's flags
      const bool rope = (int)(it & 3) == s;
      uint32_t h[2][16];
      RawUnit<KF, true> rk;
      uint32_t bad_bits = 0;                           // of this lane's two tokens: bits 0 and 1
      int n_tok = 0;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const uint32_t blk = 2 * it + half, slot = blk % NS;
        if (ok && !warp_wait(bars + 8 * (bRaw + slot), (blk / NS) & 1, p.wait_ns, abort)) ok = false;
        if (!ok) break;
        const uint8_t* raw = sm + SH::kRaw + slot * SH::kBlock;
        n_tok = slot_len[slot];
        const bool live = lane < n_tok;
        RawUnit<LF, false> r;
        if (live) load_unit<LF, false>(raw, p.L, lane, warp, r);
        else zero_unit(r);
        if (rope && half == rope_half) {
          if (live) load_unit<KF, true>(raw, p.L, lane, warp & 1, rk);
          else zero_unit(rk);
        }
        if (LF != MLA_FMT_INT8_OUTLIER) bar_arrive(bars + 8 * (bRawFree + slot));      // read: the next copy may come
        bool fine = convert_unit<LF, false>(r, h[half]);
        if constexpr (LF == MLA_FMT_INT8_OUTLIER) {    // the protected channels lie in the slot
          if (live) fine &= patch_outliers<LF>(raw, p.L, p.outl, lane, warp, h[half]);
          bar_arrive(bars + 8 * (bRawFree + slot));
        }
        if (!fine) bad_bits |= 1u << half;
      }
      if (!ok) break;
      // The piece's last holder has gone.  Releases come in the ring's order,
      // so the barrier is at most one phase behind: the parity cannot mislead.
      if (round > 0 && !warp_wait(bars + 8 * (bFree + piece), (round - 1) & 1, p.wait_ns, abort)) {
        ok = false;
        break;
      }
      const uint32_t blk_at = sb + piece * kPiece + ((warp >> 1) & 1) * kKeyBlk;
      put_unit(h[0], blk_at, lane, warp & 1);
      put_unit(h[1], blk_at, 32 + lane, warp & 1);
      if (bad_bits & 1) atomicOr(bad + 2 * f, 1u << lane);
      if (bad_bits & 2) atomicOr(bad + 2 * f + 1, 1u << lane);
      if (!rope) {
        fence_async_smem();
        bar_arrive(bars + 8 * (bWritten + piece));
      } else {
        const bool fine = convert_unit<KF, true>(rk, h[0]);
        fence_async_smem();
        bar_arrive(bars + 8 * (bWritten + piece));
        const uint32_t kb = it % NR;
        if (it >= NR && !warp_wait(bars + 8 * (bRopeF + kb), (it / NR - 1) & 1, p.wait_ns, abort)) {
          ok = false;
          break;
        }
        put_unit(h[0], sb + SH::kRope + kb * kKeyBlk, 32 * rope_half + lane, warp & 1);
        // with the last barrier before S^T: the tile's flags
        if (!fine) atomicOr(bad + 2 * f + rope_half, 1u << lane);
        if ((warp & 3) == 0 && lane == 0) tile_ok[f] = n_tok >= 0;
        fence_async_smem();
        bar_arrive(bars + 8 * (bRopeW + kb));
      }
      piece += 4;
      if (piece >= NP) {
        piece -= NP;
        ++round;
      }
    }
    if (!ok) {
      set_err(p.dev_err, MLA_DEVERR_TIMEOUT);
      *abort = 1;
    }
  } else if (warp < RO::kIssue) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(RO::kRegsSoftmax));
    // ---- softmax.  A group of four warps has kGroupRows rows of the tile.
    // Thread (w, lane) holds keys 16 w + lane / 4 and + 8, rows 8 j + 2 (lane %
    // 4) and the next (j < J) of the group.  The group votes once per tile, so
    // its warps leave together: one that gave up a wait says so before a vote.
    Walk wk;
    wk.open(p);
    if (work) wk.start(lo, hi);
    constexpr int GR = RO::kGroupRows, J = GR / 8;
    const int w = warp & 3, gq = (warp - RO::kSoftmax) >> 2, bar_id = 1 + gq;
    const uint32_t tl = (uint32_t)(32 * w) << 16;
    float* red = reinterpret_cast<float*>(sm + SH::kRed) + gq * 4 * GR;
    uint32_t it = 0;
    bool late = false;                     // this warp gave up a wait since the last vote
    while (work && ok && wk.next()) {
      const int row0 = wk.item * R + gq * GR, rows = min(GR, wk.s.n * p.H - row0);       // rows <= 0: padding alone
      const int ctx = wk.s.len - wk.s.n;
      const int pos_min = ctx + row0 / p.H;          // the earliest row's position
      float m[2 * J], l[2 * J];            // the running maxima less kHead, and the sums of the weights
#pragma unroll
      for (int i = 0; i < 2 * J; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
      }
      for (int t = wk.t0; t < wk.t1; ++t, ++it) {
        const uint32_t g = it & 1, f = it & 3;
        if (late || !warp_wait(bars + 8 * (bS + g), (it >> 1) & 1, p.wait_ns, abort)) quit[2 * gq + g] = 1;
        __syncwarp();
        fence_after();
        const bool page_ok = tile_ok[f] != 0;
        const uint32_t bad_lo = *(volatile uint32_t*)(bad + 2 * f), bad_hi = *(volatile uint32_t*)(bad + 2 * f + 1);
        const bool masked = !page_ok || t * kKeyTile + kKeyTile - 1 > pos_min || (bad_lo | bad_hi);
        float v[4 * J];
        // the tile's scores, masked: hidden keys -inf, non-finite ones NaN, the
        // padding's rows (whose queries hold anything) 0
        auto load_scores = [&]() {
          uint32_t r[4 * J];
          tmem_load_16x256b<J>(t_s + g * R + gq * GR + tl, r);
#pragma unroll
          for (int i = 0; i < 4 * J; ++i) v[i] = __uint_as_float(r[i]);
          if (masked) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int key = 16 * w + (lane >> 2) + 8 * e, kp = t * kKeyTile + key;
              const bool is_bad = ((key < 32 ? bad_lo : bad_hi) >> (key & 31)) & 1u;
#pragma unroll
              for (int i = 0; i < 2 * J; ++i) {
                const int c = 8 * (i >> 1) + 2 * (lane & 3) + (i & 1);
                const bool sees = page_ok && kp <= ctx + (row0 + c) / p.H;
                float& s = v[4 * (i >> 1) + 2 * e + (i & 1)];
                s = sees ? (is_bad ? NAN : s) : -INFINITY;
              }
            }
          }
          if (rows < GR) {
#pragma unroll
            for (int i = 0; i < 2 * J; ++i)
              if (8 * (i >> 1) + 2 * (lane & 3) + (i & 1) >= rows) v[4 * (i >> 1) + (i & 1)] = v[4 * (i >> 1) + 2 + (i & 1)] = 0.f;
          }
        };
        load_scores();
        // Scores relative to their rows' running maxima.  Does one pass the
        // slack?  The maxima themselves are needed only then (the first tile of
        // a segment, and seldom after it).
        float over = -INFINITY;            // NaN from a NaN score or a row that has seen nothing yet
#pragma unroll
        for (int i = 0; i < 2 * J; ++i) {
          float &a = v[4 * (i >> 1) + (i & 1)], &b = v[4 * (i >> 1) + 2 + (i & 1)];
          a -= m[i];
          b -= m[i];
          over = max_nan(over, max_nan(a, b));
        }
        uint32_t any;
        asm volatile(
            "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.or.pred q, %2, 128, p;\n"
            " selp.u32 %0, 1, 0, q;\n}\n"
            : "=r"(any)
            : "r"((uint32_t)!(over <= kSlack + kHead)), "r"(bar_id)
            : "memory");
        if (quit[2 * gq + g]) {
          ok = false;
          break;
        }
        float alpha[2 * J];
        if (any) {
          load_scores();
#pragma unroll
          for (int j = 0; j < J; ++j) {
            float a = fmaxf(v[4 * j], v[4 * j + 2]), b = fmaxf(v[4 * j + 1], v[4 * j + 3]);
#pragma unroll
            for (int o = 4; o <= 16; o <<= 1) {
              a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
              b = fmaxf(b, __shfl_xor_sync(0xffffffffu, b, o));
            }
            if (lane < 4) *reinterpret_cast<float2*>(red + w * GR + 8 * j + 2 * lane) = make_float2(a, b);
          }
          asm volatile("bar.sync %0, 128;\n" ::"r"(bar_id) : "memory");
#pragma unroll
          for (int j = 0; j < J; ++j) {
            float2 a = make_float2(-INFINITY, -INFINITY);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const float2 b = *reinterpret_cast<const float2*>(red + q * GR + 8 * j + 2 * (lane & 3));
              a.x = fmaxf(a.x, b.x);
              a.y = fmaxf(a.y, b.y);
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int i = 2 * j + e;
              const float top = e ? a.y : a.x;
              const bool raise = top > m[i] + (kSlack + kHead);      // from -inf: the first key seen
              alpha[i] = raise ? ex2(m[i] - (top - kHead)) : 1.f;
              if (raise) m[i] = top - kHead;
              // a row that has seen nothing yet keeps m = -inf: its weights are 0
              const float base = m[i] == -INFINITY ? 0.f : m[i];
              v[4 * j + e] -= base;
              v[4 * j + 2 + e] -= base;
            }
          }
        }
        // the O^T of the tile before is complete: P is free, O^T may be
        // rescaled, and every group has read that tile's flags
        if (it >= 1) {
          if (!warp_wait(bars + 8 * bO, (it - 1) & 1, p.wait_ns, abort)) {
            late = true;
            continue;
          }
          const uint32_t before = (it - 1) & 3;
          if (threadIdx.x == 32 * RO::kSoftmax) bad[2 * before] = bad[2 * before + 1] = 0;
        }
        if (any) {
#pragma unroll
          for (int i = 0; i < 2 * J; ++i) l[i] *= alpha[i];
          if (t > wk.t0) {
            fence_after();
#pragma unroll
            for (int c0 = 0; c0 < GR; c0 += 16) {
              float al[16];
#pragma unroll
              for (int c = 0; c < 16; ++c)
                al[c] = __shfl_sync(0xffffffffu, alpha[2 * ((c0 + c) >> 3) + (c & 1)], (c & 7) >> 1);
#pragma unroll 1
              for (int blk = 0; blk < 4; ++blk) {
                uint32_t r[16];
                tmem_load16(tbase + blk * R + gq * GR + c0 + tl, r);
#pragma unroll
                for (int c = 0; c < 16; ++c) r[c] = __float_as_uint(__uint_as_float(r[c]) * al[c]);
                tmem_store16(tbase + blk * R + gq * GR + c0 + tl, r);
              }
            }
          }
        }
        // P^T as rows of 64 keys: the fragment transposed
#pragma unroll
        for (int j = 0; j < J; j += 2) {
          uint32_t h[4];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int i = j + e;
            const float p0 = ex2(v[4 * i]), p1 = ex2(v[4 * i + 1]), p2 = ex2(v[4 * i + 2]), p3 = ex2(v[4 * i + 3]);
            l[2 * i] += p0 + p2;
            l[2 * i + 1] += p1 + p3;
            h[2 * e] = half2_bits(p0, p1);
            h[2 * e + 1] = half2_bits(p2, p3);
          }
          const int mat = lane >> 3, rr = gq * GR + 8 * (j + (mat >> 1)) + (lane & 7), oct = 2 * w + (mat & 1);
          stmatrix_x4_trans(sb + SH::kP + rr * 128 + ((oct ^ (rr & 7)) << 4), h[0], h[1], h[2], h[3]);
        }
        fence_async_smem();
        fence_before();
        bar_arrive(bars + 8 * (bP + g));
      }
      if (!ok) break;
      // ---- the segment's end: sums over all keys, then O^T
#pragma unroll
      for (int i = 0; i < 2 * J; ++i) {
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], 4);
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], 8);
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], 16);
      }
      asm volatile("bar.sync %0, 128;\n" ::"r"(bar_id) : "memory");         // the last maxima have been read
      if (lane < 4) {
#pragma unroll
        for (int j = 0; j < J; ++j)
          *reinterpret_cast<float2*>(red + w * GR + 8 * j + 2 * lane) = make_float2(l[2 * j], l[2 * j + 1]);
      }
      asm volatile("bar.sync %0, 128;\n" ::"r"(bar_id) : "memory");
#pragma unroll
      for (int j = 0; j < J; ++j) {
        float2 a = make_float2(0.f, 0.f);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float2 b = *reinterpret_cast<const float2*>(red + q * GR + 8 * j + 2 * (lane & 3));
          a.x += b.x;
          a.y += b.y;
        }
        l[2 * j] = a.x;
        l[2 * j + 1] = a.y;
      }
      asm volatile("bar.sync %0, 128;\n" ::"r"(bar_id) : "memory");         // the sums have been read: the next maxima may come
      if (late || !warp_wait(bars + 8 * bO, (it - 1) & 1, p.wait_ns, abort)) {
        late = true;                       // leaves at the next vote, or with the run
        continue;
      }
      fence_after();
      const bool whole = wk.first && wk.last;
      const int slot = 2 * x + (wk.first ? 1 : 0);
      float* part = p.parts + (int64_t)slot * partial_floats(R) + (int64_t)gq * GR * kDc;
      const int64_t out0 = (int64_t)wk.s.tok0 * p.H + row0;
#pragma unroll
      for (int c0 = 0; c0 < GR; c0 += 16) {
        float inv[16];
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          const float sum = __shfl_sync(0xffffffffu, l[2 * ((c0 + c) >> 3) + (c & 1)], (c & 7) >> 1);
          inv[c] = sum == 0.f ? 0.f : 1.f / sum;       // nothing seen: 0 (a NaN sum stays NaN)
        }
#pragma unroll 1
        for (int blk = 0; blk < 4; ++blk) {
          uint32_t r[16];
          tmem_load16(tbase + blk * R + gq * GR + c0 + tl, r);
          const int ch = 128 * blk + 32 * w + lane;
          if (whole) {
#pragma unroll
            for (int c = 0; c < 16; ++c)
              if (c0 + c < rows)
                reinterpret_cast<__half*>(p.o_lat)[(out0 + c0 + c) * kDc + ch] = __float2half_rn(__uint_as_float(r[c]) * inv[c]);
          } else {
#pragma unroll
            for (int c = 0; c < 16; ++c)
              if (c0 + c < rows) part[(c0 + c) * kDc + ch] = __uint_as_float(r[c]);
          }
        }
      }
      if (!whole && w == 0 && lane < 4) {
        float* ml = p.parts + (int64_t)slot * partial_floats(R) + R * kDc + gq * GR;
#pragma unroll
        for (int i = 0; i < 2 * J; ++i) {
          const int c = 8 * (i >> 1) + 2 * lane + (i & 1);
          ml[c] = m[i];
          ml[R + c] = l[i];
        }
      }
      if (wk.first && !wk.last && warp == RO::kSoftmax && lane == 0) {
        // the row tile goes on in the blocks behind: up to the one that holds its last unit
        const int64_t end = wk.s.unit0 + (int64_t)(wk.item + 1) * (wk.s.tiles + kItemCost);
        SplitRec rec;
        rec.first = x;
        rec.last = run_of(U, end - 1, G);
        rec.rows = min(R, wk.s.n * p.H - wk.item * R);
        rec.pad = 0;
        rec.row0 = out0;
        p.splits[atomicAdd(&p.counts->s_splits, 1)] = rec;
      }
      fence_before();                                  // O^T has been read: ordered before the next P's arrival
    }
    if (!ok || late) {
      set_err(p.dev_err, MLA_DEVERR_TIMEOUT);
      *abort = 1;
    }
  } else {
    if constexpr (RO::kRegsIssue > RO::kLaunch) {
      asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(RO::kRegsIssue));
    } else {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(RO::kRegsIssue));
    }
    if (work && warp == RO::kIssue) {
      // ---- one thread: the query tiles' copies and the S^T MMAs
      Walk wk;
      wk.open(p);
      wk.start(lo, hi);
      if (elect_one()) {
        constexpr uint32_t kId = f16_idesc(64, R, false, false);
        constexpr int kQBytes = kQBlocks * R * 128;
        const uint64_t d_q = sw128_desc(sb + SH::kQ, 16, 1024), d_k = sw128_desc(sb, 16, 1024),
                       d_r = sw128_desc(sb + SH::kRope, 16, 1024);
        uint32_t it = 0, seg = 0, piece = 0, round = 0;
        while (ok && wk.next()) {
          // the query tile: its readers, the S^T MMAs of the segment before, are done
          if (seg > 0 && !bar_wait(bars + 8 * (bS + ((it - 1) & 1)), ((it - 1) >> 1) & 1, p.wait_ns, abort)) {
            ok = false;
            break;
          }
          bar_expect(bars + 8 * bQ, kQBytes);
          bulk_copy(sb + SH::kQ, p.q_tiles + (int64_t)(wk.s.item0 + wk.item) * kQBytes, kQBytes, bars + 8 * bQ);
          ++seg;
          if (!bar_wait(bars + 8 * bQ, (seg - 1) & 1, p.wait_ns, abort)) {
            ok = false;
            break;
          }
          for (int t = wk.t0; t < wk.t1 && ok; ++t, ++it) {
            const uint32_t g = it & 1, kb = it % NR, d = t_s + g * R;
            // the softmax has read this S^T buffer's last tile
            if (it >= 2 && !bar_wait(bars + 8 * (bP + g), ((it - 2) >> 1) & 1, p.wait_ns, abort)) {
              ok = false;
              break;
            }
#pragma unroll
            for (int s = 0; s < 4; ++s) {
              if (!bar_wait(bars + 8 * (bWritten + piece), round & 1, p.wait_ns, abort)) {
                ok = false;
                break;
              }
              fence_after();
              const uint64_t a = d_k + (uint64_t)(piece * (kPiece >> 4));
              umma4<2, 2>(d, a, d_q + (2 * s * R * 128 >> 4), kId, s != 0);
              umma4<2, 2>(d, a + (kKeyBlk >> 4), d_q + ((2 * s + 1) * R * 128 >> 4), kId, 1u);
              if (++piece == NP) {
                piece = 0;
                ++round;
              }
            }
            if (ok && !bar_wait(bars + 8 * (bRopeW + kb), (it / NR) & 1, p.wait_ns, abort)) ok = false;
            if (!ok) break;
            fence_after();
            umma4<2, 2>(d, d_r + (uint64_t)(kb * (kKeyBlk >> 4)), d_q + (8 * R * 128 >> 4), kId, 1u);
            umma_commit(bars + 8 * (bRopeF + kb));           // read here only
            umma_commit(bars + 8 * (bS + g));
          }
        }
        if (!ok) {
          set_err(p.dev_err, MLA_DEVERR_TIMEOUT);
          *abort = 1;
        }
        if (seg > 0) drain_wait(bars + 8 * bQ, (seg - 1) & 1);     // no copy is in flight when the block ends
        umma_commit(bars + 8 * bFinS);
        drain_wait(bars + 8 * bFinS, 0);
      }
      __syncwarp();
    } else if (work && warp == RO::kIssue + 1) {
      // ---- one thread: the O^T MMAs
      Walk wk;
      wk.open(p);
      wk.start(lo, hi);
      if (elect_one()) {
        constexpr uint32_t kId = f16_idesc(128, R, true, false);
        const uint64_t d_p = sw128_desc(sb + SH::kP, 16, 1024), d_v = sw128_desc(sb, kKeyBlk, 1024);
        uint32_t it = 0, piece = 0;
        while (ok && wk.next()) {
          for (int t = wk.t0; t < wk.t1; ++t, ++it) {
            const uint32_t g = it & 1;
            if (!bar_wait(bars + 8 * (bP + g), (it >> 1) & 1, p.wait_ns, abort)) {
              ok = false;
              break;
            }
            fence_after();
#pragma unroll
            for (int s = 0; s < 4; ++s) {
              umma4<(2048 >> 4), 2>(tbase + s * R, d_v + (uint64_t)(piece * (kPiece >> 4)), d_p, kId, t > wk.t0);
              umma_commit(bars + 8 * (bFree + piece));
              if (++piece == NP) piece = 0;
            }
            umma_commit(bars + 8 * bO);
          }
        }
        if (!ok) {
          set_err(p.dev_err, MLA_DEVERR_TIMEOUT);
          *abort = 1;
        }
        umma_commit(bars + 8 * bFinO);
        drain_wait(bars + 8 * bFinO, 0);
      }
      __syncwarp();
    } else if (work && warp == RO::kIssue + 2) {
      // ---- the cache's blocks into the raw slots.  The lanes fetch 32
      // page ids of the segment at a time, lane 0 issues.
      Walk wk;
      wk.open(p);
      wk.start(lo, hi);
      uint32_t blk = 0;
      while (ok && wk.next()) {
        const int32_t* pages = p.block_table + (int64_t)wk.s.b * p.max_pages;
        for (int t0 = wk.t0; t0 < wk.t1 && ok; t0 += 32) {
          const int mine = t0 + lane < wk.t1 ? __ldcg(pages + t0 + lane) : 0;
          for (int t = t0; t < min(wk.t1, t0 + 32) && ok; ++t) {
            const int page = __shfl_sync(0xffffffffu, mine, t - t0);
            const bool page_ok = page >= 0 && page < p.num_pages;
            if (!page_ok && lane == 0) set_err(p.dev_err, MLA_DEVERR_PAGE);
#pragma unroll
            for (int half = 0; half < 2; ++half, ++blk) {
              const uint32_t slot = blk % NS;
              if (blk >= NS && !warp_wait(bars + 8 * (bRawFree + slot), ((blk / NS) - 1) & 1, p.wait_ns, abort)) {
                ok = false;
                break;
              }
              if (lane == 0) {
                const int n_tok = min(32, max(0, wk.s.len - t * kKeyTile - 32 * half));
                slot_len[slot] = page_ok ? n_tok : -1;
                if (page_ok && n_tok > 0) {
                  bar_expect(bars + 8 * (bRaw + slot), SH::kBlock);
                  bulk_copy(sb + SH::kRaw + slot * SH::kBlock, p.pool + (int64_t)page * p.L.page_bytes + half * p.L.block_bytes,
                            SH::kBlock, bars + 8 * (bRaw + slot));
                } else {
                  bar_arrive(bars + 8 * (bRaw + slot));
                }
              }
              __syncwarp();
            }
          }
        }
      }
      if (!ok) {
        if (lane == 0) set_err(p.dev_err, MLA_DEVERR_TIMEOUT);
        *abort = 1;
      }
      // the copies in flight land before the block ends
      for (uint32_t s = 0; s < NS; ++s)
        if (blk > s) drain_wait(bars + 8 * (bRaw + s), ((blk - 1 - s) / NS) & 1);
    } else if (work && warp == RO::kIssue + 3) {
      // ---- the run's key tiles, for the converting warps (counted in a
      // softmax warp they cost its loop registers: 201 -> 208 us for 32 x 32768)
      Walk wk;
      wk.open(p);
      const int64_t all = U - (int64_t)kItemCost * __ldcg(&p.counts->s_items);
      const int64_t n = (x + 1 == G ? all : wk.tiles_before(hi)) - wk.tiles_before(lo);
      if (lane == 0) {
        *run_tiles = (uint32_t)n;
        bar_arrive(bars + 8 * bTiles);
      }
    }
  }
  fence_before();
  __syncthreads();
  if (warp == RO::kIssue) {
    fence_after();
    tmem_free(tbase, kCols);
  }
}

// short_combine_kernel: the blocks stride over the rows of the split row
// tiles.  A row's parts lie in the slots of its blocks, 2 first + 1 and then 2
// (first + i), merged in that order.  Few parts: four groups of threads take a
// row each.  Many (a single long context has a part in every block): the parts'
// maxima and sums are read side by side, then every group adds up its share of
// the parts, so that the loads overlap, and the groups are added in order.
// With many rows a block takes whole rows (COLS = 1); where the call has few row
// tiles for the SMs, so that rows are few and their parts many, four blocks
// share a row by columns and have four times the groups (COLS = 4).  One
// sequence of 4096 tokens: 23.5 us a captured call with COLS = 1, 20.8 with 4; 24 drafts
// 175 and 293; 32 sequences of 32768 tokens 201 and 211.  Bound by latency in the
// first case, by reading the partials from L2 in the others.
constexpr int kCombineThreads = 512;
constexpr int kCombineParts = 1024;      // most parts per row: blocks of the attention
// Up to 8 parts a row's merge is one batch of loads either way, and rows side by
// side leave fewer idle threads (24 drafts: 198 us a call without this, 176
// with it); a single context of 4096 tokens has 64 parts, which one thread after
// the other would add up in 64 steps (42 us a call).
constexpr int kCombineFew = 8;

template <int COLS>
__global__ void __launch_bounds__(kCombineThreads, 2) short_combine_kernel(const ChunkParams p, int R) {
  constexpr int kWidth = 128 / COLS, kGroups = kCombineThreads / kWidth;       // 16-byte columns of a block, groups of threads
  constexpr int kAhead = COLS == 1 ? 4 : 5;      // loads of a thread in flight: 32 and 80 parts a round
  __shared__ float s_w[kCombineParts];
  __shared__ float s_red[2][kCombineThreads / 32];
  __shared__ float4 s_acc[kGroups - 1][kWidth];
  pdl_launch_dependents();
  pdl_wait();
  const int tid = threadIdx.x, group = tid / kWidth, mine = tid % kWidth;
  // the first record comes along with the count (its place is in the list:
  // the blocks before it have 16 rows each at least)
  int4 rec = __ldcg(reinterpret_cast<const int4*>(p.splits + blockIdx.x / (R * COLS)));
  int64_t row0 = __ldcg(&p.splits[blockIdx.x / (R * COLS)].row0);
  const int total = __ldcg(&p.counts->s_splits) * R * COLS;
  for (int w = blockIdx.x; w < total; w += gridDim.x) {
    const int c = w / COLS % R, col = w % COLS * kWidth + mine;
    if (w != (int)blockIdx.x) {
      rec = __ldcg(reinterpret_cast<const int4*>(p.splits + w / (R * COLS)));
      row0 = __ldcg(&p.splits[w / (R * COLS)].row0);
    }
    if (c >= rec.z) continue;              // the same for the whole block
    const int64_t stride = 2 * partial_floats(R);
    const float* part = p.parts + (int64_t)(2 * rec.x + 1) * partial_floats(R);
    const int n = rec.y - rec.x + 1;
    // part i > 0 lies one slot before the regular stride
    auto at = [&](int i) { return part + i * stride - (i ? partial_floats(R) : 0); };
    if (COLS == 1 && n <= kCombineFew) {   // rows c .. c + 3, once
      const int cq = c + group;
      if ((c & 3) || cq >= rec.z) continue;
      float m = -INFINITY, l = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int i = 0; i < n; ++i) {
        const float* s = at(i);
        const float mi = __ldcg(s + R * kDc + cq), li = __ldcg(s + R * kDc + R + cq);
        const float4 v = __ldcg(reinterpret_cast<const float4*>(s + (int64_t)cq * kDc) + col);
        const float top = fmaxf(m, mi), base = top == -INFINITY ? 0.f : top;
        const float a = tc::ex2(m - base), b = tc::ex2(mi - base);
        m = top;
        l = l * a + li * b;
        acc.x = acc.x * a + v.x * b;
        acc.y = acc.y * a + v.y * b;
        acc.z = acc.z * a + v.z * b;
        acc.w = acc.w * a + v.w * b;
      }
      const float inv = l == 0.f ? 0.f : 1.f / l;
      reinterpret_cast<uint2*>(p.o_lat + (row0 + cq) * kDc)[col] =
          make_uint2(tc::half2_bits(acc.x * inv, acc.y * inv), tc::half2_bits(acc.z * inv, acc.w * inv));
      continue;
    }
    // the first parts are under way while the weights are made
    float4 v[kAhead];
    auto fetch = [&](int i0) {
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        if (i0 + kGroups * k < n) v[k] = __ldcg(reinterpret_cast<const float4*>(at(i0 + kGroups * k) + (int64_t)c * kDc) + col);
    };
    fetch(group);
    float mi[kCombineParts / kCombineThreads], li[kCombineParts / kCombineThreads], mx = -INFINITY;
#pragma unroll
    for (int k = 0; k < kCombineParts / kCombineThreads; ++k) {
      const int i = tid + k * kCombineThreads;
      mi[k] = i < n ? __ldcg(at(i) + R * kDc + c) : -INFINITY;
      li[k] = i < n ? __ldcg(at(i) + R * kDc + R + c) : 0.f;
      mx = fmaxf(mx, mi[k]);
    }
    for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    if ((tid & 31) == 0) s_red[0][tid >> 5] = mx;
    __syncthreads();
    mx = s_red[0][0];
#pragma unroll
    for (int k = 1; k < kCombineThreads / 32; ++k) mx = fmaxf(mx, s_red[0][k]);
    if (mx == -INFINITY) mx = 0.f;
    float l = 0.f;
#pragma unroll
    for (int k = 0; k < kCombineParts / kCombineThreads; ++k) {
      const float wt = tc::ex2(mi[k] - mx);
      l = fmaf(wt, li[k], l);
      s_w[tid + k * kCombineThreads] = wt;
    }
    for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    if ((tid & 31) == 0) s_red[1][tid >> 5] = l;
    __syncthreads();
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = group; i0 < n; i0 += kGroups * kAhead) {
      if (i0 != group) fetch(i0);
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        if (i0 + kGroups * k >= n) break;
        const float wt = s_w[i0 + kGroups * k];
        acc.x = fmaf(wt, v[k].x, acc.x);
        acc.y = fmaf(wt, v[k].y, acc.y);
        acc.z = fmaf(wt, v[k].z, acc.z);
        acc.w = fmaf(wt, v[k].w, acc.w);
      }
    }
    if (group) s_acc[group - 1][mine] = acc;
    __syncthreads();
    if (!group) {
      l = 0.f;
#pragma unroll
      for (int k = 0; k < kCombineThreads / 32; ++k) l += s_red[1][k];
      const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
      for (int k = 0; k < kGroups - 1; ++k) {
        const float4 a = s_acc[k][mine];
        acc.x += a.x;
        acc.y += a.y;
        acc.z += a.z;
        acc.w += a.w;
      }
      reinterpret_cast<uint2*>(p.o_lat + (row0 + c) * kDc)[col] =
          make_uint2(tc::half2_bits(acc.x * inv, acc.y * inv), tc::half2_bits(acc.z * inv, acc.w * inv));
    }
    __syncthreads();                       // s_acc and s_red have been read
  }
}

template <int LF, int KF, int R>
mla_status launch_r(const ChunkParams& p, cudaStream_t stream) {
  static int configured[64] = {0};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !configured[dev]) {
    const mla_status st = cuda_status(cudaFuncSetAttribute(
        short_attention_kernel<LF, KF, R>, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape<LF, KF, R>::kBytes));
    if (st != MLA_OK) return st;
    if (dev >= 0 && dev < 64) configured[dev] = 1;
  }
  const mla_status st = cuda_status(launch_pdl(short_attention_kernel<LF, KF, R>, dim3(p.grid), dim3(Roles<R>::kThreads),
                                               Shape<LF, KF, R>::kBytes, stream, p));
  if (st != MLA_OK) return st;
  const dim3 grid(4 * p.grid + 1), block(kCombineThreads);
  if (p.row_tiles * kCombineFew <= p.grid) return cuda_status(launch_pdl(short_combine_kernel<4>, grid, block, 0, stream, p, R));
  return cuda_status(launch_pdl(short_combine_kernel<1>, grid, block, 0, stream, p, R));
}

template <int LF, int KF>
mla_status launch_fmt(const ChunkParams& p, int R, cudaStream_t stream) {
  return R == 16 ? launch_r<LF, KF, 16>(p, stream) : (R == 32 ? launch_r<LF, KF, 32>(p, stream) : launch_r<LF, KF, 64>(p, stream));
}

}  // namespace

}  // namespace mla
