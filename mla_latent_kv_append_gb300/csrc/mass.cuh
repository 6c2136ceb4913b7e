// mla_token_mass: the attention weight that every cached token received.
//
//   mass[slot(t)] = decay mass[slot(t)] + sum_r exp2(S[t][r] - lse_r)
//   S = X Q^T        [128 keys] x [R rows], contraction over 576 channels
// with X a tile of 128 cached tokens and Q the rows r = i H + h of a sequence
// (query i, head h), the softmax scale and log2 e folded in.  Keys are the MMAs'
// M side: a thread of the epilogue then has a key's scores in its TMEM lane and
// adds up their exponentials by itself, no reduction across threads; and a
// decode has only 16 rows, which as M would waste most of the tensor core.
//
// Precision: the result is fp32, so a score needs more than the 11 bits of one
// fp16 operand.  Both operands are split into two halves, x = hi + lo and q = hi +
// lo (22 bits), and three of the four products are taken; a bf16 value fits hi
// alone.  Powers of two (kKeyGain, kQueryGain) keep the low halves out of
// fp16's subnormal range and are taken back in the exponent's FMA.
//
// X lies in TMEM as the MMAs' A: as shared-memory operands, two halves of 128
// keys do not fit (288 KB), and writing and reading them would cost 5700 cycles
// of shared-memory time a tile.
#pragma once

#include <math.h>

#include "dequant.cuh"
#include "mass_params.cuh"
#include "tc.cuh"

namespace mla {
namespace {

using namespace tc;

// Warps: 16 convert, 4 read the scores, then one each issues the MMAs, the
// cache's copies and the queries' copies; one is idle.
constexpr int kMassConvert = 16, kMassRead = 16, kMassMma = 20, kMassRaw = 21, kMassQ = 22, kMassWarps = 24;
constexpr int kMassThreads = 32 * kMassWarps;
constexpr int kMassSmem = 232448 - 1024;               // a block's shared memory, less the alignment slack
constexpr int kMassMaxRaw = 8;
constexpr int kMassAligned = 1024;

// Barriers.
enum { mA = 0, mAFree = mA + 8, mS = mAFree + 8, mE = mS + 2, mRaw = mE + 2, mRawFree = mRaw + kMassMaxRaw, mQ = mRawFree + kMassMaxRaw,
       mQFree = mQ + 9, mQDone = mQFree + 9, mFin, mCount };
constexpr int kMassMisc = 8 * mCount + 64 + kMassMaxRows * 4;      // barriers, words, the rows' lse
static_assert(8 * mCount + 64 <= 1024, "barriers and words");

template <int LF, int KF>
struct MassShape {
  static constexpr int kBlock = block_bytes<LF, KF>();
  static constexpr bool kSplit = LF != MLA_FMT_BF16;   // a latent piece has a low half
  static constexpr int kCols = kSplit ? 64 : 32;       // TMEM columns of a piece (64 channels)
  static constexpr int kSlots = 256 / 64;              // pieces in TMEM
  // shared memory: queries of R rows in `qs` pieces, then raw blocks
  static constexpr int query_pieces(int R) {
    const int room = kMassSmem - 2048, piece = R * 256;
    if (9 * piece + 5 * kBlock <= room) return 9;
    return (room - 5 * kBlock) / piece >= 2 ? (room - 5 * kBlock) / piece : 2;
  }
  static constexpr int raw_slots(int R) {
    const int n = (kMassSmem - 2048 - query_pieces(R) * R * 256) / kBlock;
    return n < kMassMaxRaw ? n : kMassMaxRaw;
  }
  static_assert(raw_slots(kMassMaxRows) >= 4 && raw_slots(64) >= 4 && raw_slots(32) >= 4 && raw_slots(16) >= 4, "a whole key tile");
};

// A block's walk over its passes (a row block of a key tile).
struct MassWalk {
  const MassSeq* seqs;
  int n_seqs, k, tile, rb, R, cost;                    // cost: of a full row block
  int64_t at, hi;
  MassSeq s;

  __device__ __forceinline__ void load() {
    const int4* r = reinterpret_cast<const int4*>(seqs + k);
    int4* d = reinterpret_cast<int4*>(&s);
#pragma unroll
    for (int i = 0; i < (int)sizeof(MassSeq) / 16; ++i) d[i] = __ldcg(r + i);
  }
  __device__ __forceinline__ void open(const MassParams& p) {
    seqs = p.seqs;
    n_seqs = __ldcg(&p.counts->seqs);
    R = p.R;
    cost = mass_cost(R);
    k = -1;
  }
  // All lanes of a warp: the sequence of unit u, 32 probes per round.
  __device__ __forceinline__ void find(int64_t u) {
    const int lane = threadIdx.x & 31;
    int a = 0, n = n_seqs;                             // the answer is in [a, a + n)
    while (n > 1) {
      const int step = (n + 31) / 32, at_ = a + lane * step;
      const bool le = at_ < a + n && __ldcg(&seqs[at_].unit0) <= u;
      const int c = __popc(__ballot_sync(0xffffffffu, le));        // at least 1: lane 0's is <= u
      const int na = a + (c - 1) * step;
      n = min(step, a + n - na);
      a = na;
    }
    if (a != k) {
      k = a;
      load();
    }
  }
  // All lanes of a warp: passes that start before unit v.
  __device__ __forceinline__ int64_t passes_before(int64_t v) {
    find(v);
    const int64_t d = v - s.unit0, t = d / s.tile_cost;
    const int off = (int)(d - t * s.tile_cost);
    return s.pass0 + t * s.blocks + min(s.blocks, (off + cost - 1) / cost);
  }
  __device__ __forceinline__ void start(int64_t lo, int64_t hi_) {
    hi = hi_;
    find(lo);
    const int64_t d = lo - s.unit0;
    tile = (int)(d / s.tile_cost);
    rb = ((int)(d - (int64_t)tile * s.tile_cost) + cost - 1) / cost;
    settle();
  }
  __device__ __forceinline__ void settle() {
    if (rb >= s.blocks) {
      rb = 0;
      if (++tile >= s.tiles) {
        tile = 0;
        if (++k < n_seqs) load();
        else {
          at = hi;
          return;
        }
      }
    }
    at = s.unit0 + (int64_t)tile * s.tile_cost + (int64_t)rb * cost;
  }
  __device__ __forceinline__ bool valid() const { return at < hi; }
  __device__ __forceinline__ void next() {
    ++rb;
    settle();
  }
  __device__ __forceinline__ int rows() const { return min(R, s.n * s.heads - rb * R); }
};

__device__ __forceinline__ __half2 as_half2(uint32_t w) { return *reinterpret_cast<const __half2*>(&w); }
__device__ __forceinline__ uint32_t as_word(__half2 h) { return *reinterpret_cast<const uint32_t*>(&h); }

// (a, b) as halves: hi + lo.
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(a, b);
  hi = as_word(h);
  lo = as_word(__floats2half2_rn(a - __low2float(h), b - __high2float(h)));
}

// The unit's 32 channels times kKeyGain: hi[i] + lo[i] = channels (2i, 2i + 1).
template <int FMT, bool KPE>
__device__ __forceinline__ void split_any(const RawUnit<FMT, KPE>& r, uint32_t* hi, uint32_t* lo) {
  using S = UnitShape<FMT, KPE>;
  if constexpr (S::kInt4) {
    const uint32_t w[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int k = 0; k < 4; ++k) {                    // nibbles k and k + 4 are adjacent channels
        const int ch = int4_nibble_channel(j, k), g = ch / S::kGroup;
        const float z = S::kZeros ? r.z[S::kZeros ? g : 0] : 8.f, s = r.s[g] * kKeyGain;
        split2(((float)((w[j] >> (4 * k)) & 15u) - z) * s, ((float)((w[j] >> (4 * k + 16)) & 15u) - z) * s, hi[ch / 2], lo[ch / 2]);
      }
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t w[4] = {r.w[i].x, r.w[i].y, r.w[i].z, r.w[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int k = 0; k < 4; k += 2) {
          const int ch = 16 * i + (!KPE && S::kGroup == 8 ? 2 * j + 4 * k : 4 * j + k);
          const float s = r.s[S::kScales > 1 ? ch / S::kGroup : 0] * kKeyGain;
          split2((float)(int8_t)(w[j] >> (8 * k)) * s, (float)(int8_t)(w[j] >> (8 * k + 8)) * s, hi[ch / 2], lo[ch / 2]);
        }
    }
  }
}

template <int FMT, bool KPE>
__device__ __forceinline__ void split_unit(const RawUnit<FMT, KPE>& r, uint32_t* hi, uint32_t* lo) {
  if constexpr (FMT == MLA_FMT_BF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w[4] = {r.w[i].x, r.w[i].y, r.w[i].z, r.w[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) hi[4 * i + j] = half2_bits(bf16lo(w[j]) * kKeyGain, bf16hi(w[j]) * kKeyGain);
    }
  } else {
    split_any<FMT, KPE>(r, hi, lo);
  }
}

// INT8_OUTLIER: puts the protected channels of unit c in their places.
template <int FMT>
__device__ __forceinline__ void patch_split(const uint8_t* blk, const PageLayout& L, const OutlierSet& outl, int u, int c,
                                            uint32_t* hi, uint32_t* lo) {
  if constexpr (FMT == MLA_FMT_INT8_OUTLIER) {
    if (!outl.mask[c]) return;
    const uint16_t* ov = reinterpret_cast<const uint16_t*>(blk + L.outlier_off);
    for (int k = 0; k < kNOut; ++k) {
      const int ch = outl.ch[k];
      if ((ch >> 5) != c) continue;
      const float v = bf16f(ov[k * kBlockTokens + u]) * kKeyGain;
      uint32_t h, l;
      split2(v, v, h, l);
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (i == ((ch & 31) >> 1)) {
          const uint32_t m = (ch & 1) ? 0xFFFF0000u : 0xFFFFu;
          hi[i] = (hi[i] & ~m) | (h & m);
          lo[i] = (lo[i] & ~m) | (l & m);
        }
    }
  }
}

__device__ __forceinline__ void tmem_put16(uint32_t t, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n" ::"r"(t),
      MLA_V8(v, 0), MLA_V8(v, 8)
      : "memory");
}
__device__ __forceinline__ void tmem_put_wait() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }

// Whether any thread of the four reading warps says so; also their barrier.
__device__ __forceinline__ bool vote_128(bool mine) {
  uint32_t any;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.or.pred q, 1, 128, p;\n selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(any)
      : "r"((uint32_t)mine)
      : "memory");
  return any != 0;
}

template <int LF, int KF>
__global__ void __launch_bounds__(kMassThreads, 1) mass_kernel(const MassParams p) {
  using SH = MassShape<LF, KF>;
  constexpr int NA = SH::kSlots, COLS = 64;
  extern __shared__ uint8_t mass_smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(mass_smem_raw) + kMassAligned - 1) & ~(uintptr_t)(kMassAligned - 1));
  const int R = p.R, QS = p.query_pieces, NS = p.raw_slots;
  const bool resident = QS == 9;
  const uint32_t sb = smem_u32(sm), s_raw = QS * R * 256, bars = sb + s_raw + NS * SH::kBlock;
  uint8_t* words = sm + s_raw + NS * SH::kBlock + 8 * mCount;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(words);
  volatile int* abort = reinterpret_cast<volatile int*>(words + 4);
  volatile int* s_last = reinterpret_cast<volatile int*>(words + 8);
  float* s_lse = reinterpret_cast<float*>(words + 64);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 8; ++i) {
      bar_init(bars + 8 * (mA + i), 128);              // four warps write a piece
      bar_init(bars + 8 * (mAFree + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(bars + 8 * (mS + i), 1);
      bar_init(bars + 8 * (mE + i), 128);
    }
    for (int i = 0; i < kMassMaxRaw; ++i) {
      bar_init(bars + 8 * (mRaw + i), 1);
      bar_init(bars + 8 * (mRawFree + i), 128);        // the four warps of the block's lanes
    }
    for (int i = 0; i < 9; ++i) {
      bar_init(bars + 8 * (mQ + i), 1);
      bar_init(bars + 8 * (mQFree + i), 1);
    }
    bar_init(bars + 8 * mQDone, 1);
    bar_init(bars + 8 * mFin, 1);
    *abort = 0;
    bar_init_fence();
  }
  if (warp == kMassMma) tmem_alloc(smem_u32(tmem_slot), 512);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tbase = *tmem_slot, t_a = tbase + 256;              // scores: two buffers of 128 columns; then the pieces
  pdl_launch_dependents();
  pdl_wait();

  const int64_t U = __ldcg(&p.counts->units);
  const int G = (int)(U < gridDim.x ? U : gridDim.x), x = blockIdx.x;
  const bool work = x < G;
  const int64_t lo = work ? mass_run(U, x, G) : 0, hi = work ? mass_run(U, x + 1, G) : 0;
  bool ok = true;
  if (work && warp < kMassConvert) {
    // ---- Warp (s, d): lanes 32 d .. 32 d + 31 (a 32-token block of the tile) of
    // the pieces s, s + 4, ... of the run; lane = token.
    const int s = warp >> 2, d = warp & 3;
    const uint32_t tl = (uint32_t)(32 * d) << 16;
    int64_t n_pass;
    {
      MassWalk wk;
      wk.open(p);
      n_pass = (x + 1 == G ? __ldcg(&p.counts->passes) : wk.passes_before(hi)) - wk.passes_before(lo);
    }
    uint32_t kb = s, blk = d, turn = 0;                // piece of the pass, raw block, how many pieces this warp has made
    for (int64_t it = 0; it < n_pass;) {
      const uint32_t slot = blk % NS;
      if (!warp_wait(bars + 8 * (mRaw + slot), (blk / NS) & 1, p.wait_ns, abort)) {
        ok = false;
        break;
      }
      const uint8_t* raw = sm + s_raw + slot * SH::kBlock;
      const uint32_t a = t_a + s * COLS + tl;
      bool split = true;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t h[16], l[16];
        if (kb < 8) {
          RawUnit<LF, false> r;
          load_unit<LF, false>(raw, p.L, lane, 2 * kb + half, r);
          split_unit<LF, false>(r, h, l);
          patch_split<LF>(raw, p.L, p.outl, lane, 2 * kb + half, h, l);
          split = LF != MLA_FMT_BF16;
        } else {
          RawUnit<KF, true> r;
          load_unit<KF, true>(raw, p.L, lane, half, r);
          split_unit<KF, true>(r, h, l);
          split = KF != MLA_FMT_BF16;
        }
        // the piece before, four earlier, has been multiplied
        if (half == 0 && turn > 0 && !warp_wait(bars + 8 * (mAFree + s), (turn - 1) & 1, p.wait_ns, abort)) {
          ok = false;
          break;
        }
        fence_after();
        tmem_put16(a + 16 * half, h);
        if (split) tmem_put16(a + 32 + 16 * half, l);
      }
      if (!ok) break;
      tmem_put_wait();
      fence_before();
      bar_arrive(bars + 8 * (mA + s));
      ++turn;
      kb += 4;
      if (kb >= 9) {                                   // this warp's last piece of the pass
        bar_arrive(bars + 8 * (mRawFree + slot));
        kb -= 9;
        blk += 4;
        ++it;
      }
    }
    if (!ok) {
      set_err(p.dev_err, MLA_DEVERR_TIMEOUT);
      *abort = 1;
    }
  } else if (work && warp >= kMassRead && warp < kMassMma) {
    // ---- the scores: thread = key
    MassWalk wk;
    wk.open(p);
    wk.start(lo, hi);
    const int key = threadIdx.x - 32 * kMassRead;
    const uint32_t tl = (uint32_t)(32 * (warp & 3)) << 16;
    uint32_t it = 0;
    int held_k = -1, held_rb = -1;
    bool odd = false, fresh = true, late = false;      // odd: a row without a finite lse
    float total = 0.f;
    int page = -1, parts = 0;
    for (; wk.valid(); ++it) {
      const uint32_t g = it & 1;
      const int rows = wk.rows(), row0 = wk.rb * R, t = wk.tile * kMassKeys + key, len = wk.s.len;
      if (fresh) {
        total = 0.f;
        parts = 0;
        page = t < len ? __ldcg(p.table + (int64_t)wk.s.b * p.max_pages + t / kPage) : -1;
        if (t < len && (page < 0 || page >= p.num_pages)) {
          set_err(p.dev_err, MLA_DEVERR_PAGE);
          page = -1;
        }
      }
      if (wk.k != held_k || wk.rb != held_rb) {
        held_k = wk.k;
        held_rb = wk.rb;
        const float v = key < rows ? __ldcg(p.lse + (int64_t)wk.s.q0 * p.H + row0 + key) * -1.4426950408889634f : 0.f;
        const bool fin = fabsf(v) < INFINITY;
        asm volatile("bar.sync 1, 128;\n" ::: "memory");             // the old ones have been read
        s_lse[key] = fin ? v : -INFINITY;
        odd = vote_128(!fin);
      }
      // the four warps meet at barriers: they leave together
      late = !warp_wait(bars + 8 * (mS + g), (it >> 1) & 1, p.wait_ns, abort);
      if (late) *abort = 1;
      if (vote_128(late)) {
        late = true;
        break;
      }
      fence_after();
      // rows from `first` on see the key
      const int pos = t - (len - wk.s.n), first = pos > 0 ? (pos >= wk.s.n ? rows : max(pos * p.H - row0, 0)) : 0;
      const bool plain = !odd && __all_sync(0xffffffffu, first == 0);
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
      for (int c0 = 0; c0 < rows; c0 += 16) {
        uint32_t r[16];
        tmem_load16(tbase + g * kMassMaxRows + c0 + tl, r);
        if (plain) {
#pragma unroll
          for (int c = 0; c < 16; ++c) sum[c & 3] += ex2(fmaf(__uint_as_float(r[c]), kMassUngain, s_lse[c0 + c]));
        } else {
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            const float y = s_lse[c0 + c];
            const float w = ex2(fmaf(__uint_as_float(r[c]), kMassUngain, y));
            sum[c & 3] += c0 + c >= first && y > -INFINITY ? w : 0.f;
          }
        }
      }
      fence_before();
      bar_arrive(bars + 8 * (mE + g));
      total += (sum[0] + sum[1]) + (sum[2] + sum[3]);
      ++parts;
      // the tile's last pass of this block?
      const MassSeq seq = wk.s;
      const int tile = wk.tile, k = wk.k;
      wk.next();
      fresh = !wk.valid() || wk.k != k || wk.tile != tile;
      if (!fresh) continue;
      if (parts == seq.blocks) {
        if (page >= 0) mass_store(p, page, t, seq.counted, total);
        continue;
      }
      // several blocks share the tile: its parts are added up, in the blocks'
      // order, by whichever is the last to finish
      const int64_t u0 = seq.unit0 + (int64_t)tile * seq.tile_cost;
      const int x0 = mass_run_of(U, u0, G), x1 = mass_run_of(U, u0 + (int64_t)(seq.blocks - 1) * wk.cost, G);
      __stcg(p.parts + (int64_t)(2 * x + (x == x0 ? 1 : 0)) * kMassKeys + key, total);
      __threadfence();
      asm volatile("bar.sync 1, 128;\n" ::: "memory");
      if (key == 0) *s_last = atomicAdd(p.done + x0, parts) + parts == seq.blocks;
      asm volatile("bar.sync 1, 128;\n" ::: "memory");
      const bool last = *s_last != 0;
      asm volatile("bar.sync 1, 128;\n" ::: "memory");
      if (last) {
        __threadfence();
        float sum_all = 0.f;
        for (int y = x0; y <= x1; ++y) {
          // a block whose run holds no pass of the tile has no part
          const int64_t from = mass_run(U, y, G) - u0, to = mass_run(U, y + 1, G) - u0;
          const int64_t r0 = from <= 0 ? 0 : (from + wk.cost - 1) / wk.cost;
          if (r0 < seq.blocks && r0 * wk.cost < to) sum_all += __ldcg(p.parts + (int64_t)(2 * y + (y == x0 ? 1 : 0)) * kMassKeys + key);
        }
        if (page >= 0) mass_store(p, page, t, seq.counted, sum_all);
      }
    }
    if (late) set_err(p.dev_err, MLA_DEVERR_TIMEOUT);
  } else if (work && warp == kMassMma) {
    // ---- one thread issues the MMAs
    MassWalk wk;
    wk.open(p);
    wk.start(lo, hi);
    if (elect_one()) {
      const uint64_t d_q = sw128_desc(sb, 16, 1024);
      uint32_t it = 0, piece = 0, q = 0;               // passes, pieces, query pieces
      int held_k = -1, held_rb = -1;
      for (; ok && wk.valid(); wk.next(), ++it) {
        const uint32_t g = it & 1, d = tbase + g * kMassMaxRows, id = f16_idesc(128, wk.rows(), false, false);
        const bool held = resident && wk.k == held_k && wk.rb == held_rb;
        held_k = wk.k;
        held_rb = wk.rb;
        // the scores of two passes before have been read
        if (it >= 2 && !bar_wait(bars + 8 * (mE + g), ((it - 2) >> 1) & 1, p.wait_ns, abort)) {
          ok = false;
          break;
        }
        if (held) q -= 9;
        else if (resident && it > 0) umma_commit(bars + 8 * mQDone);       // the old queries' last reader
        for (uint32_t kb = 0; kb < 9; ++kb, ++piece, ++q) {
          const uint32_t slot = piece % NA, qs = q % QS;
          if (!held && !bar_wait(bars + 8 * (mQ + qs), (q / QS) & 1, p.wait_ns, abort)) {
            ok = false;
            break;
          }
          if (!bar_wait(bars + 8 * (mA + slot), (piece / NA) & 1, p.wait_ns, abort)) {
            ok = false;
            break;
          }
          fence_after();
          const uint32_t a = t_a + slot * COLS;
          const uint64_t b_hi = d_q + (uint64_t)(qs * R * 256 >> 4), b_lo = b_hi + (uint64_t)(R * 128 >> 4);
          umma4_ta<2>(d, a, b_hi, id, kb != 0);
          umma4_ta<2>(d, a, b_lo, id, 1u);
          if (kb < 8 ? LF != MLA_FMT_BF16 : KF != MLA_FMT_BF16) umma4_ta<2>(d, a + 32, b_hi, id, 1u);
          umma_commit(bars + 8 * (mAFree + slot));
          if (!resident) umma_commit(bars + 8 * (mQFree + qs));
        }
        if (ok) umma_commit(bars + 8 * (mS + g));
      }
      if (!ok) {
        set_err(p.dev_err, MLA_DEVERR_TIMEOUT);
        *abort = 1;
      }
      umma_commit(bars + 8 * mFin);
      drain_wait(bars + 8 * mFin, 0);
    }
    __syncwarp();
  } else if (work && warp == kMassRaw) {
    // ---- the cache's blocks, a pass ahead with the page ids
    MassWalk wk;
    wk.open(p);
    wk.start(lo, hi);
    auto pages = [&]() {                               // lane i < 4: the page of block i of the walk's tile, -1: nothing to load
      const int t = wk.tile * kMassKeys + 32 * (lane & 3);
      return wk.valid() && lane < 4 && t < wk.s.len ? __ldcg(p.table + (int64_t)wk.s.b * p.max_pages + t / kPage) : -1;
    };
    uint32_t blk = 0;
    int ids = pages();
    while (ok && wk.valid()) {
      const int mine = ids >= 0 && ids < p.num_pages ? ids : -1;
      wk.next();
      ids = pages();
      for (int i = 0; i < 4; ++i, ++blk) {
        const uint32_t slot = blk % NS;
        if (blk >= (uint32_t)NS && !warp_wait(bars + 8 * (mRawFree + slot), ((blk / NS) - 1) & 1, p.wait_ns, abort)) {
          ok = false;
          break;
        }
        const int page = __shfl_sync(0xffffffffu, mine, i);
        if (lane == 0) {
          if (page >= 0) {
            bar_expect(bars + 8 * (mRaw + slot), SH::kBlock);
            bulk_copy(sb + s_raw + slot * SH::kBlock, p.pool + (int64_t)page * p.L.page_bytes + (i & 1) * p.L.block_bytes,
                      SH::kBlock, bars + 8 * (mRaw + slot));
          } else {
            bar_arrive(bars + 8 * (mRaw + slot));      // the lanes' keys are not read: whatever lies there will do
          }
        }
        __syncwarp();
      }
    }
    if (!ok) {
      if (lane == 0) set_err(p.dev_err, MLA_DEVERR_TIMEOUT);
      *abort = 1;
    }
    // the copies in flight land before the block ends
    for (uint32_t s = 0; s < (uint32_t)NS; ++s)
      if (blk > s) drain_wait(bars + 8 * (mRaw + s), ((blk - 1 - s) / NS) & 1);
  } else if (work && warp == kMassQ) {
    // ---- the queries: pieces of 64 channels of the row block, high halves then low ones
    MassWalk wk;
    wk.open(p);
    wk.start(lo, hi);
    if (elect_one()) {
      uint32_t q = 0;
      int held_k = -1, held_rb = -1;
      for (; ok && wk.valid(); wk.next()) {
        if (resident) {
          if (wk.k == held_k && wk.rb == held_rb) continue;
          held_k = wk.k;
          held_rb = wk.rb;
          // the old ones have been read
          if (q > 0 && !bar_wait(bars + 8 * mQDone, (q / 9 - 1) & 1, p.wait_ns, abort)) {
            ok = false;
            break;
          }
        }
        const int rows = wk.rows();
        const int64_t row = (int64_t)wk.s.q0 * p.H + wk.rb * R;
        for (int kb = 0; kb < 9; ++kb, ++q) {
          const uint32_t qs = q % QS;
          if (!resident && q >= (uint32_t)QS && !bar_wait(bars + 8 * (mQFree + qs), (q / QS - 1) & 1, p.wait_ns, abort)) {
            ok = false;
            break;
          }
          const uint8_t* src = p.q_tiles + ((int64_t)kb * p.rows + row) * 128;
          const uint32_t dst = sb + qs * R * 256;
          bar_expect(bars + 8 * (mQ + qs), rows * 256);
          bulk_copy(dst, src, rows * 128, bars + 8 * (mQ + qs));
          bulk_copy(dst + R * 128, src + (int64_t)9 * p.rows * 128, rows * 128, bars + 8 * (mQ + qs));
        }
      }
      if (!ok) {
        set_err(p.dev_err, MLA_DEVERR_TIMEOUT);
        *abort = 1;
      }
      for (uint32_t s = 0; s < (uint32_t)QS; ++s)
        if (q > s) drain_wait(bars + 8 * (mQ + s), ((q - 1 - s) / QS) & 1);
    }
    __syncwarp();
  }
  fence_before();
  __syncthreads();
  if (warp == kMassMma) {
    fence_after();
    tmem_free(tbase, 512);
  }
}

template <int LF, int KF>
mla_status launch_mass_fmt(const MassParams& p0, cudaStream_t stream) {
  using SH = MassShape<LF, KF>;
  MassParams p = p0;
  p.query_pieces = SH::query_pieces(p.R);
  p.raw_slots = SH::raw_slots(p.R);
  const int smem = p.query_pieces * p.R * 256 + p.raw_slots * SH::kBlock + kMassMisc + kMassAligned;
  static int configured[64] = {0};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !configured[dev]) {
    const mla_status st =
        cuda_status(cudaFuncSetAttribute(mass_kernel<LF, KF>, cudaFuncAttributeMaxDynamicSharedMemorySize, 232448));
    if (st != MLA_OK) return st;
    if (dev >= 0 && dev < 64) configured[dev] = 1;
  }
  return cuda_status(launch_pdl(mass_kernel<LF, KF>, dim3(p.grid), dim3(kMassThreads), smem, stream, p));
}

}  // namespace

}  // namespace mla
