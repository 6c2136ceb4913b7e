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
//
// What bounds it: the MMAs, 75 to 92 cycles each with A in TMEM, and for 128 rows the
// queries' way from L2 (295 KB for a pass, 40 bytes a cycle and SM).  Measured
// (a captured call's share of many): 4 x 16000 tokens INT8, a window of 32 queries at 16 heads
// 94 us, 390 TFLOP/s of scores or 20% of the bf16 rate, of which three products make
// 60%; 24 drafts of up to 5 tokens at 64 heads, bf16, 79 us; 32 x 32768 tokens INT4
// at 32 heads 206 us, at 64 heads 241, at 128 heads 355; 32 x 16384 tokens at 32 heads
// 109 to 114 us in every format (4.0 TB/s in INT8 blocks of 8), but 288 with protected
// channels, which are put in their places one by one.  The roles' code together spills
// 184 bytes a thread at the 64 registers that 1024 threads leave.
//
// Work split: all passes (a key tile, up to 128 rows) in a row, cut into runs of equal
// cost, one to an SM.  A tile that several blocks share is added up by whichever
// finishes last, in the blocks' order, so that results repeat bit for bit.
#pragma once

#include <math.h>

#include "dequant.cuh"
#include "mass_params.cuh"
#include "tc.cuh"

namespace mla {
namespace {

using namespace tc;

// Warps: 24 convert, 4 read the scores, then one each issues the MMAs, the
// cache's copies and the queries' copies; one is idle.
constexpr int kMassGroups = 6, kMassConvert = 4 * kMassGroups, kMassRead = kMassConvert, kMassMma = kMassRead + 4, kMassRaw = kMassMma + 1,
              kMassQ = kMassMma + 2, kMassWarps = kMassMma + 4;
constexpr int kMassThreads = 32 * kMassWarps;
constexpr int kMassUnits = kLatentUnits + kKpeUnits;   // 18 units of 32 channels, two to a piece
static_assert(kMassUnits == 3 * kMassGroups && kMassThreads == 1024, "a converting warp has three units of a tile");
constexpr int kMassSmem = 232448 - 1024;               // a block's shared memory, less the alignment slack
constexpr int kMassMaxRaw = 8;
constexpr int kMassAligned = 1024;

// Barriers.
enum { mA = 0, mAFree = mA + 8, mS = mAFree + 8, mE = mS + 2, mRaw = mE + 2, mRawFree = mRaw + kMassMaxRaw, mQ = mRawFree + kMassMaxRaw,
       mQFree = mQ + 9, mQDone = mQFree + 9, mFin, mCount };
constexpr int kMassMisc = 8 * mCount + 64 + kMassMaxRows * 4;      // barriers, words, the rows' lse
static_assert(8 * mCount + 64 <= 1024, "barriers and words");

// Byte offsets in a 32-token block of a format pair (compute_layout's), known
// at compile time: with runtime ones a fifth of the conversion's instructions
// were address arithmetic.
template <int LF, int KF>
struct BlockAt {
  static constexpr int kRow = 16 * UnitShape<LF, false>::kWords * kLatentUnits, kKpeRow = 16 * UnitShape<KF, true>::kWords * kKpeUnits;
  static constexpr int kScale = kBlockTokens * kRow;
  static constexpr int kGroups = LF == MLA_FMT_BF16 ? 0 : kDc / latent_group_size(LF);
  static constexpr int kZero = kScale + 128 * kGroups;
  static constexpr int kOutlier = kZero + (LF == MLA_FMT_INT4_ASYM ? 128 * kGroups : 0);
  static constexpr int kKpe = kOutlier + (LF == MLA_FMT_INT8_OUTLIER ? kOutFieldBytes : 0);
  static constexpr int kKpeScale = kKpe + kBlockTokens * kKpeRow;
  static constexpr int kBytes = kKpeScale + (KF == MLA_FMT_BF16 ? 0 : 128 * kNKG) + (LF == MLA_FMT_BF16 ? 0 : 128);
  static_assert(kBytes == block_bytes<LF, KF>(), "the documented block");
};

__device__ __forceinline__ uint4 lds16(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];\n" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ float lds4(uint32_t at) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];\n" : "=f"(v) : "r"(at) : "memory");
  return v;
}

// Unit c of token u: row = the token's code row in shared memory (on a 32-byte
// boundary or more, so that chunk i of the unit is chunk 0's address with i's bits
// flipped), scale and zero = the token's entries of group 0.
template <int FMT, bool KPE>
__device__ __forceinline__ void load_split(uint32_t row, uint32_t scale, uint32_t zero, int u, int c, RawUnit<FMT, KPE>& r) {
  using S = UnitShape<FMT, KPE>;
  const uint32_t at = row + 16 * (KPE ? kpe_chunk_pos(c * S::kWords, u, FMT) : latent_chunk_pos(c * S::kWords, u));
#pragma unroll
  for (int i = 0; i < S::kWords; ++i) r.w[i] = lds16(at ^ (16 * i));
  if constexpr (S::kScales > 0) {
    const uint32_t g = 128 * (c * kUnitChannels / S::kGroup);
#pragma unroll
    for (int i = 0; i < S::kScales; ++i) {
      r.s[i] = lds4(scale + g + 128 * i);
      if constexpr (S::kZeros) r.z[i] = lds4(zero + g + 128 * i);
    }
  }
}

template <int LF, int KF>
struct MassShape {
  static constexpr int kBlock = BlockAt<LF, KF>::kBytes;
  // A bulk copy costs 85 ns of the copy engine besides its bytes, and a block of
  // 4-bit codes is 18 KB: whole pages of those (a stream of nothing but copies:
  // 18.5 KB each 5.6 TB/s, 23.7 KB 7.0, 37 KB 6.9).
  static constexpr int kBlocks = kBlock < 20000 ? 2 : 1;             // 32-token blocks of a copy
  static constexpr int kCopy = kBlocks * kBlock;
  static constexpr int kTileCopies = 4 / kBlocks;
  // TMEM columns of a piece (64 channels): a bf16 value has no low half
  static constexpr int kCols = LF == MLA_FMT_BF16 && KF == MLA_FMT_BF16 ? 32 : 64;
  // shared memory: queries of R rows in `qs` pieces, then the copies
  static constexpr int query_pieces(int R) {
    const int room = kMassSmem - 2048 - (kTileCopies + 1) * kCopy, piece = R * 256;
    return 9 * piece <= room ? 9 : (room / piece >= 2 ? room / piece : 2);
  }
  static constexpr int raw_slots(int R) {
    const int n = (kMassSmem - 2048 - query_pieces(R) * R * 256) / kCopy;
    return n < kMassMaxRaw ? n : kMassMaxRaw;
  }
  static_assert(raw_slots(kMassMaxRows) >= kTileCopies && raw_slots(64) >= kTileCopies && raw_slots(32) >= kTileCopies &&
                    raw_slots(16) >= kTileCopies,
                "a whole key tile");
};

// A block's walk over its passes (a row block of a key tile).
struct MassWalk {
  const MassSeq* seqs;
  int n_seqs, k, tile, rb, R, cost;                    // cost: of a full row block
  int64_t left;                                        // passes, the current one included
  MassSeq s;

  __device__ __forceinline__ void load() {
    const int4* r = reinterpret_cast<const int4*>(seqs + k);
    int4* d = reinterpret_cast<int4*>(&s);
#pragma unroll
    for (int i = 0; i < (int)sizeof(MassSeq) / 16; ++i) d[i] = __ldcg(r + i);
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
  // All lanes of a warp: passes that start before unit v, and the first that does not.
  __device__ __forceinline__ int64_t passes_before(int64_t v) {
    find(v);
    const int64_t d = v - s.unit0, t = d / s.tile_cost;
    tile = (int)t;
    rb = min(s.blocks, ((int)(d - t * s.tile_cost) + cost - 1) / cost);
    return s.pass0 + t * s.blocks + rb;
  }
  __device__ __forceinline__ void open(const MassParams& p, int64_t U, int64_t lo, int64_t hi) {
    seqs = p.seqs;
    n_seqs = __ldcg(&p.counts->seqs);
    R = p.R;
    cost = mass_cost(R);
    k = -1;
    left = hi == U ? __ldcg(&p.counts->passes) : passes_before(hi);
    left -= passes_before(lo);
    if (left > 0 && rb == s.blocks) step();
  }
  __device__ __forceinline__ bool valid() const { return left > 0; }
  // From behind a tile's last row block.
  __device__ __forceinline__ void step() {
    rb = 0;
    if (++tile >= s.tiles) {
      tile = 0;
      ++k;
      load();
    }
  }
  __device__ __forceinline__ void next() {
    --left;
    if (++rb >= s.blocks && left > 0) step();
  }
  __device__ __forceinline__ int rows() const { return min(R, s.n * s.heads - rb * R); }
};

__device__ __forceinline__ __half2 as_half2(uint32_t w) { return *reinterpret_cast<const __half2*>(&w); }
__device__ __forceinline__ uint32_t as_word(__half2 h) { return *reinterpret_cast<const uint32_t*>(&h); }

// (a, b) as halves: lo - hi.
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(-a, -b);
  hi = as_word(h);
  lo = as_word(__floats2half2_rn(a + __low2float(h), b + __high2float(h)));
}

// The unit's 32 channels times kKeyGain: lo[i] - hi[i] = channels (2i, 2i + 1).
// Any scale and zero-point.
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
  using S = UnitShape<FMT, KPE>;
  if constexpr (FMT == MLA_FMT_BF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w[4] = {r.w[i].x, r.w[i].y, r.w[i].z, r.w[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) hi[4 * i + j] = half2_bits(bf16lo(w[j]) * -kKeyGain, bf16hi(w[j]) * -kKeyGain);
    }
  } else {
    // Two channels at a time in fp16 arithmetic.  Codes q become exact halves
    // (placed in the mantissa of 1024, the offset and zero-point taken off), the scale
    // is two halves, a + b; then with h = fl(q a) the rest q a - h is exact in a half
    // (q has at most 8 bits), and l = fl(q b + (q a - h)): three instructions a
    // pair, 2^-22 of x.  (h is made as q (-a), which the last step needs, and stays
    // negated: the MMA turns it back.)  b lies on fp16's subnormal grid, off by up to 2^-25: for
    // scales from 2^-9 on 2^-20 of them at most.  Needs scales in that range and
    // zero-points that keep q a finite; other units go through fp32.
    constexpr uint32_t kLow = 0x3B000000u, kHigh = 0x41800000u;      // 2^-9 .. 16
    uint32_t most = 0u;
    float top = 0.f;
#pragma unroll
    for (int g = 0; g < S::kScales; ++g) {
      most = max(most, __float_as_uint(r.s[g]) - kLow);
      if constexpr (S::kZeros) top = max_nan(top, fabsf(r.z[g]));
    }
    if (most > kHigh - kLow || !(top <= 127.f)) {
      split_any<FMT, KPE>(r, hi, lo);
      return;
    }
    __half2 a[S::kScales], b[S::kScales], minus_a[S::kScales];
#pragma unroll
    for (int g = 0; g < S::kScales; ++g) {
      const float s = r.s[g] * kKeyGain;
      a[g] = __float2half2_rn(s);
      minus_a[g] = as_half2(as_word(a[g]) ^ 0x80008000u);
      b[g] = __float2half2_rn(s - __low2float(a[g]));
    }
    auto put = [&](int ch, __half2 q, int g) {
      const __half2 h = __hmul2_rn(q, minus_a[g]);
      hi[ch / 2] = as_word(h);
      lo[ch / 2] = as_word(__hfma2(q, b[g], __hfma2(q, a[g], h)));
    };
    if constexpr (S::kInt4) {
      __half2 off[S::kScales], off16[S::kScales];      // -(1024 + zero), -(64 + zero): exact
#pragma unroll
      for (int g = 0; g < S::kScales; ++g) {
        const float zero = S::kZeros ? r.z[S::kZeros ? g : 0] : 8.f;
        off[g] = __float2half2_rn(-1024.f - zero);
        off16[g] = __float2half2_rn(-64.f - zero);
      }
      const __half2 sixteenth = __float2half2_rn(0.0625f);
      const uint32_t w[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          // nibbles k and k + 4 are adjacent channels; odd ones stand 16 times as high
          const uint32_t t = k < 2 ? w[j] : w[j] >> 8;
          const int ch = int4_nibble_channel(j, k), g = ch / S::kGroup;
          put(ch, (k & 1) ? __hfma2(as_half2((t & 0x00F000F0u) | 0x64006400u), sixteenth, off16[g])
                          : __hadd2(as_half2((t & 0x000F000Fu) | 0x64006400u), off[g]),
              g);
        }
    } else {
      const __half2 off = __float2half2_rn(-1152.f);   // 1024 and the codes' bias of 128
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t w[4] = {r.w[i].x ^ 0x80808080u, r.w[i].y ^ 0x80808080u, r.w[i].z ^ 0x80808080u,
                               r.w[i].w ^ 0x80808080u};
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int k = 0; k < 4; k += 2) {
            const int ch = 16 * i + (!KPE && S::kGroup == 8 ? 2 * j + 4 * k : 4 * j + k);
            put(ch, __hadd2(as_half2(__byte_perm(w[j], 0x64646464u, k ? 0x4342 : 0x4140)), off),
                S::kScales > 1 ? ch / S::kGroup : 0);
          }
      }
    }
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

constexpr uint32_t kNegateA = 1u << 13;                // instruction descriptor: the products of -A
__device__ __forceinline__ void tmem_put16(uint32_t t, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n" ::"r"(t),
      MLA_V8(v, 0), MLA_V8(v, 8)
      : "memory");
}
__device__ __forceinline__ void tmem_put_wait() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }

// One arrival for the warp (32 on one barrier are carried out one after the
// other: a tile's 3200 of them took 4700 cycles).
__device__ __forceinline__ void warp_arrive(uint32_t bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) bar_arrive(bar);
}

// A ring's copy in round `round` of its place.  Warps share the copies out among
// them, and where the places are no multiple of the shares a place goes from warp to
// warp: the copy before this one is another warp's and may land after this warp's own
// last one, and a wait by parity for this one would take the round before that for
// it.  So that one's release first, which is at most one round behind (it was issued
// before this warp's last copy); from then on `full` is in this round or behind it.
__device__ __forceinline__ bool ring_wait(uint32_t full, uint32_t free, uint32_t round, uint64_t limit_ns, volatile int* abort) {
  return (round == 0 || warp_wait(free, (round - 1) & 1, limit_ns, abort)) && warp_wait(full, round & 1, limit_ns, abort);
}

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
  constexpr int COLS = SH::kCols;
  extern __shared__ uint8_t mass_smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(mass_smem_raw) + kMassAligned - 1) & ~(uintptr_t)(kMassAligned - 1));
  const int R = p.R, QS = p.query_pieces, NS = p.raw_slots;
  const bool resident = QS == 9;
  // TMEM: two buffers of scores, then pieces of PU units.  Up to 64 rows the MMAs
  // of 64 channels take less time (256 cycles) than their thread takes for a
  // piece besides (370), so a piece has 192 channels.
  const int d_cols = mass_columns(R), PU = R <= 64 ? 6 : 2, cols = COLS / 2 * PU, NA = min(8, (512 - 2 * d_cols) / cols);
  const int pieces = kMassUnits / PU;
  const uint32_t sb = smem_u32(sm), s_raw = QS * R * 256, bars = sb + s_raw + NS * SH::kCopy;
  uint8_t* words = sm + s_raw + NS * SH::kCopy + 8 * mCount;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(words);
  volatile int* abort = reinterpret_cast<volatile int*>(words + 4);
  volatile int* s_last = reinterpret_cast<volatile int*>(words + 8);
  float* s_lse = reinterpret_cast<float*>(words + 64);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 8; ++i) {
      bar_init(bars + 8 * (mA + i), 4 * PU);           // four warps write a unit
      bar_init(bars + 8 * (mAFree + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(bars + 8 * (mS + i), 1);
      bar_init(bars + 8 * (mE + i), 4);
    }
    for (int i = 0; i < kMassMaxRaw; ++i) {
      bar_init(bars + 8 * (mRaw + i), 1);
      bar_init(bars + 8 * (mRawFree + i), kMassGroups * SH::kBlocks);    // the warps of its tokens' lanes
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
  const uint32_t tbase = *tmem_slot, t_a = tbase + 2 * d_cols;
  pdl_launch_dependents();
  pdl_wait();

  const int64_t U = __ldcg(&p.counts->units);
  const int G = (int)(U < gridDim.x ? U : gridDim.x), x = blockIdx.x;
  const bool work = x < G;
  const int64_t lo = work ? mass_run(U, x, G) : 0, hi = work ? mass_run(U, x + 1, G) : 0;
  bool ok = true;
  if (work && warp < kMassConvert) {
    // ---- Warp (e, d): lanes 32 d .. 32 d + 31 (a 32-token block of the tile) of
    // units e, e + 6 and e + 12; lane = token.
    using AT = BlockAt<LF, KF>;
    const int e = warp >> 2, d = warp & 3;
    const uint32_t tl = (uint32_t)(32 * d) << 16;
    int64_t n_pass;
    {
      MassWalk wk;
      wk.open(p, U, lo, hi);
      n_pass = wk.left;
    }
    int rs = d / SH::kBlocks, slot0 = 0;               // raw copy; TMEM place of the pass's first piece
    uint32_t raw_round = 0, round0 = 0;                // how often they went round
    for (; n_pass > 0; --n_pass) {
      if (!(ok = ring_wait(bars + 8 * (mRaw + rs), bars + 8 * (mRawFree + rs), raw_round, p.wait_ns, abort))) break;
      const uint32_t raw = s_raw + rs * SH::kCopy + (d % SH::kBlocks) * SH::kBlock, at = sb + raw;
#pragma unroll 1
      for (int j = e; j < kMassUnits; j += kMassGroups) {
        uint32_t h[16], l[16];
        const bool last = j + kMassGroups >= kMassUnits;
        bool split;
        if (j < kLatentUnits) {
          RawUnit<LF, false> r;
          load_split<LF, false>(at + lane * AT::kRow, at + AT::kScale + 4 * lane, at + AT::kZero + 4 * lane, lane, j, r);
          if (last && LF != MLA_FMT_INT8_OUTLIER) warp_arrive(bars + 8 * (mRawFree + rs));
          split_unit<LF, false>(r, h, l);
          patch_split<LF>(sm + raw, p.L, p.outl, lane, j, h, l);
          if (last && LF == MLA_FMT_INT8_OUTLIER) warp_arrive(bars + 8 * (mRawFree + rs));      // its protected channels lie there
          split = LF != MLA_FMT_BF16;
        } else {
          RawUnit<KF, true> r;
          load_split<KF, true>(at + AT::kKpe + lane * AT::kKpeRow, at + AT::kKpeScale + 4 * lane, 0u, lane, j - kLatentUnits, r);
          warp_arrive(bars + 8 * (mRawFree + rs));
          split_unit<KF, true>(r, h, l);
          split = KF != MLA_FMT_BF16;
        }
        const int piece = PU == 6 ? j / 6 : j >> 1, unit = j - piece * PU;
        int slot = slot0 + piece;
        uint32_t round = round0;
        while (slot >= NA) {
          slot -= NA;
          ++round;
        }
        // the place's last piece has been multiplied (releases come in the ring's
        // order, so the barrier is at most one phase behind)
        if (round > 0 && !(ok = warp_wait(bars + 8 * (mAFree + slot), (round - 1) & 1, p.wait_ns, abort))) break;
        fence_after();
        const uint32_t a = t_a + slot * cols + tl + 16 * unit;
        tmem_put16(a, h);
        if (split) tmem_put16(a + 16 * PU, l);
        tmem_put_wait();
        fence_before();
        warp_arrive(bars + 8 * (mA + slot));
      }
      if (!ok) break;
      rs += SH::kTileCopies;
      if (rs >= NS) {
        rs -= NS;
        ++raw_round;
      }
      slot0 += pieces;
      while (slot0 >= NA) {
        slot0 -= NA;
        ++round0;
      }
    }
    if (!ok) {
      set_err(p.dev_err, MLA_DEVERR_TIMEOUT);
      *abort = 1;
    }
  } else if (work && warp >= kMassRead && warp < kMassMma) {
    // ---- the scores: thread = key.  The walk is a pass ahead, so that a tile's
    // old masses are there when its scores are; the lanes fetch the page ids of
    // 32 tiles at a time.
    MassWalk wk;
    wk.open(p, U, lo, hi);
    const int key = threadIdx.x - 32 * kMassRead, half = (warp & 3) >> 1;        // the warp's keys lie in one page of the tile
    const uint32_t tl = (uint32_t)(32 * (warp & 3)) << 16;
    int ids = -1, ids_k = -1, ids_tile = 0, page = -1, parts = 0;
    float old = 0.f, total = 0.f;
    // the walk's tile: its page (-1: none that counts) and old mass
    auto look = [&](int& pg, float& m) {
      const int t = wk.tile * kMassKeys + key;
      if (wk.k != ids_k || wk.tile >= ids_tile + 32) {
        ids_k = wk.k;
        ids_tile = wk.tile;
        const int at = 2 * (wk.tile + lane) + half;
        ids = (int64_t)at * kPage < wk.s.len ? __ldcg(p.table + (int64_t)wk.s.b * p.max_pages + at) : -1;
      }
      pg = __shfl_sync(0xffffffffu, ids, wk.tile - ids_tile);
      m = 0.f;
      if (t >= wk.s.len) {
        pg = -1;
      } else if (pg < 0 || pg >= p.num_pages) {
        set_err(p.dev_err, MLA_DEVERR_PAGE);
        pg = -1;
      } else if (t < wk.s.counted) {
        m = __ldcg(p.mass + (int64_t)pg * kPage + (t & (kPage - 1)));
      }
    };
    if (wk.valid()) look(page, old);
    uint32_t it = 0;
    int held_k = -1, held_rb = -1;
    bool odd = false, late = false;                    // odd: a row without a finite lse
    for (; wk.valid(); ++it) {
      const uint32_t g = it & 1;
      const int rows = wk.rows(), row0 = wk.rb * R, ctx = wk.s.len - wk.s.n, n = wk.s.n, t = wk.tile * kMassKeys + key;
      const int tile = wk.tile, k = wk.k, blocks = wk.s.blocks;
      const int64_t u0 = wk.s.unit0 + (int64_t)tile * wk.s.tile_cost;
      if (k != held_k || wk.rb != held_rb) {
        held_k = k;
        held_rb = wk.rb;
        const float v = key < rows ? __ldcg(p.lse + (int64_t)wk.s.q0 * p.H + row0 + key) * -1.4426950408889634f : 0.f;
        const bool fin = fabsf(v) < INFINITY;
        asm volatile("bar.sync 1, 128;\n" ::: "memory");             // the old ones have been read
        s_lse[key] = fin ? v : -INFINITY;
        odd = vote_128(!fin);
      }
      wk.next();
      const bool done = !wk.valid() || wk.k != k || wk.tile != tile;             // the tile's last pass of this block
      int next_page = -1;
      float next_old = 0.f;
      if (done && wk.valid()) look(next_page, next_old);
      // the four warps meet at barriers: they leave together
      late = !warp_wait(bars + 8 * (mS + g), (it >> 1) & 1, p.wait_ns, abort);
      if (late) *abort = 1;
      if (vote_128(late)) {
        late = true;
        break;
      }
      fence_after();
      // rows from `first` on see the key
      const int pos = t - ctx, first = pos > 0 ? (pos >= n ? rows : max(pos * p.H - row0, 0)) : 0;
      const bool plain = __all_sync(0xffffffffu, first == 0 && !odd);
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
      for (int c0 = 0; c0 < rows; c0 += 16) {
        uint32_t r[16];
        tmem_load16(tbase + g * d_cols + c0 + tl, r);
        if (2 * rows <= d_cols) {                      // the queries' low halves have columns of their own
          uint32_t l[16];
          tmem_load16(tbase + g * d_cols + rows + c0 + tl, l);
#pragma unroll
          for (int c = 0; c < 16; ++c) r[c] = __float_as_uint(__uint_as_float(r[c]) + __uint_as_float(l[c]));
        }
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
      warp_arrive(bars + 8 * (mE + g));
      total += (sum[0] + sum[1]) + (sum[2] + sum[3]);
      ++parts;
      if (!done) continue;
      bool mine = true;
      if (parts < blocks) {
        // several blocks share the tile: its parts are added up, in the blocks'
        // order, by whichever is the last to finish
        const int x0 = mass_run_of(U, u0, G), x1 = mass_run_of(U, u0 + (int64_t)(blocks - 1) * wk.cost, G);
        __stcg(p.parts + (int64_t)(2 * x + (x == x0 ? 1 : 0)) * kMassKeys + key, total);
        __threadfence();
        asm volatile("bar.sync 1, 128;\n" ::: "memory");
        if (key == 0) *s_last = atomicAdd(p.done + x0, parts) + parts == blocks;
        asm volatile("bar.sync 1, 128;\n" ::: "memory");
        mine = *s_last != 0;
        asm volatile("bar.sync 1, 128;\n" ::: "memory");
        if (mine) {
          __threadfence();
          total = 0.f;
          for (int y = x0; y <= x1; ++y) {
            // a block whose run holds no pass of the tile has no part
            const int64_t from = mass_run(U, y, G) - u0, to = mass_run(U, y + 1, G) - u0;
            const int64_t r0 = from <= 0 ? 0 : (from + wk.cost - 1) / wk.cost;
            if (r0 < blocks && r0 * wk.cost < to) total += __ldcg(p.parts + (int64_t)(2 * y + (y == x0 ? 1 : 0)) * kMassKeys + key);
          }
        }
      }
      if (mine && page >= 0) p.mass[(int64_t)page * kPage + (t & (kPage - 1))] = fmaf(old, p.decay, total);
      page = next_page;
      old = next_old;
      total = 0.f;
      parts = 0;
    }
    if (late) set_err(p.dev_err, MLA_DEVERR_TIMEOUT);
  } else if (work && warp == kMassMma) {
    // ---- one thread issues the MMAs (with the whole warp in the loop and one lane
    // issuing, a 32-query window over 4 x 16000 tokens took 112 us)
    MassWalk wk;
    wk.open(p, U, lo, hi);
    if (elect_one()) {
      const uint64_t d_q = sw128_desc(sb, 16, 1024);
      uint32_t it = 0, q_round = 0, id = 0, id_minus = 0, id_both = 0, lo_step = 0;
      int qs = 0, slot = 0, round = 0, held_k = -1, held_rb = -1;
      bool both = false;
      while (ok && wk.valid()) {
        const uint32_t g = it & 1, d = tbase + g * d_cols;
        const bool held = resident && wk.k == held_k && wk.rb == held_rb;
        if (wk.k != held_k || wk.rb != held_rb) {
          held_k = wk.k;
          held_rb = wk.rb;
          // Where the buffer has the columns (up to 32 rows), both halves of the
          // queries are one N of twice the rows: an MMA with A in TMEM costs about
          // 75 cycles however small its N is.
          const int rows = wk.rows();
          both = 2 * rows <= d_cols;
          id = f16_idesc(128, rows, false, false);
          id_minus = id | kNegateA;
          id_both = (both ? f16_idesc(128, 2 * rows, false, false) : id) | kNegateA;
          lo_step = rows * 128 >> 4;
          if (resident && it > 0) umma_commit(bars + 8 * mQDone);      // the old queries' last reader
        }
        wk.next();
        // the scores of two passes before have been read
        if (it >= 2 && !(ok = bar_wait(bars + 8 * (mE + g), ((it - 2) >> 1) & 1, p.wait_ns, abort))) break;
        for (int kb = 0; kb < 9;) {
          if (!(ok = bar_wait(bars + 8 * (mA + slot), round & 1, p.wait_ns, abort))) break;
          uint32_t a = t_a + slot * cols;
          for (const int end = kb + PU / 2; kb < end; ++kb, a += 32) {
            if (!held && !(ok = bar_wait(bars + 8 * (mQ + qs), q_round & 1, p.wait_ns, abort))) break;
            fence_after();
            const uint64_t b_hi = d_q + (uint32_t)(qs * R * 16);
            umma4_ta<2>(d, a, b_hi, id_both, kb != 0);
            if (!both) umma4_ta<2>(d, a, b_hi + lo_step, id_minus, 1u);
            if (kb < 8 ? LF != MLA_FMT_BF16 : KF != MLA_FMT_BF16) umma4_ta<2>(d, a + 16 * PU, b_hi, id, 1u);
            if (!resident) umma_commit(bars + 8 * (mQFree + qs));
            if (++qs == QS) {
              qs = 0;
              if (!held) ++q_round;
            }
          }
          if (!ok) break;
          umma_commit(bars + 8 * (mAFree + slot));
          if (++slot == NA) {
            slot = 0;
            ++round;
          }
        }
        if (ok) umma_commit(bars + 8 * (mS + g));
        ++it;
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
    wk.open(p, U, lo, hi);
    constexpr int C = SH::kTileCopies;
    auto pages = [&]() {                               // lane i < C: the page of copy i of the walk's tile, -1: nothing to load
      const int t = wk.tile * kMassKeys + kMassKeys / C * (lane & (C - 1));
      return wk.valid() && lane < C && t < wk.s.len ? __ldcg(p.table + (int64_t)wk.s.b * p.max_pages + t / kPage) : -1;
    };
    uint32_t blk = 0;
    int ids = pages();
    while (ok && wk.valid()) {
      const int mine = ids >= 0 && ids < p.num_pages ? ids : -1;
      wk.next();
      ids = pages();
      for (int i = 0; i < C; ++i, ++blk) {
        const uint32_t slot = blk % NS;
        if (blk >= (uint32_t)NS && !warp_wait(bars + 8 * (mRawFree + slot), ((blk / NS) - 1) & 1, p.wait_ns, abort)) {
          ok = false;
          break;
        }
        const int page = __shfl_sync(0xffffffffu, mine, i);
        if (lane == 0) {
          if (page >= 0) {
            bar_expect(bars + 8 * (mRaw + slot), SH::kCopy);
            bulk_copy(sb + s_raw + slot * SH::kCopy, p.pool + (int64_t)page * p.L.page_bytes + (C == 4 ? (i & 1) * SH::kBlock : 0),
                      SH::kCopy, bars + 8 * (mRaw + slot));
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
    wk.open(p, U, lo, hi);
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
          bulk_copy(dst + rows * 128, src + (int64_t)9 * p.rows * 128, rows * 128, bars + 8 * (mQ + qs));
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
  const int smem = p.query_pieces * p.R * 256 + p.raw_slots * SH::kCopy + kMassMisc + kMassAligned;
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
