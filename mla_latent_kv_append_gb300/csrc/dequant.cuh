// Loads and dequantizes a token's cached values 32 channels at a time.
//
// A token's 512 latent channels are 16 units of 32 channels, its 64 k_pe
// channels two more.  A unit's codes are 16 (4-bit), 32 (8-bit) or 64 (bf16)
// contiguous bytes of the block: the chunk swizzle permutes chunks within an
// aligned group of eight, and keeps a unit's chunks together.  Loading is
// apart from converting, so that a caller can have several units in flight.
#pragma once

#include <cuda_fp16.h>

#include "mla_internal.cuh"

namespace mla {

constexpr int kUnitChannels = 32;
constexpr int kLatentUnits = kDc / kUnitChannels;      // 16
constexpr int kKpeUnits = kDr / kUnitChannels;         // 2

template <int FMT, bool KPE>
struct UnitShape {
  static constexpr bool kInt4 = FMT == MLA_FMT_INT4_ASYM || FMT == MLA_FMT_INT4_SYM;
  static constexpr int kWords = FMT == MLA_FMT_BF16 ? 4 : (kInt4 ? 1 : 2);         // 16-byte pieces
  static constexpr int kGroup = KPE ? kKG : latent_group_size(FMT);
  static constexpr int kScales = FMT == MLA_FMT_BF16 ? 0 : (kGroup >= kUnitChannels ? 1 : kUnitChannels / kGroup);
  static constexpr bool kZeros = FMT == MLA_FMT_INT4_ASYM;
};

template <int FMT, bool KPE>
struct RawUnit {
  using S = UnitShape<FMT, KPE>;
  uint4 w[S::kWords];
  float s[S::kScales > 0 ? S::kScales : 1];
  float z[S::kZeros ? S::kScales : 1];
};

// Bytes of a 32-token block of a format pair (compute_layout's block_bytes).
template <int LF, int KF>
constexpr int block_bytes() {
  const int codes = 32 * UnitShape<LF, false>::kWords * 16 * kLatentUnits, kpe = 32 * UnitShape<KF, true>::kWords * 16 * kKpeUnits;
  const int quant = LF == MLA_FMT_BF16 ? 0 : 128 * (kDc / latent_group_size(LF)) * (LF == MLA_FMT_INT4_ASYM ? 2 : 1) + 128;
  return codes + kpe + quant + (KF == MLA_FMT_BF16 ? 0 : 128 * kNKG) + (LF == MLA_FMT_INT8_OUTLIER ? kOutFieldBytes : 0);
}
static_assert(block_bytes<MLA_FMT_INT8_SYM, MLA_FMT_INT8_SYM>() == 32 * 740 && block_bytes<MLA_FMT_BF16, MLA_FMT_BF16>() == 32 * 1152 &&
                  block_bytes<MLA_FMT_INT4_ASYM, MLA_FMT_INT4_SYM>() == 32 * 580,
              "the documented page sizes");

// Unit c of block token u; blk is the token's 32-token block, in shared memory
// (staged by a bulk copy).  A warp with one token per lane reads without bank
// conflicts: scales lie side by side, chunks are swizzled by token.
template <int FMT, bool KPE>
__device__ __forceinline__ void load_unit(const uint8_t* blk, const PageLayout& L, int u, int c, RawUnit<FMT, KPE>& r) {
  using S = UnitShape<FMT, KPE>;
  const uint4* row = reinterpret_cast<const uint4*>(blk + (KPE ? L.kpe_off + u * L.kpe_row : L.codes_off + u * L.codes_row));
#pragma unroll
  for (int i = 0; i < S::kWords; ++i) {
    const int chunk = c * S::kWords + i;
    r.w[i] = *(row + (KPE ? kpe_chunk_pos(chunk, u, FMT) : latent_chunk_pos(chunk, u)));
  }
  if constexpr (S::kScales > 0) {
    const float* sc = reinterpret_cast<const float*>(blk + (KPE ? L.kpe_scale_off : L.scale_off));
    const int g0 = c * kUnitChannels / S::kGroup;
#pragma unroll
    for (int i = 0; i < S::kScales; ++i) r.s[i] = sc[(g0 + i) * kBlockTokens + u];
    if constexpr (S::kZeros) {
      const float* zp = reinterpret_cast<const float*>(blk + L.zero_off);
#pragma unroll
      for (int i = 0; i < S::kScales; ++i) r.z[i] = zp[(g0 + i) * kBlockTokens + u];
    }
  }
}

// Largest magnitude that stays finite in fp16.
constexpr float kHalfMax = 65504.f;

// A scale rounded to 15 significant bits (2^-15 relative, a sixteenth of the
// fp16 rounding that follows).  A code q sits in a float's mantissa as f = 1 +
// q 2^-k, and
//   fma(f, 2^k s, -(2^k + zero) s) = (q - zero) s
// is then rounded once: (2^k + zero) s fits 24 bits (for 4-bit codes with k =
// 11 it is off by up to 2^-13 s, a 2^-13th of the codes' step).  One byte
// select or mask and one FMA per value, no conversion instructions.
__device__ __forceinline__ float short_scale(float s) {
  return __uint_as_float((__float_as_uint(s) + 0x100u) & 0xFFFFFE00u);
}
__device__ __forceinline__ uint32_t half2_word(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// A unit that reads as 0.
template <int FMT, bool KPE>
__device__ __forceinline__ void zero_unit(RawUnit<FMT, KPE>& r) {
  using S = UnitShape<FMT, KPE>;
#pragma unroll
  for (int i = 0; i < S::kWords; ++i) r.w[i] = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
  for (int i = 0; i < (S::kScales > 0 ? S::kScales : 1); ++i) r.s[i] = 0.f;
#pragma unroll
  for (int i = 0; i < (S::kZeros ? S::kScales : 1); ++i) r.z[i] = 0.f;
}

// The unit's 32 channels as fp16 pairs, h[i] = channels (2i, 2i + 1); false if
// one of them is not finite in fp16 (its group, or the unit, then reads as 0).
// Any scale and zero-point.
template <int FMT, bool KPE>
__device__ __forceinline__ bool convert_any(const RawUnit<FMT, KPE>& r, uint32_t* h) {
  using S = UnitShape<FMT, KPE>;
  bool fine = true;
  if constexpr (FMT == MLA_FMT_BF16) {
    __half2 acc = __float2half2_rn(0.f);
    const __half2 zero = acc;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w[4] = {r.w[i].x, r.w[i].y, r.w[i].z, r.w[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        h[4 * i + j] = half2_word(bf16lo(w[j]), bf16hi(w[j]));
        acc = __hfma2(*reinterpret_cast<const __half2*>(&h[4 * i + j]), zero, acc);   // NaN once one is not finite
      }
    }
    fine = !(__hisnan(__low2half(acc)) || __hisnan(__high2half(acc)));
    if (!fine) {
#pragma unroll
      for (int i = 0; i < 16; ++i) h[i] = 0u;
    }
  } else if constexpr (S::kInt4) {
    // k = 11 and k = 7: a nibble at bits 12..15 or 16..19, so one shift serves two
    float m[2][S::kScales], c[2][S::kScales];
#pragma unroll
    for (int g = 0; g < S::kScales; ++g) {
      const float zero = S::kZeros ? r.z[S::kZeros ? g : 0] : 8.f;
      const bool ok = fabsf(r.s[g]) * (S::kZeros ? fabsf(zero - 7.5f) + 7.5f : 7.f) <= kHalfMax;      // false for NaN
      fine &= ok;
      const float s = ok ? short_scale(r.s[g]) : 0.f, z = ok ? zero : 0.f;
      m[0][g] = 2048.f * s;
      c[0][g] = -(2048.f + z) * s;
      m[1][g] = 128.f * s;
      c[1][g] = -(128.f + z) * s;
    }
    const uint32_t w[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float v[8];                        // nibble k's value
#pragma unroll
      for (int k = 0; k < 8; k += 2) {
        const uint32_t t = k == 0 ? w[j] << 12 : (k == 2 ? w[j] << 4 : (k == 4 ? w[j] >> 4 : w[j] >> 12));
        const int g = int4_nibble_channel(j, k) / S::kGroup;       // nibble k + 1 is in the same group
        v[k] = fmaf(__uint_as_float((t & 0x0000F000u) | 0x3F800000u), m[0][g], c[0][g]);
        v[k + 1] = fmaf(__uint_as_float((t & 0x000F0000u) | 0x3F800000u), m[1][g], c[1][g]);
      }
      // nibbles k and k + 4 are adjacent channels
#pragma unroll
      for (int k = 0; k < 4; ++k) h[int4_nibble_channel(j, k) / 2] = half2_word(v[k], v[k + 4]);
    }
  } else {
    float m[S::kScales], c[S::kScales];
#pragma unroll
    for (int g = 0; g < S::kScales; ++g) {
      const bool ok = fabsf(r.s[g]) * 127.f <= kHalfMax;
      fine &= ok;
      const float s = ok ? short_scale(r.s[g]) : 0.f;
      m[g] = 32768.f * s;
      c[g] = -32896.f * s;               // codes are biased by 128 below
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t w[4] = {r.w[i].x ^ 0x80808080u, r.w[i].y ^ 0x80808080u, r.w[i].z ^ 0x80808080u,
                             r.w[i].w ^ 0x80808080u};
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int k = 0; k < 4; k += 2) {
          // 8-channel latent groups store channels 2j, 2j+1, 8+2j, 8+2j+1 in word j
          const int ch = 16 * i + (!KPE && S::kGroup == 8 ? 2 * j + 4 * k : 4 * j + k);
          const int g = S::kScales > 1 ? ch / S::kGroup : 0;
          const float a = __uint_as_float(__byte_perm(w[j], 0x3F800000u, 0x7604 | (k << 4)));
          const float b = __uint_as_float(__byte_perm(w[j], 0x3F800000u, 0x7604 | ((k + 1) << 4)));
          h[ch / 2] = half2_word(fmaf(a, m[g], c[g]), fmaf(b, m[g], c[g]));
        }
    }
  }
  return fine;
}

// The same, two channels at a time in fp16 arithmetic where that is as exact:
// codes become exact half integers by placing them in the mantissa of
// 1024, subtracting the offset and zero-point is exact, and the scale is split
// into two halves, s = hi + lo, so that q hi + q lo is rounded once.  lo lies on
// fp16's subnormal grid, off by up to 2^-25: for scales from 2^-10 on that is
// 2^-15 of s at most, what convert_any's short scale is off by (an eighth of
// half a step of the fp16 result at most; at 2^-13 it would be a whole half step).
// 11 issue slots for four INT8 codes against 16 of convert_any (byte selects,
// logic and conversions run at half rate).  Needs scales in that range, or
// zero, and small zero-points: other units take convert_any.
template <int FMT, bool KPE>
__device__ __forceinline__ bool convert_unit(const RawUnit<FMT, KPE>& r, uint32_t* h) {
  using S = UnitShape<FMT, KPE>;
  if constexpr (FMT == MLA_FMT_BF16) {
    return convert_any<FMT, KPE>(r, h);
  } else {
    constexpr uint32_t kLow = 0x3A800000u, kHigh = S::kInt4 ? 0x42800000u : 0x44000000u;     // 2^-10 .. 64 or 512
    bool fast = true;
#pragma unroll
    for (int g = 0; g < S::kScales; ++g) {
      fast &= __float_as_uint(r.s[g]) - kLow <= kHigh - kLow || r.s[g] == 0.f;
      if constexpr (S::kZeros) fast &= fabsf(r.z[g]) <= 512.f;
    }
    if (!fast) return convert_any<FMT, KPE>(r, h);
    __half2 hi[S::kScales], lo[S::kScales];
#pragma unroll
    for (int g = 0; g < S::kScales; ++g) {
      hi[g] = __float2half2_rn(r.s[g]);
      lo[g] = __float2half2_rn(r.s[g] - __low2float(hi[g]));
    }
    auto put = [&](int ch, __half2 q, int g) {
      const __half2 x = __hfma2(q, hi[g], __hmul2(q, lo[g]));
      h[ch / 2] = *reinterpret_cast<const uint32_t*>(&x);
    };
    auto half2_of = [](uint32_t w) { return *reinterpret_cast<const __half2*>(&w); };
    if constexpr (S::kInt4) {
      __half2 off[S::kScales], off16[S::kScales];          // -(1024 + zero), -(64 + zero): exact
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
          put(ch, (k & 1) ? __hfma2(half2_of((t & 0x00F000F0u) | 0x64006400u), sixteenth, off16[g])
                          : __hadd2(half2_of((t & 0x000F000Fu) | 0x64006400u), off[g]),
              g);
        }
    } else {
      const __half2 off = __float2half2_rn(-1152.f);       // 1024 and the codes' bias of 128
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t w[4] = {r.w[i].x ^ 0x80808080u, r.w[i].y ^ 0x80808080u, r.w[i].z ^ 0x80808080u,
                               r.w[i].w ^ 0x80808080u};
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int k = 0; k < 4; k += 2) {
            const int ch = 16 * i + (!KPE && S::kGroup == 8 ? 2 * j + 4 * k : 4 * j + k);
            put(ch, __hadd2(half2_of(__byte_perm(w[j], 0x64646464u, k ? 0x4342 : 0x4140)), off),
                S::kScales > 1 ? ch / S::kGroup : 0);
          }
      }
    }
    return true;
  }
}

// INT8_OUTLIER: puts the protected channels of unit c in their places; false
// if one is not finite in fp16 (it then reads as 0).
template <int FMT>
__device__ __forceinline__ bool patch_outliers(const uint8_t* blk, const PageLayout& L, const OutlierSet& outl, int u,
                                               int c, uint32_t* h) {
  bool fine = true;
  if constexpr (FMT == MLA_FMT_INT8_OUTLIER) {
    const uint32_t mask = outl.mask[c];
    if (!mask) return true;
    const uint16_t* ov = reinterpret_cast<const uint16_t*>(blk + L.outlier_off);
    for (int k = 0; k < kNOut; ++k) {
      const int ch = outl.ch[k];
      if ((ch >> 5) != c) continue;
      float v = bf16f(ov[k * kBlockTokens + u]);
      if (!(fabsf(v) <= kHalfMax)) {
        fine = false;
        v = 0.f;
      }
      const uint32_t bits = half2_word(v, v);
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (i == ((ch & 31) >> 1)) h[i] = (ch & 1) ? ((h[i] & 0xFFFFu) | (bits & 0xFFFF0000u)) : ((h[i] & 0xFFFF0000u) | (bits & 0xFFFFu));
    }
  }
  return fine;
}

}  // namespace mla
