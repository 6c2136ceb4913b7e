// Loads and dequantizes a token's cached values 32 channels at a time.
//
// A token's 512 latent channels are 16 units of 32 channels, its 64 k_pe
// channels two more.  A unit's codes are 16 (4-bit), 32 (8-bit) or 64 (bf16)
// contiguous bytes of the block: the chunk swizzle permutes chunks within an
// aligned group of eight, and keeps a unit's chunks together.  Loading is
// apart from converting, so that a caller can have several units in flight.
#pragma once

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

// Unit c of block token u; blk is the token's 32-token block.
template <int FMT, bool KPE>
__device__ __forceinline__ void load_unit(const uint8_t* blk, const PageLayout& L, int u, int c, RawUnit<FMT, KPE>& r) {
  using S = UnitShape<FMT, KPE>;
  const uint4* row = reinterpret_cast<const uint4*>(blk + (KPE ? L.kpe_off + u * L.kpe_row : L.codes_off + u * L.codes_row));
#pragma unroll
  for (int i = 0; i < S::kWords; ++i) {
    const int chunk = c * S::kWords + i;
    r.w[i] = __ldg(row + (KPE ? kpe_chunk_pos(chunk, u, FMT) : latent_chunk_pos(chunk, u)));
  }
  if constexpr (S::kScales > 0) {
    const float* sc = reinterpret_cast<const float*>(blk + (KPE ? L.kpe_scale_off : L.scale_off));
    const int g0 = c * kUnitChannels / S::kGroup;
#pragma unroll
    for (int i = 0; i < S::kScales; ++i) r.s[i] = __ldg(sc + (g0 + i) * kBlockTokens + u);
    if constexpr (S::kZeros) {
      const float* zp = reinterpret_cast<const float*>(blk + L.zero_off);
#pragma unroll
      for (int i = 0; i < S::kScales; ++i) r.z[i] = __ldg(zp + (g0 + i) * kBlockTokens + u);
    }
  }
}

// A byte as a float: the byte in the low mantissa bits of 2^23, exact.
__device__ __forceinline__ float byte_float(uint32_t w, int j, float minus) {
  return __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7440 + j)) - minus;
}

// x[0..31] = the unit's dequantized channels in order, x_hat exactly as
// include/mla.h defines it (fp32, one rounding per product).
template <int FMT, bool KPE>
__device__ __forceinline__ void convert_unit(const RawUnit<FMT, KPE>& r, float* x) {
  using S = UnitShape<FMT, KPE>;
  if constexpr (FMT == MLA_FMT_BF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w[4] = {r.w[i].x, r.w[i].y, r.w[i].z, r.w[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[8 * i + 2 * j] = bf16lo(w[j]);
        x[8 * i + 2 * j + 1] = bf16hi(w[j]);
      }
    }
  } else if constexpr (S::kInt4) {
    const uint32_t w[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      // even and odd nibbles as bytes: byte m of lo is nibble 2m, of hi 2m + 1
      const uint32_t lo = w[j] & 0x0F0F0F0Fu, hi = (w[j] >> 4) & 0x0F0F0F0Fu;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int ch = int4_nibble_channel(j, k), g = ch / S::kGroup;
        const float zero = S::kZeros ? r.z[S::kZeros ? g : 0] : 8.f;
        const float q = byte_float((k & 1) ? hi : lo, k >> 1, 8388608.f);
        x[ch] = __fmul_rn(__fsub_rn(q, zero), r.s[g]);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t w[4] = {r.w[i].x ^ 0x80808080u, r.w[i].y ^ 0x80808080u, r.w[i].z ^ 0x80808080u,
                             r.w[i].w ^ 0x80808080u};
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          // 8-channel latent groups store channels 2j, 2j+1, 8+2j, 8+2j+1 in word j
          const int ch = 16 * i + (!KPE && S::kGroup == 8 ? 2 * j + (k & 1) + 8 * (k >> 1) : 4 * j + k);
          x[ch] = __fmul_rn(byte_float(w[j], k, 8388736.f), r.s[S::kScales > 1 ? ch / S::kGroup : 0]);
        }
    }
  }
}

// INT8_OUTLIER: puts the protected channels of unit c in their places.
template <int FMT>
__device__ __forceinline__ void patch_outliers(const uint8_t* blk, const PageLayout& L, const OutlierSet& outl, int u,
                                               int c, float* x) {
  if constexpr (FMT == MLA_FMT_INT8_OUTLIER) {
    const uint32_t mask = outl.mask[c];
    if (!mask) return;
    const uint16_t* ov = reinterpret_cast<const uint16_t*>(blk + L.outlier_off);
    for (int k = 0; k < kNOut; ++k) {
      const int ch = outl.ch[k];
      if ((ch >> 5) != c) continue;
      const float v = bf16f(__ldg(ov + k * kBlockTokens + u));
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (i == (ch & 31)) x[i] = v;
    }
  }
}

}  // namespace mla
