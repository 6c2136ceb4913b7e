// mla_token_mass for sequences of 16 rows: one query of 16 heads, the decode of
// a small model, where the cache's bytes count and the tensor core has little to
// do.  As the tcgen05 kernel's (mass.cuh) A operand a K-step of 16 channels of 128
// keys costs about 75 cycles however few the rows (5400 of its 7000 cycles a
// tile); here keys are the N side of mma.sync m16n8k16, 2.04 cycles for 8 keys.
//
//   S = Q X^T     [16 rows] x [32 keys], group of 16 channels by group:
//   S += s_g[t] (sum_c q_c code_c[t] - z_g[t] sum_c q_c)
// with the codes themselves as exact fp16 operands: a group's scale and zero-point
// enter in fp32, behind the product, for any value they may have.  q is two fp16
// halves (22 bits); bf16 latents take bf16 operands, q in three parts.
//
// What bounds it: the latency of its instructions (890 a warp and 32-token block,
// half the issue slots) and three fifths of the shared-memory pipe, not the cache's
// bytes.  With the seventeenth warp, which issues the copies, one of the SM's four
// schedulers has five, which leaves a thread 96 registers: 4-bit latents, and INT8 with
// a bf16 k_pe, spill 52 to 104 bytes.  The cache comes in bulk copies into a ring; four
// warps share a 32-token block by channels (eight latent groups and 16 RoPE
// channels each), three hand their partial scores to the fourth, in turn, which
// takes the exponentials and adds up the rows.  The queries' fragments lie in
// shared memory, made anew for every sequence.
//
// Measured (a captured call's share of many): 32 x 32768 tokens INT4 207 us, 3.0 TB/s
// or 44% of a plain copy's rate; 32 x 16384 tokens INT8 108 us, bf16 136; one sequence of
// 4096 tokens INT8 11 us.  Eight warps to a block, with their queries' fragments in
// registers: 325 us for the first.
#pragma once

#include <math.h>

#include "mass.cuh"

namespace mla {
namespace {

constexpr int kFewQuads = 4, kFewCompute = 4 * kFewQuads, kFewWarps = kFewCompute + 1, kFewThreads = 32 * kFewWarps;
constexpr int kFewMaxRaw = 10;

template <int LF, int KF>
struct FewShape {
  static constexpr int kBlock = BlockAt<LF, KF>::kBytes;
  static constexpr int kBlocks = kBlock < 20000 ? 2 : 1;             // 32-token blocks of a copy (see MassShape)
  static constexpr int kCopy = kBlocks * kBlock;
  static constexpr int kUnits = kFewQuads / kBlocks;                 // copies in work at a time
  static constexpr int kLatStep = LF == MLA_FMT_BF16 ? 1536 : 1024, kKpeStep = KF == MLA_FMT_BF16 ? 1536 : 1024;      // fragments
  static constexpr int kQ = 32 * kLatStep + 4 * kKpeStep;
  static constexpr int kSums = kQ;                                   // fp32 [32 groups][16 rows]: sums of a group's queries, negated
  static constexpr int kParts = kSums + 32 * 16 * 4;                 // [quad][3][4][32] float4
  static constexpr int kLse = kParts + kFewQuads * 3 * 2048;
  static constexpr int kBars = kLse + 128;                            // and words
  static constexpr int kRaw = (kBars + 256 + 127) / 128 * 128;
  static constexpr int kFit = (232448 - 1024 - kRaw) / kCopy;
  static constexpr int kSlots = kFit < kFewMaxRaw ? kFit : kFewMaxRaw;
  static_assert(kSlots >= kUnits, "every group of four warps has its block");
  static constexpr int kBytes = kRaw + kSlots * kCopy + 1024;
};

__device__ __forceinline__ void mma_half(float* d, const uint4& a, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float* d, const uint4& a, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t lds_word(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];\n" : "=r"(v) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds_pair(uint32_t at) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];\n" : "=r"(v.x), "=r"(v.y) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ void lds_floats8(uint32_t at, float* v) {
  const uint4 a = lds16(at), b = lds16(at + 16);
  v[0] = __uint_as_float(a.x), v[1] = __uint_as_float(a.y), v[2] = __uint_as_float(a.z), v[3] = __uint_as_float(a.w);
  v[4] = __uint_as_float(b.x), v[5] = __uint_as_float(b.y), v[6] = __uint_as_float(b.z), v[7] = __uint_as_float(b.w);
}
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;\n" : "=r"(r) : "f"(b), "f"(a));
  return r;
}

// A 32-bit word of codes of one key, channels 4j .. 4j + 3 of a group, as two
// exact fp16 pairs.  4-bit: the group in the word's low bytes' halves (shift 8: the
// other group).
__device__ __forceinline__ void codes8(uint32_t w, uint32_t& b0, uint32_t& b1) {
  w ^= 0x80808080u;
  const __half2 off = __float2half2_rn(-1152.f);       // 1024 and the codes' bias of 128
  b0 = as_word(__hadd2(as_half2(__byte_perm(w, 0x64646464u, 0x4140)), off));
  b1 = as_word(__hadd2(as_half2(__byte_perm(w, 0x64646464u, 0x4342)), off));
}
template <bool SYM>
__device__ __forceinline__ void codes4(uint32_t w, uint32_t& b0, uint32_t& b1) {
  b0 = as_word(__hadd2(as_half2((w & 0x000F000Fu) | 0x64006400u), __float2half2_rn(SYM ? -1032.f : -1024.f)));
  b1 = as_word(__hfma2(as_half2((w & 0x00F000F0u) | 0x64006400u), __float2half2_rn(0.0625f), __float2half2_rn(SYM ? -72.f : -64.f)));
}

template <int LF, int KF>
__global__ void __launch_bounds__(kFewThreads, 1) mass_few_kernel(const MassParams p) {
  using SH = FewShape<LF, KF>;
  using AT = BlockAt<LF, KF>;
  constexpr bool kInt4 = LF == MLA_FMT_INT4_ASYM || LF == MLA_FMT_INT4_SYM, kKpe4 = KF == MLA_FMT_INT4_SYM;
  constexpr int NS = SH::kSlots;
  extern __shared__ uint8_t few_smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(few_smem_raw) + 1023) & ~(uintptr_t)1023);
  const uint32_t sb = smem_u32(sm), raw_full = sb + SH::kBars, raw_free = raw_full + 8 * kFewMaxRaw;
  volatile int* abort = reinterpret_cast<volatile int*>(sm + SH::kBars + 16 * kFewMaxRaw);
  float2* s_lse = reinterpret_cast<float2*>(sm + SH::kLse);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < NS; ++i) {
      bar_init(raw_full + 8 * i, 1);
      bar_init(raw_free + 8 * i, 4 * SH::kBlocks);     // the warps of its blocks
    }
    *abort = 0;
    bar_init_fence();
  }
  __syncthreads();
  pdl_launch_dependents();
  pdl_wait();
  const int64_t U = __ldcg(&p.counts->units);
  const int G = (int)(U < gridDim.x ? U : gridDim.x), x = blockIdx.x;
  if (x >= G) return;
  MassWalk wk;
  wk.open(p, U, mass_run(U, x, G), mass_run(U, x + 1, G));
  bool ok = true;
  if (warp == kFewCompute) {
    // ---- the cache's blocks, 32 page ids at a time
    int slot = 0;
    uint32_t round = 0;                                // how often the ring went round
    while (ok && wk.left > 0) {
      const int n = (int)min(wk.left, (int64_t)(wk.s.tiles - wk.tile));
      for (int i0 = 0; i0 < n && ok; i0 += 32) {
        const int at = (wk.tile + i0 + lane) * SH::kBlocks / 2;      // the unit's page
        const int mine = i0 + lane < n ? __ldcg(p.table + (int64_t)wk.s.b * p.max_pages + at) : -1;
        for (int i = i0; i < min(n, i0 + 32); ++i) {
          const int page = __shfl_sync(0xffffffffu, mine, i - i0);
          if (round > 0 && !warp_wait(raw_free + 8 * slot, (round - 1) & 1, p.wait_ns, abort)) {
            ok = false;
            break;
          }
          if (lane == 0) {
            if (page >= 0 && page < p.num_pages) {
              bar_expect(raw_full + 8 * slot, SH::kCopy);
              bulk_copy(sb + SH::kRaw + slot * SH::kCopy,
                        p.pool + (int64_t)page * p.L.page_bytes + (SH::kBlocks == 1 ? ((wk.tile + i) & 1) * SH::kBlock : 0), SH::kCopy,
                        raw_full + 8 * slot);
            } else {
              bar_arrive(raw_full + 8 * slot);         // its keys do not count: whatever lies there will do
            }
          }
          __syncwarp();
          if (++slot == NS) {
            slot = 0;
            ++round;
          }
        }
      }
      wk.left -= n;
      if (wk.left > 0) {
        wk.tile = 0;
        ++wk.k;
        wk.load();
      }
    }
    if (!ok) {
      if (lane == 0) set_err(p.dev_err, MLA_DEVERR_TIMEOUT);
      *abort = 1;
    }
    // the copies in flight land before the block ends
    for (int s = 0; s < NS; ++s)
      if (round > 0 || s < slot) drain_wait(raw_full + 8 * s, (s < slot ? round : round - 1) & 1);
    return;
  }
  // ---- Warp w of quad q: channels 128 w .. 128 w + 127 and RoPE channels 16 w ..
  // 16 w + 15 of the quad's blocks.  MMA column n of key tile nt is key 8 (n / 2) +
  // 2 nt + n % 2, so that a thread's scores are those of keys 8 j .. 8 j + 7.
  const int w = warp & 3, q = warp >> 2, n8 = lane >> 2, j = lane & 3;
  int key[4];
#pragma unroll
  for (int nt = 0; nt < 4; ++nt) key[nt] = 8 * (n8 >> 1) + 2 * nt + (n8 & 1);
  int skip = q / SH::kBlocks;                          // units of the segment before this quad's next one
  int slot = q / SH::kBlocks;                          // that unit's place in the ring
  uint32_t round = 0, turn = 0;
  bool late = false;
  float4* parts = reinterpret_cast<float4*>(sm + SH::kParts) + q * 3 * 128;
  const float gain = p.scale_log2 * kQueryGain;
  while (wk.left > 0) {
    const int n = (int)min(wk.left, (int64_t)(wk.s.tiles - wk.tile)), tile0 = wk.tile, b = wk.s.b, len = wk.s.len, counted = wk.s.counted;
    const int64_t row0 = (int64_t)wk.s.q0 * p.H;
    // the old sequence's queries have been read; a warp that gave up a wait says so here
    uint32_t any;
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.or.pred q, 1, %2, p;\n selp.u32 %0, 1, 0, q;\n}\n"
        : "=r"(any)
        : "r"((uint32_t)late), "n"(32 * kFewCompute)
        : "memory");
    if (any) break;
    // ---- the sequence's queries as A fragments: rows n8 and n8 + 8, channels 4 j
    // .. 4 j + 3 of a step of 16
    if (warp == 0 && lane < 16) {
      // -lse log2 e and what its rounding left
      const float lse = __ldcg(p.lse + row0 + lane), v = lse * -1.4426950408889634f;
      const float rest = fmaf(lse, -1.4426950408889634f, -v) - lse * 1.925963033500e-8f;
      s_lse[lane] = fabsf(v) < INFINITY ? make_float2(v, rest) : make_float2(-INFINITY, 0.f);
    }
    const bool live0 = fabsf(__ldcg(p.lse + row0 + n8)) < INFINITY, live1 = fabsf(__ldcg(p.lse + row0 + n8 + 8)) < INFINITY;
    for (int st = warp; st < 36; st += kFewCompute) {
      float a[4], c[4];                                // of the two rows
      if (st < 32) {
        *reinterpret_cast<float4*>(a) = __ldcg(reinterpret_cast<const float4*>(p.q_lat + (row0 + n8) * kDc + 16 * st + 4 * j));
        *reinterpret_cast<float4*>(c) = __ldcg(reinterpret_cast<const float4*>(p.q_lat + (row0 + n8 + 8) * kDc + 16 * st + 4 * j));
      } else {
        const uint2 ra = __ldcg(reinterpret_cast<const uint2*>(p.q_pe + (row0 + n8) * kDr + 16 * (st - 32) + 4 * j));
        const uint2 rc = __ldcg(reinterpret_cast<const uint2*>(p.q_pe + (row0 + n8 + 8) * kDr + 16 * (st - 32) + 4 * j));
        a[0] = bf16lo(ra.x), a[1] = bf16hi(ra.x), a[2] = bf16lo(ra.y), a[3] = bf16hi(ra.y);
        c[0] = bf16lo(rc.x), c[1] = bf16hi(rc.x), c[2] = bf16lo(rc.y), c[3] = bf16hi(rc.y);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a[i] = live0 ? a[i] * gain : 0.f;              // a row without a finite lse adds nothing
        c[i] = live1 ? c[i] * gain : 0.f;
      }
      const bool bf = st < 32 ? LF == MLA_FMT_BF16 : KF == MLA_FMT_BF16;
      uint8_t* at = sm + (st < 32 ? st * SH::kLatStep : 32 * SH::kLatStep + (st - 32) * SH::kKpeStep) + 16 * lane;
      if (bf) {
#pragma unroll
        for (int part = 0; part < 3; ++part) {
          const uint4 f = make_uint4(bf16_pair(a[0], a[1]), bf16_pair(c[0], c[1]), bf16_pair(a[2], a[3]), bf16_pair(c[2], c[3]));
          *reinterpret_cast<uint4*>(at + 512 * part) = f;
          a[0] -= bf16lo(f.x), a[1] -= bf16hi(f.x), c[0] -= bf16lo(f.y), c[1] -= bf16hi(f.y);
          a[2] -= bf16lo(f.z), a[3] -= bf16hi(f.z), c[2] -= bf16lo(f.w), c[3] -= bf16hi(f.w);
        }
      } else {
        if (LF == MLA_FMT_INT4_ASYM && st < 32) {
          float sa = (a[0] + a[1]) + (a[2] + a[3]), sc = (c[0] + c[1]) + (c[2] + c[3]);
#pragma unroll
          for (int o = 1; o <= 2; o <<= 1) {
            sa += __shfl_xor_sync(0xffffffffu, sa, o);
            sc += __shfl_xor_sync(0xffffffffu, sc, o);
          }
          if (j == 0) {
            float* sums = reinterpret_cast<float*>(sm + SH::kSums) + 16 * st;
            sums[n8] = -sa;
            sums[n8 + 8] = -sc;
          }
        }
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float u = (i & 1) ? c[i & 2] : a[i & 2], v = (i & 1) ? c[(i & 2) + 1] : a[(i & 2) + 1];
          const __half2 h = __floats2half2_rn(u, v);
          hi[i] = as_word(h);
          lo[i] = as_word(__floats2half2_rn(u - __low2float(h), v - __high2float(h)));
        }
        *reinterpret_cast<uint4*>(at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4*>(at + 512) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      }
    }
    asm volatile("bar.sync 1, %0;\n" ::"n"(32 * kFewCompute) : "memory");
    const float2 y0 = s_lse[n8], y1 = s_lse[n8 + 8];

    // this quad's units of the segment
    int i = skip;
    for (; i < n; i += SH::kUnits, ++turn) {
      const int at = slot, t0 = ((tile0 + i) * SH::kBlocks + q % SH::kBlocks) * kBlockTokens;
      const uint32_t its_round = round;
      slot += SH::kUnits;
      if (slot >= NS) {
        slot -= NS;
        ++round;
      }
      // a place that is always this quad's needs no look at who had it before (32 x
      // 32768 tokens INT4: 207 us, with it 212)
      if (!late && !(NS % SH::kUnits ? ring_wait(raw_full + 8 * at, raw_free + 8 * at, its_round, p.wait_ns, abort)
                                     : warp_wait(raw_full + 8 * at, its_round & 1, p.wait_ns, abort))) {
        late = true;                                   // leaves with the others, at the next sequence
        *abort = 1;
      }
      if (t0 >= len) {                                 // the page's second half holds nothing
        if (!late) warp_arrive(raw_free + 8 * at);
        continue;
      }
      // the fourth, in turn, has the result: its page and the old masses
      const bool final = (turn & 3) == (uint32_t)w;
      int page = -1;
      float old = 0.f;
      // the key whose sum this lane ends up with (below)
      const int t = t0 + 8 * j + (n8 >> 2) * 4 + ((n8 >> 1) & 1) * 2 + (n8 & 1);
      if (final) {
        page = __ldcg(p.table + (int64_t)b * p.max_pages + t0 / kPage);
        if (page < 0 || page >= p.num_pages) {
          if (lane == 0) set_err(p.dev_err, MLA_DEVERR_PAGE);
          page = -1;
        } else if (t < min(len, counted)) {
          old = __ldcg(p.mass + (int64_t)page * kPage + (t & (kPage - 1)));
        }
      }
      const uint32_t blk = sb + SH::kRaw + at * SH::kCopy + (q % SH::kBlocks) * SH::kBlock;
      float acc[4][4];
#pragma unroll
      for (int nt = 0; nt < 4; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[nt][e] = 0.f;
      uint32_t row[4], flip[4];
#pragma unroll
      for (int nt = 0; nt < 4; ++nt) {
        row[nt] = blk + key[nt] * AT::kRow;
        flip[nt] = (key[nt] & 7) << 4;
      }
#pragma unroll 2
      for (int un = 0; un < 4; ++un) {                 // 32 channels: groups g and g + 1
        const int c = 4 * w + un, g = 2 * c;
        uint32_t word[4];
        if constexpr (kInt4) {
#pragma unroll
          for (int nt = 0; nt < 4; ++nt) word[nt] = lds_word(row[nt] + ((c << 4) ^ flip[nt]) + 4 * j);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t fr = sb + (g + h) * SH::kLatStep + 16 * lane;
          if constexpr (LF == MLA_FMT_BF16) {
            const uint4 a0 = lds16(fr), a1 = lds16(fr + 512), a2 = lds16(fr + 1024);
#pragma unroll
            for (int nt = 0; nt < 4; ++nt) {
              const uint2 v = lds_pair(row[nt] + (((2 * (g + h) + (j >> 1)) << 4) ^ flip[nt]) + 8 * (j & 1));
              mma_bf16(acc[nt], a0, v.x, v.y);
              mma_bf16(acc[nt], a1, v.x, v.y);
              mma_bf16(acc[nt], a2, v.x, v.y);
            }
          } else {
            const uint4 hi = lds16(fr), lo = lds16(fr + 512);
            float s[8];
            lds_floats8(blk + AT::kScale + 128 * (g + h) + 32 * j, s);
            float z[8];
            uint64_t sum0 = 0, sum1 = 0;
            if constexpr (LF == MLA_FMT_INT4_ASYM) {
              lds_floats8(blk + AT::kZero + 128 * (g + h) + 32 * j, z);
              const float u = lds4(sb + SH::kSums + 4 * (16 * (g + h) + n8)), v = lds4(sb + SH::kSums + 4 * (16 * (g + h) + n8 + 8));
              sum0 = pack2(u, u);
              sum1 = pack2(v, v);
            }
#pragma unroll
            for (int nt = 0; nt < 4; ++nt) {
              uint32_t b0, b1;
              if constexpr (kInt4) codes4<LF == MLA_FMT_INT4_SYM>(h ? word[nt] >> 8 : word[nt], b0, b1);
              else codes8(lds_word(row[nt] + (((g + h) << 4) ^ flip[nt]) + 4 * j), b0, b1);
              float d[4] = {0.f, 0.f, 0.f, 0.f};
              if constexpr (LF == MLA_FMT_INT4_ASYM) {
                const uint64_t zz = pack2(z[2 * nt], z[2 * nt + 1]);
                unpack2(mul2(zz, sum0), d[0], d[1]);
                unpack2(mul2(zz, sum1), d[2], d[3]);
              }
              mma_half(d, hi, b0, b1);
              mma_half(d, lo, b0, b1);
              const uint64_t ss = pack2(s[2 * nt], s[2 * nt + 1]);
              unpack2(fma2(ss, pack2(d[0], d[1]), pack2(acc[nt][0], acc[nt][1])), acc[nt][0], acc[nt][1]);
              unpack2(fma2(ss, pack2(d[2], d[3]), pack2(acc[nt][2], acc[nt][3])), acc[nt][2], acc[nt][3]);
            }
          }
        }
      }
      {                                                // RoPE channels 16 w .. 16 w + 15: groups of 8
        const uint32_t fk = sb + 32 * SH::kLatStep + w * SH::kKpeStep + 16 * lane, kpe = blk + AT::kKpe;
        if constexpr (KF == MLA_FMT_BF16) {
          const uint4 a0 = lds16(fk), a1 = lds16(fk + 512), a2 = lds16(fk + 1024);
#pragma unroll
          for (int nt = 0; nt < 4; ++nt) {
            const uint2 v = lds_pair(kpe + key[nt] * AT::kKpeRow + 16 * kpe_chunk_pos(2 * w + (j >> 1), key[nt], KF) + 8 * (j & 1));
            mma_bf16(acc[nt], a0, v.x, v.y);
            mma_bf16(acc[nt], a1, v.x, v.y);
            mma_bf16(acc[nt], a2, v.x, v.y);
          }
        } else {
          const uint4 hi = lds16(fk), lo = lds16(fk + 512);
          float s0[8], s1[8];
          lds_floats8(blk + AT::kKpeScale + 128 * (2 * w) + 32 * j, s0);
          lds_floats8(blk + AT::kKpeScale + 128 * (2 * w + 1) + 32 * j, s1);
#pragma unroll
          for (int nt = 0; nt < 4; ++nt) {
            uint32_t b0, b1;
            if constexpr (kKpe4)
              codes4<true>(lds_word(kpe + key[nt] * AT::kKpeRow + 16 * kpe_chunk_pos(w >> 1, key[nt], KF) + 4 * j) >> (8 * (w & 1)), b0, b1);
            else
              codes8(lds_word(kpe + key[nt] * AT::kKpeRow + 16 * kpe_chunk_pos(w, key[nt], KF) + 4 * j), b0, b1);
            // lanes j < 2 hold the first group's channels: one product with the
            // others' channels 0, one with theirs
            float d0[4] = {0.f, 0.f, 0.f, 0.f}, d1[4] = {0.f, 0.f, 0.f, 0.f};
            const uint32_t f0 = j < 2 ? b0 : 0u, f1 = j < 2 ? b1 : 0u;
            mma_half(d0, hi, f0, f1);
            mma_half(d0, lo, f0, f1);
            mma_half(d1, hi, b0 ^ f0, b1 ^ f1);
            mma_half(d1, lo, b0 ^ f0, b1 ^ f1);
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[nt][e] = fmaf(s1[2 * nt + (e & 1)], d1[e], fmaf(s0[2 * nt + (e & 1)], d0[e], acc[nt][e]));
          }
        }
      }
      // read: the next copy may come (behind a wait given up the last one may be on its way)
      if (!late) warp_arrive(raw_free + 8 * at);
      if (!final) {
        float4* out = parts + ((w - (int)(turn & 3) + 3) & 3) * 128 + lane;
#pragma unroll
        for (int nt = 0; nt < 4; ++nt) out[32 * nt] = make_float4(acc[nt][0], acc[nt][1], acc[nt][2], acc[nt][3]);
      }
      asm volatile("bar.sync %0, 128;\n" ::"r"(2 + q) : "memory");
      if (final) {
#pragma unroll
        for (int other = 0; other < 3; ++other)
#pragma unroll
          for (int nt = 0; nt < 4; ++nt) {
            const float4 v = parts[other * 128 + 32 * nt + lane];
            acc[nt][0] += v.x, acc[nt][1] += v.y, acc[nt][2] += v.z, acc[nt][3] += v.w;
          }
      }
      asm volatile("bar.sync %0, 128;\n" ::"r"(2 + q) : "memory");
      if (!final) continue;
      // the weights of rows n8 and n8 + 8, keys 8 j + i
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float w0 = ex2(fmaf(acc[k >> 1][k & 1], 1.f / kQueryGain, y0.x) + y0.y);
        const float w1 = ex2(fmaf(acc[k >> 1][2 + (k & 1)], 1.f / kQueryGain, y1.x) + y1.y);
        v[k] = (y0.x > -INFINITY ? w0 : 0.f) + (y1.x > -INFINITY ? w1 : 0.f);
      }
      // added up over the eight lanes of a j; each keeps one key: bit 2 of n8 says
      // which half of the eight, bit 1 which pair, bit 0 which of the two
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const bool up = n8 & 4;
        const float give = up ? v[k] : v[k + 4], keep = up ? v[k + 4] : v[k];
        v[k] = keep + __shfl_xor_sync(0xffffffffu, give, 16);
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const bool up = n8 & 2;
        const float give = up ? v[k] : v[k + 2], keep = up ? v[k + 2] : v[k];
        v[k] = keep + __shfl_xor_sync(0xffffffffu, give, 8);
      }
      const bool up = n8 & 1;
      const float give = up ? v[0] : v[1], keep = up ? v[1] : v[0];
      const float sum = keep + __shfl_xor_sync(0xffffffffu, give, 4);
      if (page >= 0 && t < len && !late) p.mass[(int64_t)page * kPage + (t & (kPage - 1))] = fmaf(old, p.decay, sum);
    }
    skip = i - n;
    wk.left -= n;
    if (wk.left > 0) {
      wk.tile = 0;
      ++wk.k;
      wk.load();
    }
  }
  if (late) {
    set_err(p.dev_err, MLA_DEVERR_TIMEOUT);
    *abort = 1;
  }
}

template <int LF, int KF>
mla_status launch_mass_few(const MassParams& p, cudaStream_t stream) {
  static int configured[64] = {0};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !configured[dev]) {
    const mla_status st =
        cuda_status(cudaFuncSetAttribute(mass_few_kernel<LF, KF>, cudaFuncAttributeMaxDynamicSharedMemorySize, FewShape<LF, KF>::kBytes));
    if (st != MLA_OK) return st;
    if (dev >= 0 && dev < 64) configured[dev] = 1;
  }
  return cuda_status(launch_pdl(mass_few_kernel<LF, KF>, dim3(p.grid), dim3(kFewThreads), FewShape<LF, KF>::kBytes, stream, p));
}

template <int LF, int KF>
mla_status launch_mass_pair(const MassParams& p, cudaStream_t stream) {
  if constexpr (LF == MLA_FMT_BF16 || LF == MLA_FMT_INT8_SYM || LF == MLA_FMT_INT4_ASYM || LF == MLA_FMT_INT4_SYM) {
    if (p.few) return launch_mass_few<LF, KF>(p, stream);
  }
  return launch_mass_fmt<LF, KF>(p, stream);
}

}  // namespace
}  // namespace mla
