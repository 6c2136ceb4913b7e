// Chunk attention of sequences with few new tokens (short path): absorbed
// queries against the cached latents, so that every cached byte is read and
// dequantized once for all heads and new tokens of a row tile.
//
//   S^T = C Q^T          [64 keys] x [R rows], contraction over 576 channels
//   P^T = exp2(S^T - m)  (the softmax scale and log2 e are folded into Q)
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
// What bounds it: reading the cache (740 bytes per token for INT8).  The
// chain per tile - dequantize, S^T, softmax, O^T - is pipelined over two key
// buffers: warps 0..3 fill buffer 0, warps 4..7 buffer 1 (each thread keeps
// several 32-channel units in flight, loaded ahead of the buffer's release),
// warps 8..11 do the softmax, and one thread each of warps 12 and 13 issues
// the S^T and the O^T MMAs, so that neither waits for the other's operands.
//
// Work split: all (row tile, key tile) units of the call, in order, are cut
// into equal runs, one per SM, so ragged lengths need no care.  A row tile
// that falls into several runs leaves fp32 partials, merged by
// short_combine_kernel in block order (no atomics: results repeat bit for
// bit).
//
// Rounding: keys, queries and P enter the MMAs as fp16 (2^-11 relative);
// scores, sums, maxima and O stay fp32 until o_lat is written as fp16.
#include <math.h>

#include "chunk.cuh"
#include "dequant.cuh"
#include "tc.cuh"

namespace mla {
namespace {

using namespace tc;

constexpr int kSThreads = 14 * 32;
constexpr int kKeyBlk = kKeyTile * 128;              // one 64-key x 64-channel fp16 block: 8 KB
constexpr int kKeyBuf = kQBlocks * kKeyBlk;          // 72 KB
constexpr float kSlack = 8.f;                        // the running maximum rises only past this (P <= 2^8 in fp16)

template <int R>
struct ShortSmem {
  static constexpr int kQ = 2 * kKeyBuf;
  static constexpr int kP = kQ + kQBlocks * R * 128;
  static constexpr int kRed = kP + R * 128;          // [4 warps][R] maxima, then sums
  static constexpr int kBars = kRed + 4 * R * 4;
  static constexpr int kBytes = kBars + 192 + 1024;  // barriers and words; alignment slack
};
static_assert(ShortSmem<64>::kBytes <= 232448, "a block's shared memory");

enum { bFull0 = 0, bFull1, bP0, bP1, bFree0, bFree1, bS0, bS1, bQ, bFinS, bFinO, bCount };

// One run's walk over the units: segments (a row tile, key tiles t0 .. t1).
struct Walk {
  const ShortSeq* seqs;
  int n_seqs, k;
  int64_t u, hi;
  ShortSeq s;
  int item, t0, t1;
  bool first, last;         // the segment holds the row tile's first / last key tile

  __device__ __forceinline__ void load() {
    const int4* r = reinterpret_cast<const int4*>(seqs + k);
    int4* d = reinterpret_cast<int4*>(&s);
    d[0] = __ldcg(r);
    d[1] = __ldcg(r + 1);
    d[2] = __ldcg(r + 2);
  }
  // All lanes of a warp: the sequence of unit u, 32 probes per round.
  __device__ __forceinline__ void start(const ChunkParams& p, int64_t lo, int64_t hi_) {
    seqs = p.s_seqs;
    u = lo;
    hi = hi_;
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
    k = a;
    load();
  }
  // The next segment; false behind the run's end.
  __device__ __forceinline__ bool next() {
    if (u >= hi) return false;
    while (u >= s.unit0 + (int64_t)s.items * s.tiles) {
      ++k;
      load();
    }
    const int64_t d = u - s.unit0;
    item = (int)(d / s.tiles);
    t0 = (int)(d % s.tiles);
    t1 = (int)min((int64_t)s.tiles, t0 + (hi - u));
    first = t0 == 0;
    last = t1 == s.tiles;
    u += t1 - t0;
    return true;
  }
};

// ---- producers: dequantize a key tile into fp16 blocks
// Warp w of a group takes the tile's tokens 16 w .. 16 w + 15.  Latent steps
// 0..7: eight tokens x four units, lane = token + 8 unit, so that a quarter
// warp's 16-byte stores hit eight different swizzled positions, and a scale
// load covers whole 32-byte sectors.  The last step: k_pe, sixteen tokens x
// two units.
template <int LF, int KF>
struct Producer {
  static constexpr int kAhead = LF == MLA_FMT_BF16 ? 2 : 4;      // latent steps in flight
  static __device__ __forceinline__ int token(int w, int lane, int step) {
    return step < 8 ? 16 * w + 8 * (step >> 2) + (lane & 7) : 16 * w + (lane & 15);
  }
  static __device__ __forceinline__ int unit(int lane, int step) { return step < 8 ? 4 * (step & 3) + (lane >> 3) : lane >> 4; }
};

// A unit's 32 fp16 channels into their block, swizzled.
__device__ __forceinline__ void put_unit(const uint32_t* h, uint32_t buf, int tok, int unit) {
  const uint32_t row = buf + (unit >> 1) * kKeyBlk + tok * 128, flip = (4 * (unit & 1) ^ (tok & 7)) << 4;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};\n" ::"r"(row + (flip ^ (i << 4))), "r"(h[4 * i]),
                 "r"(h[4 * i + 1]), "r"(h[4 * i + 2]), "r"(h[4 * i + 3])
                 : "memory");
}

template <int LF, int KF, int R>
__global__ void __launch_bounds__(kSThreads, 1) short_attention_kernel(const ChunkParams p) {
  using SM = ShortSmem<R>;
  using PR = Producer<LF, KF>;
  extern __shared__ uint8_t short_smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(short_smem_raw) + 1023) & ~(uintptr_t)1023);
  const uint32_t sb = smem_u32(sm), bars = sb + SM::kBars;
  uint8_t* words = sm + SM::kBars + 8 * bCount;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(words);
  volatile int* abort = reinterpret_cast<volatile int*>(words + 4);
  volatile int* tile_ok = reinterpret_cast<volatile int*>(words + 8);        // [2 buffers]
  uint32_t* bad = reinterpret_cast<uint32_t*>(words + 16);                   // [2 buffers][2]: a bit per token
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kCols = R == 64 ? 512 : 8 * R;       // 6 R columns used, a power of two allocated

  if (threadIdx.x == 0) {
    for (int i = 0; i < bCount; ++i) bar_init(bars + 8 * i, i <= bP1 ? 128 : 1);
    *abort = 0;
    for (int i = 0; i < 4; ++i) bad[i] = 0;
    bar_init_fence();
  }
  if (warp == 12) tmem_alloc(smem_u32(tmem_slot), kCols);
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
  const int64_t lo = work ? U * x / G : 0, hi = work ? U * (x + 1) / G : 0;
  Walk wk;
  wk.n_seqs = __ldcg(&p.counts->s_seqs);
  bool ok = true;
  if (work && warp < 8) {
    // ---- producers
    wk.start(p, lo, hi);
    const int g = warp >> 2, w = warp & 3;
    const uint32_t buf = sb + g * kKeyBuf;
    uint32_t* mybad = bad + 2 * g;
    // This group's tiles, every second of the run, are visited one ahead of
    // the loads: `next` holds the tile whose page id is under way.
    struct Tile {
      int page, pos, len;
    } next = {-1, 0, 0};
    int t = 0, seg_t1 = 0, skip = g;
    const int32_t* pages = nullptr;
    auto advance = [&]() -> bool {           // next = the group's next tile; false at the end
      t += skip;
      while (t >= seg_t1) {
        const int over = t - seg_t1;
        if (!wk.next()) return false;
        seg_t1 = wk.t1;
        t = wk.t0 + over;
        next.len = wk.s.len;
        pages = p.block_table + (int64_t)wk.s.b * p.max_pages;
      }
      skip = 2;
      next.pos = t * kKeyTile;
      next.page = __ldg(pages + t);
      return true;
    };
    RawUnit<LF, false> ring[PR::kAhead];
    RawUnit<KF, true> kpe;
    const uint8_t* page = nullptr;           // the loading tile; tokens from t_len on read as 0
    int t_len = 0;
    bool page_ok = false, more = advance(), after = false;
    auto enter = [&]() {                     // `next` becomes the loading tile
      page_ok = next.page >= 0 && next.page < p.num_pages;
      page = p.pool + (int64_t)(page_ok ? next.page : 0) * p.L.page_bytes;
      t_len = page_ok ? next.len - next.pos : 0;
      if (!page_ok && (threadIdx.x & 127) == 0) set_err(p.dev_err, MLA_DEVERR_PAGE);
      after = advance();
    };
    auto load_step = [&](int step, RawUnit<LF, false>& r) {
      const int tok = PR::token(w, lane, step);
      if (tok < t_len) load_unit<LF, false>(page + (tok >> 5) * p.L.block_bytes, p.L, tok & 31, PR::unit(lane, step), r);
    };
    if (more) {
      enter();
#pragma unroll
      for (int i = 0; i < PR::kAhead; ++i) load_step(i, ring[i]);
    }
    uint32_t n = 0;                          // the group's tiles so far
    while (more) {
      // the tile being stored, while page / t_len move on to the next
      const uint8_t* s_page = page;
      const int s_len = t_len;
      const bool s_ok = page_ok;
      {
        const int tok = PR::token(w, lane, 8);
        if (tok < s_len)
          load_unit<KF, true>(s_page + (tok >> 5) * p.L.block_bytes, p.L, tok & 31, PR::unit(lane, 8), kpe);
      }
      if (n >= 1 && !bar_wait(bars + 8 * (bFree0 + g), (n - 1) & 1, p.wait_ns, abort)) {
        ok = false;
        break;
      }
      uint32_t bad_lo = 0, bad_hi = 0;
      const bool go_on = after;
#pragma unroll
      for (int step = 0; step < 8; ++step) {
        const int tok = PR::token(w, lane, step), unit = PR::unit(lane, step);
        uint32_t h[16];
        bool fine = true;
        if (tok < s_len) {
          fine = convert_unit<LF, false>(ring[step % PR::kAhead], h);
          fine &= patch_outliers<LF>(s_page + (tok >> 5) * p.L.block_bytes, p.L, p.outl, tok & 31, unit, h);
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) h[i] = 0u;
        }
        if (step + PR::kAhead < 8) {
          load_step(step + PR::kAhead, ring[step % PR::kAhead]);
        } else {
          if (step + PR::kAhead == 8 && go_on) enter();
          if (go_on) load_step(step + PR::kAhead - 8, ring[step % PR::kAhead]);
        }
        put_unit(h, buf, tok, unit);
        if (!fine) (tok < 32 ? bad_lo : bad_hi) |= 1u << (tok & 31);
      }
      {
        const int tok = PR::token(w, lane, 8), unit = PR::unit(lane, 8);
        uint32_t h[16];
        bool fine = true;
        if (tok < s_len) {
          fine = convert_unit<KF, true>(kpe, h);
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) h[i] = 0u;
        }
        put_unit(h, buf, tok, kLatentUnits + unit);
        if (!fine) (tok < 32 ? bad_lo : bad_hi) |= 1u << (tok & 31);
      }
      if (bad_lo) atomicOr(mybad, bad_lo);
      if (bad_hi) atomicOr(mybad + 1, bad_hi);
      if ((threadIdx.x & 127) == 0) tile_ok[g] = s_ok;
      fence_async_smem();
      bar_arrive(bars + 8 * (bFull0 + g));
      ++n;
      more = go_on;
    }
  } else if (work && warp < 12) {
    // ---- softmax.  Thread (w, lane) holds keys 16 w + lane / 4 and + 8 of
    // the tile, rows 8 j + 2 (lane % 4) and the next (j < R / 8).
    wk.start(p, lo, hi);
    const int w = warp & 3;
    const uint32_t tl = (uint32_t)(32 * w) << 16;
    constexpr int J = R / 8;
    float* red = reinterpret_cast<float*>(sm + SM::kRed);
    uint32_t it = 0;
    while (ok && wk.next()) {
      const int row0 = wk.item * R, rows = min(R, wk.s.n * p.H - row0);
      const int ctx = wk.s.len - wk.s.n;
      const int pos_min = ctx + row0 / p.H;          // the earliest row's position
      float m[2 * J], l[2 * J];
#pragma unroll
      for (int i = 0; i < 2 * J; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
      }
      for (int t = wk.t0; t < wk.t1; ++t, ++it) {
        const uint32_t g = it & 1;
        if (!warp_wait(bars + 8 * (bS0 + g), (it >> 1) & 1, p.wait_ns, abort)) {
          ok = false;
          break;
        }
        fence_after();
        float v[4 * J];
        {
          uint32_t r[4 * J];
          tmem_load_16x256b<J>(t_s + g * R + tl, r);
#pragma unroll
          for (int i = 0; i < 4 * J; ++i) v[i] = __uint_as_float(r[i]);
        }
        const bool page_ok = tile_ok[g] != 0;
        const uint32_t bad_lo = *(volatile uint32_t*)(bad + 2 * g), bad_hi = *(volatile uint32_t*)(bad + 2 * g + 1);
        if (!page_ok || t * kKeyTile + kKeyTile - 1 > pos_min || (bad_lo | bad_hi)) {
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
        float mx[2 * J];
#pragma unroll
        for (int i = 0; i < 2 * J; ++i) {
          float a = fmaxf(v[4 * (i >> 1) + (i & 1)], v[4 * (i >> 1) + 2 + (i & 1)]);
          a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 4));
          a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 8));
          mx[i] = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 16));
        }
        if (lane < 4) {
#pragma unroll
          for (int j = 0; j < J; ++j)
            *reinterpret_cast<float2*>(red + w * R + 8 * j + 2 * lane) = make_float2(mx[2 * j], mx[2 * j + 1]);
        }
        asm volatile("bar.sync 1, 128;\n" ::: "memory");
        if ((bad_lo | bad_hi) && threadIdx.x == 8 * 32) bad[2 * g] = bad[2 * g + 1] = 0;    // all four warps have read them
        bool any = false;
        float alpha[2 * J];
#pragma unroll
        for (int j = 0; j < J; ++j) {
          float2 a = make_float2(-INFINITY, -INFINITY);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float2 b = *reinterpret_cast<const float2*>(red + q * R + 8 * j + 2 * (lane & 3));
            a.x = fmaxf(a.x, b.x);
            a.y = fmaxf(a.y, b.y);
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int i = 2 * j + e;
            const float top = e ? a.y : a.x;
            const bool raise = top > m[i] + kSlack || (m[i] == -INFINITY && top > -INFINITY);
            alpha[i] = raise ? ex2(m[i] - top) : 1.f;
            if (raise) m[i] = top;
            any |= raise;
          }
        }
        any = __any_sync(0xffffffffu, any);
        // the O^T of the tile before is complete: P is free, and O^T may be rescaled
        if (it >= 1 && !warp_wait(bars + 8 * (bFree0 + (g ^ 1)), ((it - 1) >> 1) & 1, p.wait_ns, abort)) {
          ok = false;
          break;
        }
        if (any) {
#pragma unroll
          for (int i = 0; i < 2 * J; ++i) l[i] *= alpha[i];
          if (t > wk.t0) {
            fence_after();
#pragma unroll
            for (int c0 = 0; c0 < R; c0 += 16) {
              float al[16];
#pragma unroll
              for (int c = 0; c < 16; ++c)
                al[c] = __shfl_sync(0xffffffffu, alpha[2 * ((c0 + c) >> 3) + (c & 1)], (c & 7) >> 1);
#pragma unroll 1
              for (int blk = 0; blk < 4; ++blk) {
                uint32_t r[16];
                tmem_load16(tbase + blk * R + c0 + tl, r);
#pragma unroll
                for (int c = 0; c < 16; ++c) r[c] = __float_as_uint(__uint_as_float(r[c]) * al[c]);
                tmem_store16(tbase + blk * R + c0 + tl, r);
              }
            }
          }
        }
        uint32_t h[2 * J];
#pragma unroll
        for (int j = 0; j < J; ++j) {
          // a row that has seen nothing yet keeps m = -inf: its weights are 0
          const float m0 = m[2 * j] == -INFINITY ? 0.f : m[2 * j], m1 = m[2 * j + 1] == -INFINITY ? 0.f : m[2 * j + 1];
          const float p0 = ex2(v[4 * j] - m0), p1 = ex2(v[4 * j + 1] - m1);
          const float p2 = ex2(v[4 * j + 2] - m0), p3 = ex2(v[4 * j + 3] - m1);
          l[2 * j] += p0 + p2;
          l[2 * j + 1] += p1 + p3;
          h[2 * j] = half2_bits(p0, p1);
          h[2 * j + 1] = half2_bits(p2, p3);
        }
        // P^T as rows of 64 keys: the fragment transposed
#pragma unroll
        for (int j = 0; j < J; j += 2) {
          const int mat = lane >> 3, rr = 8 * (j + (mat >> 1)) + (lane & 7), oct = 2 * w + (mat & 1);
          stmatrix_x4_trans(sb + SM::kP + rr * 128 + ((oct ^ (rr & 7)) << 4), h[2 * j], h[2 * j + 1], h[2 * j + 2],
                            h[2 * j + 3]);
        }
        fence_async_smem();
        fence_before();
        bar_arrive(bars + 8 * (bP0 + g));
      }
      if (!ok) break;
      // ---- the segment's end: sums over all keys, then O^T
#pragma unroll
      for (int i = 0; i < 2 * J; ++i) {
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], 4);
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], 8);
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], 16);
      }
      asm volatile("bar.sync 1, 128;\n" ::: "memory");         // the last maxima have been read
      if (lane < 4) {
#pragma unroll
        for (int j = 0; j < J; ++j)
          *reinterpret_cast<float2*>(red + w * R + 8 * j + 2 * lane) = make_float2(l[2 * j], l[2 * j + 1]);
      }
      asm volatile("bar.sync 1, 128;\n" ::: "memory");
#pragma unroll
      for (int j = 0; j < J; ++j) {
        float2 a = make_float2(0.f, 0.f);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float2 b = *reinterpret_cast<const float2*>(red + q * R + 8 * j + 2 * (lane & 3));
          a.x += b.x;
          a.y += b.y;
        }
        l[2 * j] = a.x;
        l[2 * j + 1] = a.y;
      }
      if (!warp_wait(bars + 8 * (bFree0 + ((it - 1) & 1)), ((it - 1) >> 1) & 1, p.wait_ns, abort)) {
        ok = false;
        break;
      }
      fence_after();
      const bool whole = wk.first && wk.last;
      const int slot = 2 * x + (wk.first ? 1 : 0);
      float* part = p.parts + (int64_t)slot * partial_floats(R);
      const int64_t out0 = (int64_t)wk.s.tok0 * p.H + row0;
#pragma unroll
      for (int c0 = 0; c0 < R; c0 += 16) {
        float inv[16];
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          const float sum = __shfl_sync(0xffffffffu, l[2 * ((c0 + c) >> 3) + (c & 1)], (c & 7) >> 1);
          inv[c] = sum == 0.f ? 0.f : 1.f / sum;       // nothing seen: 0 (a NaN sum stays NaN)
        }
#pragma unroll 1
        for (int blk = 0; blk < 4; ++blk) {
          uint32_t r[16];
          tmem_load16(tbase + blk * R + c0 + tl, r);
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
#pragma unroll
        for (int i = 0; i < 2 * J; ++i) {
          const int c = 8 * (i >> 1) + 2 * lane + (i & 1);
          part[R * kDc + c] = m[i];
          part[R * kDc + R + c] = l[i];
        }
      }
      if (wk.first && !wk.last && w == 0 && lane == 0) {
        // the row tile goes on in the blocks behind: up to the one that holds its last unit
        const int64_t end = wk.s.unit0 + (int64_t)(wk.item + 1) * wk.s.tiles;
        int y = x + 1;
        while (U * (y + 1) / G < end) ++y;
        SplitRec rec;
        rec.rows = rows;
        rec.last = y;
        rec.row0 = out0;
        p.splits[x] = rec;
      }
      fence_before();                                  // O^T has been read: ordered before the next P's arrival
    }
    if (!ok) {
      set_err(p.dev_err, MLA_DEVERR_TIMEOUT);
      *abort = 1;
    }
  } else if (work && warp == 12) {
    // ---- one thread: the query tiles' copies and the S^T MMAs
    wk.start(p, lo, hi);
    if (lane == 0) {
      constexpr uint32_t kId = f16_idesc(64, R, false, false);
      constexpr int kQBytes = kQBlocks * R * 128;
      const uint64_t d_q = sw128_desc(sb + SM::kQ, 16, 1024), d_k = sw128_desc(sb, 16, 1024);
      uint32_t it = 0, seg = 0;
      while (ok && wk.next()) {
        // the query tile: its readers, the S^T MMAs of the segment before, are done
        if (seg > 0 && !bar_wait(bars + 8 * (bS0 + ((it - 1) & 1)), ((it - 1) >> 1) & 1, p.wait_ns, abort)) {
          ok = false;
          break;
        }
        bar_expect(bars + 8 * bQ, kQBytes);
        bulk_copy(sb + SM::kQ, p.q_tiles + (int64_t)(wk.s.item0 + wk.item) * kQBytes, kQBytes, bars + 8 * bQ);
        ++seg;
        if (!bar_wait(bars + 8 * bQ, (seg - 1) & 1, p.wait_ns, abort)) {
          ok = false;
          break;
        }
        for (int t = wk.t0; t < wk.t1; ++t, ++it) {
          const uint32_t g = it & 1;
          // the keys are there, and the softmax has read this S^T buffer's last tile
          if (!bar_wait(bars + 8 * (bFull0 + g), (it >> 1) & 1, p.wait_ns, abort) ||
              (it >= 2 && !bar_wait(bars + 8 * (bP0 + g), ((it - 2) >> 1) & 1, p.wait_ns, abort))) {
            ok = false;
            break;
          }
          fence_after();
          const uint64_t a = d_k + (uint64_t)(g * (kKeyBuf >> 4));
#pragma unroll
          for (int kb = 0; kb < kQBlocks; ++kb)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              umma(t_s + g * R, a + ((kb * kKeyBlk + 32 * k) >> 4), d_q + ((kb * R * 128 + 32 * k) >> 4), kId, (kb | k) != 0);
          umma_commit(bars + 8 * (bS0 + g));
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
  } else if (work) {
    // ---- warp 13, one thread: the O^T MMAs
    wk.start(p, lo, hi);
    if (lane == 0) {
      constexpr uint32_t kId = f16_idesc(128, R, true, false);
      const uint64_t d_p = sw128_desc(sb + SM::kP, 16, 1024), d_v = sw128_desc(sb, kKeyBlk, 1024);
      uint32_t it = 0;
      while (ok && wk.next()) {
        for (int t = wk.t0; t < wk.t1; ++t, ++it) {
          const uint32_t g = it & 1;
          if (!bar_wait(bars + 8 * (bP0 + g), (it >> 1) & 1, p.wait_ns, abort)) {
            ok = false;
            break;
          }
          fence_after();
          const uint64_t a = d_v + (uint64_t)(g * (kKeyBuf >> 4));
#pragma unroll
          for (int blk = 0; blk < 4; ++blk)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              umma(tbase + blk * R, a + ((2 * blk * kKeyBlk + 2048 * k) >> 4), d_p + ((32 * k) >> 4), kId, t > wk.t0 || k != 0);
          umma_commit(bars + 8 * (bFree0 + g));
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
  }
  if (warp < 8 && !ok) {
    set_err(p.dev_err, MLA_DEVERR_TIMEOUT);
    *abort = 1;
  }
  fence_before();
  __syncthreads();
  if (warp == 12) {
    fence_after();
    tmem_free(tbase, kCols);
  }
}

// short_combine_kernel: grid (blocks of the attention, R), block 128.  Row y
// of the row tile whose first part block x holds: parts x (slot 2x + 1) and
// x + 1 .. last (slots 2 (x + i)), merged with the running maxima's weights.
__global__ void __launch_bounds__(128) short_combine_kernel(const ChunkParams p, int R) {
  pdl_launch_dependents();
  pdl_wait();
  const int x = blockIdx.x, c = blockIdx.y, tid = threadIdx.x;
  const SplitRec rec = p.splits[x];
  if (c >= rec.rows) return;
  const int64_t stride = 2 * partial_floats(R);
  const float* part = p.parts + (int64_t)(2 * x + 1) * partial_floats(R);
  const int n = rec.last - x + 1;
  // part 0 is slot 2x + 1, part i > 0 slot 2 (x + i): one slot before the regular stride
  auto at = [&](int i) { return part + i * stride - (i ? partial_floats(R) : 0); };
  float mx = -INFINITY;
  for (int i = 0; i < n; ++i) mx = fmaxf(mx, at(i)[R * kDc + c]);
  if (mx == -INFINITY) mx = 0.f;
  float l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int i = 0; i < n; ++i) {
    const float* s = at(i);
    const float wt = tc::ex2(s[R * kDc + c] - mx);
    const float4 v = reinterpret_cast<const float4*>(s + (int64_t)c * kDc)[tid];
    l = fmaf(wt, s[R * kDc + R + c], l);
    acc.x = fmaf(wt, v.x, acc.x);
    acc.y = fmaf(wt, v.y, acc.y);
    acc.z = fmaf(wt, v.z, acc.z);
    acc.w = fmaf(wt, v.w, acc.w);
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  reinterpret_cast<uint2*>(p.o_lat + (rec.row0 + c) * kDc)[tid] =
      make_uint2(tc::half2_bits(acc.x * inv, acc.y * inv), tc::half2_bits(acc.z * inv, acc.w * inv));
}

template <int LF, int KF, int R>
mla_status launch_r(const ChunkParams& p, cudaStream_t stream) {
  static int configured[64] = {0};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !configured[dev]) {
    const mla_status st = cuda_status(cudaFuncSetAttribute(
        short_attention_kernel<LF, KF, R>, cudaFuncAttributeMaxDynamicSharedMemorySize, ShortSmem<R>::kBytes));
    if (st != MLA_OK) return st;
    if (dev >= 0 && dev < 64) configured[dev] = 1;
  }
  const mla_status st = cuda_status(launch_pdl(short_attention_kernel<LF, KF, R>, dim3(p.grid), dim3(kSThreads),
                                               ShortSmem<R>::kBytes, stream, p));
  if (st != MLA_OK) return st;
  return cuda_status(launch_pdl(short_combine_kernel, dim3(p.grid, R), dim3(128), 0, stream, p, R));
}

template <int LF, int KF>
mla_status launch_fmt(const ChunkParams& p, int R, cudaStream_t stream) {
  return R == 16 ? launch_r<LF, KF, 16>(p, stream) : (R == 32 ? launch_r<LF, KF, 32>(p, stream) : launch_r<LF, KF, 64>(p, stream));
}

}  // namespace

mla_status launch_short_attention(const ChunkParams& p, int lf, int kf, int R, cudaStream_t stream) {
#define MLA_CHUNK_CASE(A, K) \
  if (lf == A && kf == K) return launch_fmt<A, K>(p, R, stream);
  MLA_CHUNK_FORMATS(MLA_CHUNK_CASE)
#undef MLA_CHUNK_CASE
  return MLA_ERR_UNSUPPORTED;
}

}  // namespace mla
