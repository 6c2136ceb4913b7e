// mla_chunk_attention: causal attention of a ragged batch of new tokens over
// the paged latent cache, from the projected queries to the per-head outputs.
//
//   s[i,h,t] = (q_nope[i,h] . (W_UK[h] c_hat[t]) + q_pe[i,h] . kpe_hat[t]) scale
//   o[i,h]   = sum_t softmax(s[i,h])[t] c_hat[t] W_UV[h]
//
// Bracketed two ways.  Absorbed, (q_nope W_UK) . c and (sum_t w c) W_UV: 2 x
// 1088 operations per (query, head, key), and every cached byte serves all
// heads.  Expanded, with keys c W_UK^T and values c W_UV made once per head:
// 2 x 320 operations per (query, head, key), plus 2 x 512 x 256 per (key,
// head).  Sequences with at most MLA_CHUNK_SHORT = 64 new tokens take the
// first (chunk_short.cuh), the others the second (chunk_long.cu).  The rule
// looks at the new tokens alone, which the host bounds.  The absorbed form's
// time grows with them, the expanded form's is flat up to 256 (one item per
// head); where the two meet depends on the context too.  Absorbed / expanded,
// microseconds of a captured call, INT8 (bf16 and INT4 at 64 heads are within 8 %):
//                                  n = 16        32         48         64         96
//   16 heads, 16 x   500 cached    72/99      98/100    128/100    149/101    217/104
//             16 x  4000          122/381    211/382    296/383    372/383    529/386
//   64 heads,  1 x   200           58/43      40/43      49/43      58/48      65/48
//             16 x   500          146/252    249/257    348/259    453/262    697/268
//             16 x  4000          360/1218   662/1224   980/1227  1288/1230  1901/1236
//              1 x 30000          176/580    271/582    395/584    515/585    757/592
//  128 heads, 16 x   500          251/448    452/457    649/461    845/467   1329/480
//              1 x 30000          274/1093   516/1094   756/1099   993/1099  1470/1122
// So they meet at about 64 new tokens after thousands of cached ones and at 32
// after a few hundred, where 33 to 64 new tokens cost up to 1.8 times what the
// expanded form would.  That form also needs 512 bytes of workspace per token
// and head, within a bound that the host has to give for such sequences.
//
// This file: the device plan (which sequences take which path, prefix sums
// of their work; lengths never visit the host), the query absorption, the
// output projection and the host side.
#include <cuda_bf16.h>
#include <math.h>

#include "chunk.cuh"
#include "tc.cuh"

namespace mla {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanPer = kMaxBatch / kPlanThreads;      // sequences per thread: 4
constexpr int kPlanFused = 128;                         // most sequences the absorption plans itself: a thread each

// Exclusive block scan of one int64 per thread.
__device__ __forceinline__ int64_t scan(int64_t v, int64_t* red, int64_t* total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int64_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) red[warp] = x;
  __syncthreads();
  int64_t s = lane < (int)(blockDim.x >> 5) ? red[lane] : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += y;
  }
  *total = __shfl_sync(0xffffffffu, s, 31);
  const int64_t base = __shfl_sync(0xffffffffu, s, warp > 0 ? warp - 1 : 0);
  return (warp ? base : 0) + x - v;
}

// Checks every sequence, sorts it to a path, and makes the path's records with
// the prefix sums of rows and work units.  Up to PER sequences per thread of the
// block.  Returns the short path's number of tokens; note(record, first token
// row, its short-path tokens and row tiles before it) is called for each of its
// sequences by some thread.  One block of a grid has write set: it also writes
// the records and counts, reports what does not fit, and zeroes the rows of
// sequences that are empty or refused.
template <int PER, class Note>
__device__ __forceinline__ int plan_sequences(const ChunkParams& p, int R, bool write, int64_t* red, uint32_t* zero_mask,
                                              Note note) {
  const int tid = threadIdx.x;
  const bool long_path = PER > 1 && p.l_seqs != nullptr;
  if (write)
    for (int i = tid; i < kMaxBatch / 32; i += blockDim.x) zero_mask[i] = 0;
  const int per = PER == 1 ? 1 : (p.B + blockDim.x - 1) / blockDim.x, b0 = tid * per;
  int q0[PER], n[PER], len[PER];
  bool order = true;
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    const int b = b0 + k;
    q0[k] = n[k] = len[k] = 0;
    if (k < per && b < p.B) {
      q0[k] = __ldcg(p.q_start + b);
      const int q1 = __ldcg(p.q_start + b + 1);
      len[k] = __ldcg(p.seq_lens + b);
      order &= q0[k] >= 0 && q1 >= q0[k] && q1 <= p.N;
      n[k] = q1 - q0[k];
    }
  }
  // rows out of order could overlap: then nobody is served
  const bool ordered = !__syncthreads_or(!order);
  int64_t mine = 0, units = 0, l_mine = 0;
  bool bad = !ordered, zero = false;
  int items[PER], tiles[PER];
  bool is_long[PER];
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    const int b = b0 + k;
    items[k] = tiles[k] = 0;
    is_long[k] = false;
    if (!(k < per && b < p.B) || (ordered && n[k] == 0)) continue;
    const bool fits = ordered && n[k] <= p.max_new && len[k] >= 0 && (len[k] == 0 || len[k] >= n[k]) &&
                      (int64_t)len[k] <= (int64_t)p.max_pages * kPage && (n[k] <= kChunkShort || len[k] == 0 || long_path);
    if (!fits || len[k] == 0) {
      bad |= !fits;
      zero = true;
      atomicOr(zero_mask + (b >> 5), 1u << (b & 31));
      continue;
    }
    if (n[k] > kChunkShort) {
      is_long[k] = true;
      tiles[k] = (len[k] - 1) / kLongKeys + 1;         // len + 127 may pass 31 bits
      l_mine += ((int64_t)1 << 48) + tiles[k];
      continue;
    }
    items[k] = (n[k] * p.H + R - 1) / R;
    tiles[k] = (len[k] + kKeyTile - 1) / kKeyTile;
    // at most 2^12 sequences, 2^18 tokens and 2^22 row tiles: one word
    mine += ((int64_t)1 << 48) + ((int64_t)items[k] << 20) + n[k];
    units += (int64_t)items[k] * (tiles[k] + kItemCost);
  }
  int64_t total, total_units = 0, unit = 0;
  int64_t at = scan(mine, red, &total);
  if (write) unit = scan(units, red, &total_units);
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    if (items[k] == 0) continue;
    note((int)(at >> 48), q0[k], (int)(at & 0xFFFFF), (int)((at >> 20) & 0xFFFFFFF));
    if (!write) continue;
    ShortSeq s;
    s.unit0 = unit;
    s.b = b0 + k;
    s.q0 = q0[k];
    s.n = n[k];
    s.len = len[k];
    s.item0 = (int)((at >> 20) & 0xFFFFFFF);
    s.tok0 = (int)(at & 0xFFFFF);
    s.tiles = tiles[k];
    s.items = items[k];
    p.s_seqs[at >> 48] = s;
    for (int i = 0; i < n[k]; ++i) p.s_toks[s.tok0 + i] = make_int2(q0[k] + i, s.item0 * R + i * p.H);
    at += ((int64_t)1 << 48) + ((int64_t)items[k] << 20) + n[k];
    unit += (int64_t)items[k] * (tiles[k] + kItemCost);
  }
  if (!write) return (int)(total & 0xFFFFF);
  ChunkCounts c = {};
  c.s_seqs = (int)(total >> 48);
  c.s_items = (int)((total >> 20) & 0xFFFFFFF);
  c.s_toks = (int)(total & 0xFFFFF);
  c.s_units = total_units;
  if (long_path) {
    // key tiles in the order of the batch, as far as the caller's bound goes:
    // with the refused ones' counted, nobody behind the first refusal fits
    int64_t l_total, l_units = 0;
    int64_t l_at = scan(l_mine, red, &l_total);
    const int64_t room = p.kv_tokens / kLongKeys;
    int64_t kv = l_at & 0xFFFFFFFFFFFF;
    int per_head[PER];
    int served = 0, served_tiles = 0;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      per_head[k] = 0;
      if (!is_long[k]) continue;
      if (kv + tiles[k] > room) {
        is_long[k] = false;
        bad = zero = true;
        atomicOr(zero_mask + ((b0 + k) >> 5), 1u << ((b0 + k) & 31));
      } else {
        for (int pr = 0; pr * kLongRows < n[k]; ++pr) per_head[k] += pair_tiles(len[k] - n[k], n[k], pr) + kPairCost;
        l_units += (int64_t)per_head[k] * p.H;
        ++served;
        served_tiles += tiles[k];
      }
      kv += tiles[k];
    }
    int64_t l_unit = scan(l_units, red, &c.l_units);
    int64_t kv_at = l_at & 0xFFFFFFFFFFFF, rec = l_at >> 48;
    // the served sequences are a prefix of the long ones, so the scans of all of them place them
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      if (!is_long[k]) continue;
      LongSeq s;
      s.unit0 = l_unit;
      s.b = b0 + k;
      s.q0 = q0[k];
      s.n = n[k];
      s.len = len[k];
      s.kv0 = (int)kv_at;
      s.kvt = tiles[k];
      s.per_head = per_head[k];
      s.pad = 0;
      p.l_seqs[rec] = s;
      ++rec;
      kv_at += tiles[k];
      l_unit += (int64_t)per_head[k] * p.H;
    }
    int64_t done;
    scan(((int64_t)served << 48) + served_tiles, red, &done);
    c.l_seqs = (int)(done >> 48);
    c.l_tiles = (int)(done & 0xFFFFFFFFFFFF);
  }
  if (tid == 0) *p.counts = c;
  if (bad) set_err(p.dev_err, MLA_DEVERR_SEQLEN);
  if (__syncthreads_or(zero)) {
    for (int b = 0; b < p.B; ++b) {
      if (!((zero_mask[b >> 5] >> (b & 31)) & 1u)) continue;
      const int64_t lo = max(__ldcg(p.q_start + b), 0), hi = min(__ldcg(p.q_start + b + 1), p.N);
      uint4* rows = reinterpret_cast<uint4*>(p.o);
      for (int64_t i = lo * p.H * (kDv / 8) + tid; i < hi * p.H * (kDv / 8); i += blockDim.x)
        rows[i] = make_uint4(0u, 0u, 0u, 0u);
    }
  }
  return c.s_toks;
}

// chunk_plan_kernel: the plan by one block of its own, for calls with a long path
// or more than kPlanFused sequences.  Bound by the latency of two dependent
// reads and the scans' barriers: about 3 us for up to 128 sequences.
__global__ void __launch_bounds__(kPlanThreads, 1) chunk_plan_kernel(const ChunkParams p, int R) {
  __shared__ int64_t red[32];
  __shared__ uint32_t zero_mask[kMaxBatch / 32];
  pdl_launch_dependents();
  pdl_wait();
  plan_sequences<kPlanPer>(p, R, true, red, zero_mask, [](int, int, int, int) {});
}

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void mma_bf16(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// ---------------------------------------------------------------------------
// absorb_tiles_kernel: the short path's query tiles.  Row r = (token, head h):
// q_lat = q_nope W_UK[h] (bf16 products, fp32 sums), times scale log2 e, one
// rounding to fp16; its last 64 channels are q_pe, likewise.
// Grid (H, 9, z), block 128: a CTA takes 64 channels of a head (y = 8: the
// RoPE part, a copy) and every z-th 16-token tile.  The weight slice sits in
// shared memory; a decode's cost is reading the weights once, most of it
// during the plan.
// PLAN: the call has at most kPlanFused sequences and no long path: every block
// makes the plan for itself (three words per sequence) instead of waiting for a
// kernel that does, and one of them writes it down.  One sequence of 4096 tokens
// 20.7 us a captured call with the plan's own kernel, 19.0 without; 24 drafts 164.8 and
// 163.3.
// ---------------------------------------------------------------------------
constexpr int kAbWS = 64 + 8;        // W slice row stride: ldmatrix without conflicts
constexpr int kAbAS = kDn + 8;

// 4 bytes (channels c, c + 1 of block kb) of padded row `row`
__device__ __forceinline__ uint32_t* tile_word(const ChunkParams& p, int R, int64_t row, int kb, int c) {
  const int rr = (int)(row % R);
  return reinterpret_cast<uint32_t*>(p.q_tiles + ((row / R) * kQBlocks + kb) * (int64_t)R * 128 + rr * 128 +
                                     (((c >> 3) ^ (rr & 7)) << 4) + (c & 7) * 2);
}

template <bool PLAN>
__global__ void __launch_bounds__(128) absorb_tiles_kernel(const ChunkParams p, int R) {
  pdl_launch_dependents();
  __shared__ __align__(16) uint16_t ws[kDn * kAbWS];
  __shared__ __align__(16) uint16_t as[16 * kAbAS];
  __shared__ int2 toks[16];
  const int h = blockIdx.x, kb = blockIdx.y;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, r = lane >> 2, j = lane & 3;
  // the weights are no kernel's output: their fetch overlaps the plan
  if (kb < 8) {
    const uint16_t* wsrc = p.w_uk + (size_t)h * kDn * kDc + 64 * kb;
    uint4 v[kDn * 8 / 128];
#pragma unroll
    for (int i = 0; i < kDn * 8 / 128; ++i) {
      const int e = tid + 128 * i;
      v[i] = __ldcg(reinterpret_cast<const uint4*>(wsrc + (size_t)(e >> 3) * kDc + 8 * (e & 7)));
    }
#pragma unroll
    for (int i = 0; i < kDn * 8 / 128; ++i) {
      const int e = tid + 128 * i;
      *reinterpret_cast<uint4*>(ws + (e >> 3) * kAbWS + 8 * (e & 7)) = v[i];
    }
  }
  pdl_wait();
  __shared__ int3 seqs[PLAN ? kPlanFused : 1];       // first token row, short-path tokens and row tiles before
  int n, n_seqs = 0;
  int2 first = make_int2(0, 0);
  if constexpr (PLAN) {
    __shared__ int64_t red[32];
    __shared__ uint32_t zero_mask[kMaxBatch / 32];
    __shared__ int used;
    if (tid == 0) used = 0;
    // (the scan's barriers lie between)
    n = plan_sequences<1>(p, R, blockIdx.x == 0 && kb == 8 && blockIdx.z == 0, red, zero_mask,
                          [&](int rec, int q0, int tok0, int item0) {
                            seqs[rec] = make_int3(q0, tok0, item0);
                            atomicMax(&used, rec + 1);
                          });
    __syncthreads();
    n_seqs = used;
  } else {
    // the first tokens' records come along with their number (at most 15 places
    // behind the list, still in the workspace)
    if (tid < 16) first = __ldcg(p.s_toks + 16 * blockIdx.z + tid);
    n = __ldcg(&p.counts->s_toks);
  }
  // short-path token t: its row, and its first row in the padded row tiles
  auto token = [&](int t) -> int2 {
    if constexpr (PLAN) {
      int lo = 0, m = n_seqs;                            // the last sequence with tok0 <= t
      while (m > 1) {
        const int half = m >> 1;
        if (seqs[lo + half].y <= t) {
          lo += half;
          m -= half;
        } else {
          m = half;
        }
      }
      const int i = t - seqs[lo].y;
      return make_int2(seqs[lo].x + i, seqs[lo].z * R + i * p.H);
    } else {
      return t < 16 * (int)blockIdx.z + 16 ? first : __ldcg(p.s_toks + t);
    }
  };
  if (16 * (int)blockIdx.z >= n) return;
  auto token_row = [&](int t) -> int64_t {
    if constexpr (PLAN) return token(t).x;
    else return __ldcg(&p.s_toks[t].x);
  };
  const uint32_t a_base = tc::smem_u32(as) + (((lane & 7) + 8 * ((lane >> 3) & 1)) * kAbAS + 8 * (lane >> 4)) * 2;
  const uint32_t b_base =
      tc::smem_u32(ws) + (((lane & 7) + 8 * ((lane >> 3) & 1)) * kAbWS + 16 * warp + 8 * (lane >> 4)) * 2;
  uint4 v[2];
  auto fetch = [&](int t0) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int t = t0 + 8 * i + (tid >> 4);
      v[i] = make_uint4(0, 0, 0, 0);
      if (t < n) v[i] = __ldcg(reinterpret_cast<const uint4*>(p.qn + token_row(t) * p.qn_tok + h * p.qn_head + 8 * (tid & 15)));
    }
  };
  if (kb < 8) fetch(16 * blockIdx.z);
  for (int t0 = 16 * blockIdx.z; t0 < n; t0 += 16 * gridDim.z) {
    __syncthreads();
    if (tid < 16) toks[tid] = t0 + tid < n ? token(t0 + tid) : make_int2(-1, 0);
    __syncthreads();
    if (kb == 8) {
      for (int i = tid; i < 16 * 8; i += 128) {
        const int2 tk = toks[i >> 3];
        const int c = i & 7;
        if (tk.x < 0) continue;
        const uint4 v = __ldcg(reinterpret_cast<const uint4*>(p.qp + tk.x * p.qp_tok + h * p.qp_head + 8 * c));
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        uint32_t o[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) o[q] = tc::half2_bits(bf16lo(w[q]) * p.scale_log2, bf16hi(w[q]) * p.scale_log2);
        *reinterpret_cast<uint4*>(tile_word(p, R, tk.y + h, 8, 8 * c)) = make_uint4(o[0], o[1], o[2], o[3]);
      }
      continue;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) *reinterpret_cast<uint4*>(as + (8 * i + (tid >> 4)) * kAbAS + 8 * (tid & 15)) = v[i];
    fetch(t0 + 16 * gridDim.z);            // the next tile's, while this one is multiplied
    __syncthreads();
    float acc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
    for (int ks = 0; ks < kDn / 16; ++ks) {
      uint32_t a[4], bf[4];
      ldsm_x4(a_base + 32 * ks, a);
      ldsm_x4_t(b_base + 16 * ks * kAbWS * 2, bf);
      mma_bf16(acc[0], a, bf[0], bf[1]);
      mma_bf16(acc[1], a, bf[2], bf[3]);
    }
#pragma unroll
    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int2 tk = toks[r + 8 * e];
        if (tk.x >= 0)
          *tile_word(p, R, tk.y + h, kb, 16 * warp + 8 * nt + 2 * j) =
              tc::half2_bits(acc[nt][2 * e] * p.scale_log2, acc[nt][2 * e + 1] * p.scale_log2);
      }
  }
}

// ---------------------------------------------------------------------------
// project_kernel: o = o_lat W_UV[h] for the short path's rows, fp16 operands
// (W_UV converted as it is staged: exact for weights of normal fp16 range),
// fp32 sums, one rounding to bf16.  Grid (H, 128 / 32, z), block 128: a CTA
// takes 32 columns of a head and every z-th 16-token tile; warp w sums the
// channels 128 w .. 128 w + 127, the four sums are added through shared memory.
// Bound by reading o_lat from L2, once per column block: 16 bytes a lane, a tile
// ahead (50 sequences of 26 tokens at 128 heads: 854 -> 728 us a captured call, of
// which this and the absorption had been 400; 24 drafts at 64 heads 163 -> 159).
// ---------------------------------------------------------------------------
constexpr int kPrN = 32;
constexpr int kPrWS = kPrN + 8;

__global__ void __launch_bounds__(128) project_kernel(const ChunkParams p) {
  pdl_launch_dependents();
  __shared__ __align__(16) uint16_t ws[kDc * kPrWS];
  __shared__ float red[4][16][kPrN + 1];
  const int h = blockIdx.x, n0 = blockIdx.y * kPrN;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, r = lane >> 2, j = lane & 3;
  const uint16_t* wsrc = p.w_uv + (size_t)h * kDc * kDv + n0;
  // the weights are no kernel's output: their fetch overlaps the attention
#pragma unroll
  for (int j0 = 0; j0 < kDc * (kPrN / 8) / 128; j0 += 8) {
    uint4 v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = tid + 128 * (j0 + i);
      v[i] = __ldcg(reinterpret_cast<const uint4*>(wsrc + (size_t)(e / (kPrN / 8)) * kDv + 8 * (e % (kPrN / 8))));
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = tid + 128 * (j0 + i);
      // a lane's 16 bytes of A are two steps' fragments: the rows of 32 channels
      // are stored in the order in which the steps then take them
      const int c = e / (kPrN / 8), at = (c & ~31) | (c & 4) << 2 | (c & 2) << 2 | (c >> 2 & 6) | (c & 1);
      *reinterpret_cast<uint4*>(ws + at * kPrWS + 8 * (e % (kPrN / 8))) =
          make_uint4(tc::half2_bits(bf16lo(v[i].x), bf16hi(v[i].x)), tc::half2_bits(bf16lo(v[i].y), bf16hi(v[i].y)),
                     tc::half2_bits(bf16lo(v[i].z), bf16hi(v[i].z)), tc::half2_bits(bf16lo(v[i].w), bf16hi(v[i].w)));
    }
  }
  pdl_wait();
  const int n = __ldcg(&p.counts->s_toks);
  if (16 * (int)blockIdx.z >= n) return;
  const uint32_t b_base = tc::smem_u32(ws) + ((128 * warp + (lane & 7) + 8 * ((lane >> 3) & 1)) * kPrWS + 8 * (lane >> 4)) * 2;
  // A: o_lat rows t0 + r and t0 + r + 8 of this head, the warp's 128 channels
  uint4 x[2][4];
  auto fetch = [&](int t0) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int t = t0 + r + 8 * e;
      const uint4* row = reinterpret_cast<const uint4*>(p.o_lat + ((int64_t)t * p.H + h) * kDc + 128 * warp + 8 * j);
#pragma unroll
      for (int g = 0; g < 4; ++g) x[e][g] = t < n ? __ldcg(row + 4 * g) : make_uint4(0u, 0u, 0u, 0u);
    }
  };
  fetch(16 * blockIdx.z);
  for (int t0 = 16 * blockIdx.z; t0 < n; t0 += 16 * gridDim.z) {
    __syncthreads();
    uint32_t a[8][4];
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        a[2 * g][e] = x[e][g].x;
        a[2 * g][e + 2] = x[e][g].y;
        a[2 * g + 1][e] = x[e][g].z;
        a[2 * g + 1][e + 2] = x[e][g].w;
      }
    fetch(t0 + 16 * gridDim.z);            // the next tile's, while this one is multiplied
    float acc[4][4] = {};
#pragma unroll
    for (int ks = 0; ks < 8; ++ks)
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        uint32_t bf[4];
        ldsm_x4_t(b_base + (16 * ks * kPrWS + 16 * q) * 2, bf);
        mma_f16(acc[2 * q], a[ks], bf[0], bf[1]);
        mma_f16(acc[2 * q + 1], a[ks], bf[2], bf[3]);
      }
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int e = 0; e < 4; ++e) red[warp][r + 8 * (e >> 1)][8 * q + 2 * j + (e & 1)] = acc[q][e];
    __syncthreads();
    for (int i = tid; i < 16 * (kPrN / 2); i += 128) {
      const int m = i / (kPrN / 2), c = 2 * (i % (kPrN / 2));
      if (t0 + m >= n) continue;
      float s0 = 0.f, s1 = 0.f;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        s0 += red[w][m][c];
        s1 += red[w][m][c + 1];
      }
      uint32_t bits;
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;\n" : "=r"(bits) : "f"(s1), "f"(s0));
      const int tok = __ldcg(p.s_toks + t0 + m).x;
      *reinterpret_cast<uint32_t*>(p.o + ((int64_t)tok * p.H + h) * kDv + n0 + c) = bits;
    }
  }
}

bool al(const void* p, uintptr_t a) { return p && ((uintptr_t)p & (a - 1)) == 0; }

bool sizes_ok(int batch, int n_tokens, int heads, int max_new, int64_t kv_tokens) {
  return batch >= 0 && batch <= kMaxBatch && n_tokens >= 0 && heads >= 16 && heads <= 128 && heads % 16 == 0 &&
         (int64_t)n_tokens * heads <= (int64_t)INT32_MAX && max_new >= 0 && max_new <= n_tokens && kv_tokens >= 0 &&
         kv_tokens <= kLongMost;
}

// Most new tokens that can belong to sequences of the short path.
int64_t short_tokens(int batch, int n_tokens, int max_new) {
  const int64_t most = (int64_t)batch * (max_new < kChunkShort ? max_new : kChunkShort);
  return n_tokens < most ? n_tokens : most;
}

// Workspace of a call; carves it into p where base is not null.
int64_t carve(ChunkParams* p, char* base, int batch, int n_tokens, int heads, int max_new, int64_t kv_tokens, int grid) {
  const int R = short_rows_per_tile(max_new, heads);
  const int64_t toks = short_tokens(batch, n_tokens, max_new);
  const int64_t seqs = batch < n_tokens ? batch : n_tokens;       // with at least one new token
  // a sequence's last row tile may be padded
  const int64_t tiles = (toks * heads + R - 1) / R + seqs;
  const bool lng = has_long(max_new, kv_tokens);
  const int64_t kvt = lng ? kv_tokens / kLongKeys : 0;
  const int64_t l_seqs = lng ? (seqs < n_tokens / (kChunkShort + 1) ? seqs : n_tokens / (kChunkShort + 1)) : 0;
  const int64_t sizes[15] = {(int64_t)sizeof(ChunkCounts),
                             seqs * (int64_t)sizeof(ShortSeq),
                             toks * 8,
                             tiles * kQBlocks * R * 128,
                             toks * heads * kDc * 2,
                             2 * grid * partial_floats(R) * 4,
                             grid * (int64_t)sizeof(SplitRec),
                             l_seqs * (int64_t)sizeof(LongSeq),
                             kvt * kCTile,
                             kvt * kBlkBytes,
                             kvt * 32,
                             lng ? (int64_t)heads * kWHead : 0,
                             kvt * heads * kHeadTile,
                             lng ? 2 * grid * long_partial_floats() * 4 : 0,
                             lng ? grid * (int64_t)sizeof(SplitRec) : 0};
  int64_t off = 0;
  char* at[15];
  for (int i = 0; i < 15; ++i) {
    at[i] = base ? base + off : nullptr;
    off += align256(sizes[i]);
  }
  if (base) {
    p->row_tiles = tiles;
    p->counts = (ChunkCounts*)at[0];
    p->s_seqs = (ShortSeq*)at[1];
    p->s_toks = (int2*)at[2];
    p->q_tiles = (uint8_t*)at[3];
    p->o_lat = (uint16_t*)at[4];
    p->parts = (float*)at[5];
    p->splits = (SplitRec*)at[6];
    p->l_seqs = lng ? (LongSeq*)at[7] : nullptr;
    p->c_tiles = (uint8_t*)at[8];
    p->k_rope = (uint8_t*)at[9];
    p->kflags = (uint32_t*)at[10];
    p->w_tiles = (uint8_t*)at[11];
    p->kv_tiles = (uint8_t*)at[12];
    p->l_parts = (float*)at[13];
    p->l_splits = (SplitRec*)at[14];
  }
  return off;
}

// Blocks of the attention kernels: one per SM.  Without a device (sizes asked
// for on a machine that has none) the GB300's 152.
int chunk_grid() {
  const int sms = device_sm_count();
  return sms > 0 ? (sms < 1024 ? sms : 1024) : 152;
}

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" {

size_t mla_chunk_workspace_bytes(int32_t batch, int32_t n_tokens, int32_t heads, int32_t max_new, int64_t kv_tokens) {
  if (!sizes_ok(batch, n_tokens, heads, max_new, kv_tokens)) return 0;
  return (size_t)carve(nullptr, nullptr, batch, n_tokens, heads, max_new, kv_tokens, chunk_grid());
}

mla_status mla_chunk_attention(const mla_cache_layer* cache, const uint16_t* q_nope, int64_t qn_token_stride,
                               int64_t qn_head_stride, const uint16_t* q_pe, int64_t qp_token_stride,
                               int64_t qp_head_stride, const uint16_t* w_uk, const uint16_t* w_uv,
                               const int32_t* block_table, int32_t max_pages, const int32_t* q_start,
                               const int32_t* seq_lens, int32_t batch, int32_t n_tokens, int32_t heads,
                               int32_t max_new, int64_t kv_tokens, float softmax_scale, void* workspace,
                               size_t workspace_bytes_, uint16_t* o, int32_t* dev_err, mla_stream_t stream) {
  ChunkParams p;
  if (!cache_check(cache, &p.L, &p.outl) || !sizes_ok(batch, n_tokens, heads, max_new, kv_tokens))
    return MLA_ERR_INVALID_ARG;
  if (!(softmax_scale > 0.f) || !isfinite(softmax_scale)) return MLA_ERR_INVALID_ARG;
  if (batch == 0 || n_tokens == 0) return MLA_OK;
  if (max_pages < 1 || (int64_t)max_pages * kPage > (int64_t)INT32_MAX || max_new < 1) return MLA_ERR_INVALID_ARG;
  const int64_t strides[4] = {qn_token_stride, qn_head_stride, qp_token_stride, qp_head_stride};
  for (int i = 0; i < 4; ++i)
    if (strides[i] < 0 || strides[i] % 8) return MLA_ERR_INVALID_ARG;
  if (!al(q_nope, 16) || !al(q_pe, 16) || !al(w_uk, 16) || !al(w_uv, 16) || !al(block_table, 4) || !al(q_start, 4) ||
      !al(seq_lens, 4) || !al(workspace, 256) || !al(o, 16) || (dev_err && !al(dev_err, 4)))
    return MLA_ERR_INVALID_ARG;
  p.grid = chunk_grid();
  if ((int64_t)workspace_bytes_ < carve(&p, (char*)workspace, batch, n_tokens, heads, max_new, kv_tokens, p.grid))
    return MLA_ERR_INVALID_ARG;
  p.pool = (const uint8_t*)cache->pool;
  p.num_pages = cache->num_pages;
  p.qn = q_nope;
  p.qp = q_pe;
  p.qn_tok = qn_token_stride;
  p.qn_head = qn_head_stride;
  p.qp_tok = qp_token_stride;
  p.qp_head = qp_head_stride;
  p.w_uk = w_uk;
  p.w_uv = w_uv;
  p.block_table = block_table;
  p.max_pages = max_pages;
  p.q_start = q_start;
  p.seq_lens = seq_lens;
  p.B = batch;
  p.N = n_tokens;
  p.H = heads;
  p.max_new = max_new;
  p.kv_tokens = kv_tokens;
  p.scale_log2 = softmax_scale * 1.4426950408889634f;
  p.o = o;
  p.dev_err = dev_err;
  p.wait_ns = wait_limit_ns();
  const cudaStream_t st = (cudaStream_t)stream;
  const int R = short_rows_per_tile(max_new, heads);
  const bool fused = batch <= kPlanFused && !p.l_seqs;
  mla_status s = MLA_OK;
  if (!fused) {
    // a thread per sequence; small blocks synchronise faster
    const int plan_threads = batch <= 128 ? 128 : (batch <= 512 ? 512 : kPlanThreads);
    s = cuda_status(launch_pdl(chunk_plan_kernel, dim3(1), dim3(plan_threads), 0, st, p, R));
    if (s != MLA_OK) return s;
  }
  if (p.l_seqs) {
    s = launch_long(p, cache->latent_fmt, cache->kpe_fmt, st);
    if (s != MLA_OK) return s;
  }
  // 16-token tiles of the projections: enough CTAs for four per SM
  const int tok_tiles = (int)((short_tokens(batch, n_tokens, max_new) + 15) / 16);
  const int za = 4 * p.grid / (9 * heads) + 1, zp = 4 * p.grid / (4 * heads) + 1;
  const dim3 ga(heads, 9, tok_tiles < za ? tok_tiles : za);
  s = fused ? cuda_status(launch_pdl(absorb_tiles_kernel<true>, ga, dim3(128), 0, st, p, R))
            : cuda_status(launch_pdl(absorb_tiles_kernel<false>, ga, dim3(128), 0, st, p, R));
  if (s != MLA_OK) return s;
  const int lf = cache->latent_fmt, kf = cache->kpe_fmt;
  s = lf == MLA_FMT_BF16       ? launch_short_bf16(p, lf, kf, R, st)
      : lf == MLA_FMT_INT8_SYM ? launch_short_int8(p, lf, kf, R, st)
      : is_int8_latent(lf)     ? launch_short_int8_blocks(p, lf, kf, R, st)
                               : launch_short_int4(p, lf, kf, R, st);
  if (s != MLA_OK) return s;
  return cuda_status(launch_pdl(project_kernel, dim3(heads, kDv / kPrN, tok_tiles < zp ? tok_tiles : zp), dim3(128), 0, st, p));
}

}  // extern "C"
