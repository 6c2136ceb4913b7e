// mla_verify_drafts: drafted tokens against the target's probabilities, and
// the token sampled behind the accepted ones.
//
// Row r of sequence b (rows row_start[b] .. row_start[b + 1] - 1, one more
// than its drafts) judges the draft d_r.  With c(x) = x for 0 < x < inf, else 0:
//   d_r passes where u_r c(q_r(d_r)) < c(p_r(d_r)); the first that does not
//   ends the accepted ones, at row j; w(v) = max(c(p_j(v)) - c(q_j(v)), 0)
//   (all passed: j is the last row and w = c(p_j)), and the next token is the
//   smallest v with sum of w up to v > u total(w).
// The product and the subtraction round nothing (below), and the sums are good to
// 2^-40: a border between two tokens is 1 / vocab wide, and an fp32 sum would
// pick a neighbour now and then.  Rows need not be probabilities: where a sum passes
// fp32's range it is made in fp64.
//
// What bounds it: reading row j of p and q once (a megabyte for 131072 fp32
// probabilities); one sequence is latency.  A cluster of blocks shares a
// sequence, so that a few sequences spread over many SMs.  A warp sums tiles of
// 1024 values: w and its rounding error by Dekker's difference (c(p) >= min(c(p),
// c(q)) >= 0), the sum by a two-sum, 14 fp32 operations a value (an fp64 addition
// costs 64 times an fp32 one here: 33.5 million of them 55 us).  The tiles' sums
// meet in distributed shared memory; one warp then reads the tile that holds the
// border again, in fp64.
//
// Measured (a captured call's share of many): 256 sequences of up to 4 drafts over
// 131072 fp32 values 68 us, 3.2 TB/s of the 216 MB read (one row where all drafts
// passed, else two) or 48% of a plain copy's rate; half the bytes, in 16 bits or from the
// target's row alone (drafts that were certain, or none), 60 to 62 us: the additions of
// a value, and rows that begin and end in step, bound it then.  64 sequences with rows
// that are not aligned with each other 48 us, 45 in 16 bits.  One of 4 drafts over 32003
// values 9.6 us, latency: lengths, drafts, their probabilities, the row, two meetings of
// the cluster and the last tile follow one another.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "checks.cuh"
#include "mla_internal.cuh"
#include "tc.cuh"

namespace mla {
namespace {

namespace cg = cooperative_groups;

constexpr int kVerThreads = 256, kVerWarps = kVerThreads / 32;
constexpr int kVerTile = 1024;                         // values per tile
constexpr int kVerMaxVocab = 1 << 22;

struct VerifyParams {
  const void *p, *q;
  int64_t p_row, q_row;                                // row strides in elements
  int vocab;
  const int32_t *drafts, *row_start;
  const float *u_accept, *u_sample;
  int B, rows, width;
  const int32_t* seq_lens;
  int32_t *accepted, *tokens, *kept_lens;
  int32_t* dev_err;
};

template <typename T>
__device__ __forceinline__ float to_f(T x);
template <>
__device__ __forceinline__ float to_f(float x) { return x; }
template <>
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
template <>
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }

__device__ __forceinline__ float positive(float x) { return x > 0.f && x < INFINITY ? x : 0.f; }

// Elements e .. e + N - 1 of a row (N fill 16 bytes), 0 outside [0, vocab):
// one 16-byte load where they are all inside and aligned.  (The rows may come from a
// kernel that still runs when this one starts: no non-coherent loads, though they
// would take 0.5% less.)
template <typename T, int N>
__device__ __forceinline__ void load_row(const T* row, int e, int vocab, float* v) {
  if (e >= 0 && e + N <= vocab && (reinterpret_cast<uintptr_t>(row + e) & 15) == 0) {
    const uint4 raw = __ldcg(reinterpret_cast<const uint4*>(row + e));
    const T* x = reinterpret_cast<const T*>(&raw);
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = positive(to_f(x[i]));
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = e + i >= 0 && e + i < vocab ? positive(to_f(row[e + i])) : 0.f;
  }
}

template <typename T, int N>
__device__ __forceinline__ void widen(const uint4& raw, float* v) {      // NaN and what is below 0: 0
  const T* x = reinterpret_cast<const T*>(&raw);
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = fmaxf(to_f(x[i]), 0.f);
}

// (h, l) += w exactly up to l's rounding.
__device__ __forceinline__ void two_sum(float& h, float& l, float w) {
  const float s = __fadd_rn(h, w), b = __fadd_rn(s, -h);
  l = __fadd_rn(l, __fadd_rn(__fadd_rn(h, -__fadd_rn(s, -b)), __fadd_rn(w, -b)));
  h = s;
}

// A lane's sum over a tile in fp64, value by value: what lies beside the loop over
// the tiles must be short and need few registers.
template <typename T>
__device__ __forceinline__ double wide_sum(const T* pr, const T* qr, int first, int vocab, int skip) {
  double sum = 0.0;
#pragma unroll 1
  for (int e = max(first, 0) + (int)(threadIdx.x & 31); e < min(first + kVerTile, vocab); e += 32) {
    const float a = e == skip ? 0.f : positive(to_f(pr[e]));
    sum += (double)a - (double)fminf(a, qr ? positive(to_f(qr[e])) : 0.f);
  }
  return sum;
}

template <typename T>
__global__ void __launch_bounds__(kVerThreads, 4) verify_kernel(const VerifyParams p, int CL) {
  constexpr int N = 16 / sizeof(T), kSweeps = kVerTile / (32 * N), kBatch = 4;
  extern __shared__ double s_sums[];                   // this block's tiles' sums; in the last block's turn all of them
  __shared__ int s_fail;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), b = blockIdx.x / CL;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_launch_dependents();
  pdl_wait();
  // a row_start that decreases or leaves the rows anywhere refuses all sequences
  bool bad = false;
  for (int i = tid; i < p.B; i += kVerThreads) {
    const int lo = __ldcg(p.row_start + i), hi = __ldcg(p.row_start + i + 1);
    bad |= lo < 0 || hi < lo || hi > p.rows;
  }
  if (tid == 0) s_fail = 0x7FFFFFFF;
  bad = __syncthreads_or(bad);
  const int r0 = __ldcg(p.row_start + b), n = bad ? 0 : __ldcg(p.row_start + b + 1) - r0;
  const bool fits = n <= p.width;
  int32_t* out = p.tokens + (int64_t)b * p.width;
  if (n == 0 || !fits) {                               // the whole cluster alike
    if (rank == 0) {
      for (int i = tid; i < p.width; i += kVerThreads) out[i] = -1;
      if (tid == 0) {
        p.accepted[b] = 0;
        if (p.kept_lens) p.kept_lens[b] = __ldcg(p.seq_lens + b);
        if (bad || !fits) set_err(p.dev_err, MLA_DEVERR_SEQLEN);
      }
    }
    return;
  }
  const T *P = reinterpret_cast<const T*>(p.p), *Q = reinterpret_cast<const T*>(p.q);
  for (int i = tid; i < n - 1; i += kVerThreads) {
    const int64_t r = (int64_t)r0 + i;
    const int d = __ldcg(p.drafts + r);
    bool pass = false;
    if (d >= 0 && d < p.vocab) {
      const double pd = positive(to_f(P[r * p.p_row + d])), qd = Q ? positive(to_f(Q[r * p.q_row + d])) : 1.f;
      pass = (double)__ldcg(p.u_accept + r) * qd < pd;               // exact: 48 bits
    } else if (rank == 0) {
      set_err(p.dev_err, MLA_DEVERR_TOKEN);
    }
    if (!pass) atomicMin(&s_fail, i);
  }
  __syncthreads();
  const int acc = min(s_fail, n - 1);
  const bool rejected = acc < n - 1;
  const int64_t row = (int64_t)r0 + acc;
  const T *pr = P + row * p.p_row, *qr = rejected && Q ? Q + row * p.q_row : nullptr;
  int skip = rejected && !Q ? __ldcg(p.drafts + row) : -1;           // a draft that was certain has no weight left
  const int mis = (int)((reinterpret_cast<uintptr_t>(pr) & 15) / sizeof(T));     // tiles lie on p's 16-byte boundaries
  const int tiles = (p.vocab + mis + kVerTile - 1) / kVerTile;

  double total = 0.0;
  for (int attempt = 0; attempt < 2; ++attempt) {
    for (int t = rank + CL * warp; t < tiles; t += CL * kVerWarps) {
      float h[2] = {0.f, 0.f}, l[2] = {0.f, 0.f};      // two chains of additions side by side
      float top = 0.f;                                 // the draft's largest entry
      const int e0 = t * kVerTile - mis + lane * N, first = t * kVerTile - mis;
      auto add = [&](const float* a, const float* c, int e) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
          if (c) {
            // w + err = a - min(a, c) exactly
            const float q = fminf(a[i], c[i]), w = __fadd_rn(a[i], -q), err = __fadd_rn(__fadd_rn(a[i], -w), -q);
            two_sum(h[i & 1], l[i & 1], w);
            l[i & 1] = __fadd_rn(l[i & 1], err);
          } else {
            two_sum(h[i & 1], l[i & 1], e + i == skip ? 0.f : a[i]);
          }
        }
      };
      bool careful = qr && (reinterpret_cast<uintptr_t>(qr + first) & 15) != 0;
      if (!careful) {
        // aligned: kBatch loads of a lane and row in flight; what the row's ends
        // leave of a lane's 16 bytes comes one by one
#pragma unroll
        for (int s0 = 0; s0 < kSweeps; s0 += kBatch) {
          uint4 ra[kBatch], rc[kBatch];
          const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
          for (int s = 0; s < kBatch; ++s) {
            const int e = e0 + (s0 + s) * 32 * N;
            ra[s] = e >= 0 && e + N <= p.vocab ? __ldcg(reinterpret_cast<const uint4*>(pr + e)) : zero;
          }
          if (qr) {
#pragma unroll
            for (int s = 0; s < kBatch; ++s) {
              const int e = e0 + (s0 + s) * 32 * N;
              rc[s] = e >= 0 && e + N <= p.vocab ? __ldcg(reinterpret_cast<const uint4*>(qr + e)) : zero;
            }
          }
#pragma unroll
          for (int s = 0; s < kBatch; ++s) {
            const int e = e0 + (s0 + s) * 32 * N;
            float a[N], c[N];
            widen<T, N>(ra[s], a);
            if (qr) {
              widen<T, N>(rc[s], c);
#pragma unroll
              for (int i = 0; i < N; i += 2) top = tc::max3(top, c[i], c[i + 1]);
              add(a, c, e);
            } else {
              add(a, nullptr, e);
            }
          }
        }
#pragma unroll 1
        for (int end = 0; end < 2; ++end) {
          // the lane's 16 bytes over the row's beginning, or over its end
          const int at = end ? (p.vocab + mis) / N * N - mis : -mis, k = at - e0;
          if (k < 0 || k >= kVerTile || k % (32 * N) || (at >= 0 && at + N <= p.vocab) || (end && at <= 0)) continue;
          float a[N], c[N];
          load_row<T, N>(pr, at, p.vocab, a);
          if (qr) load_row<T, N>(qr, at, p.vocab, c);
          add(a, qr ? c : nullptr, at);
        }
        // an infinite entry (which has no weight) has spoilt a sum, or, the draft's,
        // has taken a finite one of the target away
        careful = __any_sync(0xffffffffu, !(h[0] + h[1] < INFINITY) || top == INFINITY);
        if (careful) h[0] = h[1] = l[0] = l[1] = 0.f;
      }
      if (careful) {
#pragma unroll 1
        for (int s = 0; s < kSweeps; ++s) {
          const int e = e0 + s * 32 * N;
          float a[N], c[N];
          load_row<T, N>(pr, e, p.vocab, a);
          if (qr) load_row<T, N>(qr, e, p.vocab, c);
          add(a, qr ? c : nullptr, e);
        }
      }
      double sum = ((double)h[0] + (double)l[0]) + ((double)h[1] + (double)l[1]);
      // finite entries whose sum no fp32 holds
      if (careful && __any_sync(0xffffffffu, !(h[0] + h[1] < INFINITY))) sum = wide_sum<T>(pr, qr, first, p.vocab, skip);
#pragma unroll
      for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (lane == 0) s_sums[t / CL] = sum;
    }
    cluster.sync();
    // every block adds up all tiles' sums in the same order
    total = 0.0;
    for (int t = lane; t < tiles; t += 32) total += cluster.map_shared_rank(s_sums, t % CL)[t / CL];
#pragma unroll
    for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    if (total > 0.0 || !rejected || attempt) break;
    // nothing left of the target's row: the draft's has as much everywhere
    qr = nullptr;
    skip = -1;
    cluster.sync();                                    // the sums have been read
  }
  if (rank == 0 && warp == 0) {
    double u = (double)__ldcg(p.u_sample + b);
    u = u > 0.0 ? (u < 1.0 ? u : 1.0) : 0.0;           // NaN: 0
    const double target = u * total;
    int pick = -1;
    if (total > 0.0) {
      // the first tile whose running sum passes the target, else the last with any weight
      double base = 0.0, at_base = 0.0;
      int tile = -1;
      bool found = false;
      for (int t0 = 0; t0 < tiles && !found; t0 += 32) {
        const int t = t0 + lane;
        const double mine = t < tiles ? cluster.map_shared_rank(s_sums, t % CL)[t / CL] : 0.0;
        double incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const double y = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += y;
        }
        const uint32_t hit = __ballot_sync(0xffffffffu, mine > 0.0 && base + incl > target);
        const uint32_t some = __ballot_sync(0xffffffffu, mine > 0.0);
        found = hit != 0;
        if (some) {
          const int l = found ? __ffs(hit) - 1 : 31 - __clz(some);
          tile = t0 + l;
          at_base = base + __shfl_sync(0xffffffffu, incl - mine, l);
        }
        base += __shfl_sync(0xffffffffu, incl, 31);
      }
      // and in it the first value, in fp64
      double before = at_base;
      found = false;
#pragma unroll 1
      for (int s = 0; s < kSweeps && !found; ++s) {
        const int e = tile * kVerTile - mis + (s * 32 + lane) * N;
        float a[N], c[N];
        load_row<T, N>(pr, e, p.vocab, a);
        if (qr) load_row<T, N>(qr, e, p.vocab, c);
        double w[N], sum = 0.0;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const double x = qr ? (double)a[i] - (double)c[i] : (double)a[i];
          w[i] = x > 0.0 && e + i != skip ? x : 0.0;
          sum += w[i];
        }
        double incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const double y = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += y;
        }
        double cum = before + (incl - sum);
        int first = -1, last = -1;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          cum += w[i];
          if (w[i] > 0.0) {
            last = e + i;
            if (first < 0 && cum > target) first = e + i;
          }
        }
        const uint32_t hit = __ballot_sync(0xffffffffu, first >= 0), some = __ballot_sync(0xffffffffu, last >= 0);
        found = hit != 0;
        if (found) pick = __shfl_sync(0xffffffffu, first, __ffs(hit) - 1);
        else if (some) pick = __shfl_sync(0xffffffffu, last, 31 - __clz(some));
        before += __shfl_sync(0xffffffffu, incl, 31);
      }
    }
    for (int i = lane; i < p.width; i += 32)
      out[i] = i < acc ? __ldcg(p.drafts + r0 + i) : (i == acc ? pick : -1);
    if (lane == 0) {
      p.accepted[b] = acc;
      if (pick < 0) set_err(p.dev_err, MLA_DEVERR_TOKEN);
      if (p.kept_lens) {
        const int len = __ldcg(p.seq_lens + b), kept = len - (n - 1 - acc);
        p.kept_lens[b] = kept < 0 ? 0 : kept;
        if (kept < 0) set_err(p.dev_err, MLA_DEVERR_SEQLEN);
      }
    }
  }
  cluster.sync();                                      // no block leaves while its sums may be read
}

template <typename T>
mla_status launch_verify(const VerifyParams& p, cudaStream_t stream) {
  // Blocks of a sequence: 8 where there are few sequences, so that their rows
  // spread over the SMs; with many, no more blocks than run side by side, four to an
  // SM (256 sequences of 131072 fp32 values: 96 us with 1, 68 with 2, 83 with 4, 112
  // with 8, which come in four waves; three blocks to an SM 88, five 83.  One sequence: 16,
  // 12, 9.8 and 9.6 us).
  const int sms = device_sm_count();
  int CL = 8;
  while (CL > 1 && (int64_t)p.B * CL > 4 * (int64_t)sms) CL /= 2;
  const int tiles = (p.vocab + kVerTile - 1) / kVerTile + 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.B * CL);
  cfg.blockDim = dim3(kVerThreads);
  cfg.dynamicSmemBytes = (size_t)((tiles + CL - 1) / CL) * sizeof(double);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = CL;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cuda_status(cudaLaunchKernelEx(&cfg, verify_kernel<T>, p, CL));
}

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" mla_status mla_verify_drafts(const void* target_probs, int64_t target_row_stride, const void* draft_probs,
                                        int64_t draft_row_stride, int32_t prob_type, int32_t vocab,
                                        const int32_t* drafts, const int32_t* row_start, int32_t batch, int32_t rows,
                                        const float* u_accept, const float* u_sample, const int32_t* seq_lens,
                                        int32_t* accepted, int32_t* tokens, int32_t max_out, int32_t* kept_lens,
                                        int32_t* dev_err, mla_stream_t stream) {
  if (batch < 0 || batch > kMaxBatch || rows < 0 || vocab < 1 || vocab > kVerMaxVocab || max_out < 1)
    return MLA_ERR_INVALID_ARG;
  if (prob_type != MLA_PROB_FP32 && prob_type != MLA_PROB_BF16 && prob_type != MLA_PROB_FP16) return MLA_ERR_INVALID_ARG;
  if (batch == 0) return MLA_OK;
  const uintptr_t size = prob_type == MLA_PROB_FP32 ? 4 : 2;
  if (rows > 0 && (!aligned_to(target_probs, size) || target_row_stride < vocab || !aligned_to(drafts, 4) ||
                   !aligned_to(u_accept, 4)))
    return MLA_ERR_INVALID_ARG;
  if (rows > 0 && draft_probs && (!aligned_to(draft_probs, size) || draft_row_stride < vocab)) return MLA_ERR_INVALID_ARG;
  if (!aligned_to(row_start, 4) || !aligned_to(u_sample, 4) || !aligned_to(accepted, 4) || !aligned_to(tokens, 4))
    return MLA_ERR_INVALID_ARG;
  if ((kept_lens != nullptr) != (seq_lens != nullptr) || (kept_lens && (!aligned_to(kept_lens, 4) || !aligned_to(seq_lens, 4))) ||
      (dev_err && !aligned_to(dev_err, 4)))
    return MLA_ERR_INVALID_ARG;
  // in place, or apart: sequences read theirs at any time
  const int64_t per = (int64_t)batch * 4;
  if (kept_lens != seq_lens && overlap({kept_lens, per}, {seq_lens, per})) return MLA_ERR_INVALID_ARG;
  if (rows > 0 && (INT64_MAX / 4) / rows < (target_row_stride > draft_row_stride || !draft_probs ? target_row_stride : draft_row_stride))
    return MLA_ERR_INVALID_ARG;
  VerifyParams p;
  p.p = target_probs;
  p.q = draft_probs;
  p.p_row = target_row_stride;
  p.q_row = draft_row_stride;
  p.vocab = vocab;
  p.drafts = drafts;
  p.row_start = row_start;
  p.u_accept = u_accept;
  p.u_sample = u_sample;
  p.B = batch;
  p.rows = rows;
  p.width = max_out;
  p.seq_lens = seq_lens;
  p.accepted = accepted;
  p.tokens = tokens;
  p.kept_lens = kept_lens;
  p.dev_err = dev_err;
  if (prob_type == MLA_PROB_FP32) return launch_verify<float>(p, (cudaStream_t)stream);
  if (prob_type == MLA_PROB_BF16) return launch_verify<__nv_bfloat16>(p, (cudaStream_t)stream);
  return launch_verify<__half>(p, (cudaStream_t)stream);
}
