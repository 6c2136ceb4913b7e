// mla_select_tokens: which tokens of each sequence stay in a smaller cache.
//
// Of a sequence's L tokens K stay: the first S = min(sinks, K), the last R =
// min(recent, K - S) and, of those in between, the M = K - S - R with the most
// weight, ties to the lower index.  Weights are ordered as unsigned integers
// (sign flipped, NaN lowest), so that the M-th largest is found digit by digit:
// three counting passes of 11, 11 and 10 bits fix a threshold and how many of its
// equals stay, and one more lists the tokens in increasing order.
//
// What bounds it: latency.  A cluster of up to 8 blocks takes a sequence; up to
// 262144 tokens a block's threads hold its weights in registers (8, 16 or 32 each,
// all of a thread's loads in flight at once), beyond that in shared memory.  The
// blocks' counts meet in distributed shared memory.  Many tokens have equal
// weights (never looked at: 0), so a warp adds those up before it counts them.
//
// Measured: one sequence of 32768 tokens cut to 2048 15 us, of which the three
// passes' meetings of the cluster and their reads of the others' counts take 8; 64 of
// 2000 to 65536 tokens, cut to a quarter, 31 us, of which the first pass's additions to
// shared memory take 10.  The table's width decides the blocks and where weights are
// held: the same 64 sequences in a table of 2048 pages take 46 us, of 4096 118, and of
// more, with weights in shared memory, 85; one sequence of 250000 tokens 36 us, of
// 300000 116, of a million 347.
#include <cooperative_groups.h>

#include "checks.cuh"
#include "mla_internal.cuh"
#include "scan.cuh"

namespace mla {
namespace {

namespace cg = cooperative_groups;

constexpr int kSelThreads = 1024, kSelWarps = kSelThreads / 32;
constexpr int kSelBins = 2048;
constexpr int kSelKeys = 32768;                        // weights that a block holds in shared memory; those behind are read again
constexpr int kSelMaxPages = 1 << 24;                  // 2^30 tokens: a block's strides past the end stay in 31 bits

struct SelectParams {
  const float* mass;
  int num_pages;
  const int32_t* table;
  int max_pages;
  const int32_t *seq_lens, *keep_lens;
  int sinks, recent;
  int32_t *kept, *kept_lens;
  int max_keep, keys;
  int32_t* dev_err;
};

// Larger weights get larger keys; NaN the smallest.  -0 and 0 are equal.
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);
  if (x != x) return 0u;
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

struct Exchange {
  uint32_t bins[3][kSelBins];                          // of each pass
  int32_t above, equal;                                // of this block's part, against the threshold
};
// The first pass's digits are a float's exponent and two bits: most weights fall
// into a few dozen bins, and additions to one word come one after the other.  So
// that pass counts in kSelCopies copies, by lane (32768 weights in one block: 16 us
// of that pass with one copy).
constexpr int kSelCopies = 8, kSelPitch = kSelBins + 4;

// One thread's weights: HELD of them in registers, or the block's part in shared
// memory and behind it in global memory (HELD = 0).  Token t_i of thread (w, lane)
// is first + 32 i + lane, first = the warp's run.
template <int HELD>
__global__ void __launch_bounds__(kSelThreads, 1) select_kernel(const SelectParams p, int CL) {
  extern __shared__ uint32_t s_keys[];
  __shared__ Exchange ex;
  __shared__ int red[kSelWarps];
  __shared__ int s_above[kSelWarps], s_equal[kSelWarps];
  __shared__ int s_digit, s_need;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), b = blockIdx.x / CL;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint32_t* copies = s_keys + p.keys;
  for (int i = tid; i < 3 * kSelBins; i += kSelThreads) (&ex.bins[0][0])[i] = 0u;
  for (int i = tid; i < kSelCopies * kSelPitch; i += kSelThreads) copies[i] = 0u;
  pdl_launch_dependents();
  pdl_wait();
  int L = __ldcg(p.seq_lens + b);
  const int K = __ldcg(p.keep_lens + b);
  int32_t* kept = p.kept + (int64_t)b * p.max_keep;
  int err = 0;
  if (L < 0 || L > p.max_pages * kPage) {
    err = MLA_DEVERR_SEQLEN;
    L = 0;
  } else if (K < 0 || (K < L && K > p.max_keep)) {
    err = MLA_DEVERR_SEQLEN;
  }
  if (err || K >= L || K == 0) {                       // the whole cluster alike
    const int n = !err && K == 0 ? 0 : L;
    for (int64_t i = (int64_t)rank * kSelThreads + tid; i < p.max_keep; i += CL * kSelThreads) kept[i] = i < n ? (int)i : -1;
    if (rank == 0 && tid == 0) {
      p.kept_lens[b] = n;
      if (err) set_err(p.dev_err, err);
    }
    return;
  }
  const int sinks = min(p.sinks, K), recent = min(p.recent, K - sinks), want = K - sinks - recent;
  // this block's tokens: whole pages; a warp's: a run of them, so that order
  // needs one exchange of counts
  const int pages = (L + kPage - 1) / kPage, per = (pages + CL - 1) / CL * kPage;
  const int t0 = min(rank * per, L), t1 = min(t0 + per, L);
  const int m0 = max(t0, sinks), m1 = min(t1, L - recent);           // those that compete
  const int run = (t1 - t0 + kSelThreads - 1) / kSelThreads, w0 = min(t0 + warp * run * 32, t1), w1 = min(w0 + run * 32, t1);
  const int32_t* table = p.table + (int64_t)b * p.max_pages;
  auto weight = [&](int page, int t) {
    return page >= 0 && page < p.num_pages ? order_key(__ldcg(p.mass + (int64_t)page * kPage + t % kPage)) : 0u;
  };
  uint32_t held[HELD ? HELD : 1];
  if constexpr (HELD > 0) {
    // lane i: where the weights of the run's i-th 32 tokens begin (they lie in one
    // page), -1: nowhere
    int mine = -1;
    if (w0 + 32 * lane < w1) {
      const int page = __ldcg(table + (w0 + 32 * lane) / kPage);
      if (page < 0 || page >= p.num_pages) set_err(p.dev_err, MLA_DEVERR_PAGE);
      else mine = page * kPage + (w0 + 32 * lane) % kPage;
    }
#pragma unroll
    for (int i = 0; i < HELD; ++i) {
      const int at = __shfl_sync(0xffffffffu, mine, i);
      held[i] = at >= 0 && 32 * i + lane < w1 - w0 ? order_key(__ldcg(p.mass + at + lane)) : 0u;
    }
  } else {
    for (int t = t0 + tid; t < t1; t += kSelThreads) {
      const int page = __ldcg(table + t / kPage);
      if (page < 0 || page >= p.num_pages) set_err(p.dev_err, MLA_DEVERR_PAGE);
      if (t - t0 < p.keys) s_keys[t - t0] = weight(page, t);
    }
    __syncthreads();
  }
  // f(token, its key) for all of the run, 32 tokens at a time, every lane
  auto each = [&](auto f) {
    for (int base = w0; base < w1; base += 32) {
      const int t = base + lane;
      f(t, t >= w1 ? 0u : (t - t0 < p.keys ? s_keys[t - t0] : weight(__ldcg(table + t / kPage), t)));
    }
  };

  // With the weights in registers, bit i of a word stands for the thread's i-th
  // token, w0 + 32 i + lane: those that compete, and the others, which stay.  (Token
  // by token, bounds and all, the 64 ragged sequences took 6 us more.)
  uint32_t competes = 0u, stays = 0u;
  if constexpr (HELD > 0) {
    auto before = [&](int t) {                         // the thread's tokens before t
      const int n = (t - w0 - lane + 31) >> 5;
      return n <= 0 ? 0u : (n >= 32 ? ~0u : (1u << n) - 1u);
    };
    competes = before(min(m1, w1)) & ~before(m0);
    stays = before(w1) & ~competes;
  }
  uint32_t prefix = 0u, mask = 0u;
  int need = want;                                     // how many stay among the keys that share the prefix
#pragma unroll 1
  for (int pass = 0; pass < 3 && want > 0; ++pass) {
    const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
    const uint32_t digits = pass == 2 ? 1023u : 2047u;
    if (pass == 0) __syncthreads();                    // the bins are clear
    // a shared-memory address: through a generic one an addition takes many times as long
    const uint32_t bins = (uint32_t)__cvta_generic_to_shared(pass == 0 ? copies + (lane % kSelCopies) * kSelPitch : ex.bins[pass]);
    // a warp's weights of 0 count at once, where there can be any
    constexpr uint32_t kZero = 0x80000000u;
    const bool zero_too = (kZero & mask) == prefix;
    auto add = [](uint32_t at, uint32_t n) { asm volatile("red.shared.add.u32 [%0], %1;\n" ::"r"(at), "r"(n) : "memory"); };
    auto count = [&](bool in, uint32_t k) {
      if (zero_too) {
        const uint32_t zeros = __ballot_sync(0xffffffffu, in && k == kZero);
        if (zeros && lane == 0) add(bins + 4 * ((kZero >> shift) & digits), (uint32_t)__popc(zeros));
        in = in && k != kZero;
      }
      if (in) add(bins + 4 * ((k >> shift) & digits), 1u);
    };
    if constexpr (HELD > 0) {
      uint32_t in = 0u;
#pragma unroll
      for (int i = 0; i < HELD; ++i) in |= (held[i] & mask) == prefix ? 1u << i : 0u;
      in &= competes;
      const uint32_t any = __reduce_or_sync(0xffffffffu, in);
#pragma unroll
      for (int i = 0; i < HELD; ++i)
        if (any >> i & 1u) count(in >> i & 1u, held[i]);
    } else {
      each([&](int t, uint32_t k) { count(t >= m0 && t < min(m1, w1) && (k & mask) == prefix, k); });
    }
    if (pass == 0) {
      __syncthreads();
      for (int i = tid; i < kSelBins; i += kSelThreads) {
        uint32_t n = 0;
#pragma unroll
        for (int c = 0; c < kSelCopies; ++c) n += copies[c * kSelPitch + i];
        ex.bins[0][i] = n;
      }
    }
    cluster.sync();
    // thread i has bins 2046 - 2 i and the next: from the largest digit down
    const int top = kSelBins - 2 - 2 * tid;
    int high = 0, low = 0;
#pragma unroll 8
    for (int r = 0; r < CL; ++r) {
      const uint2 v = *reinterpret_cast<const uint2*>(&cluster.map_shared_rank(&ex, r)->bins[pass][top]);
      low += v.x;
      high += v.y;
    }
    int total;
    const int above = block_scan<kSelThreads>(high + low, red, &total);
    if (above < need && need <= above + high) {
      s_digit = top + 1;
      s_need = need - above;
    } else if (above + high < need && need <= above + high + low) {
      s_digit = top;
      s_need = need - above - high;
    }
    __syncthreads();
    need = s_need;
    prefix |= (uint32_t)s_digit << shift;
    mask |= digits << shift;
    __syncthreads();                                   // both have been read
  }

  // Which tokens stay
  auto classes = [&](int t, uint32_t k, bool& more, bool& same) {
    const bool competes = t >= m0 && t < m1 && want > 0;
    more = t < w1 && (competes ? k > prefix : (t < sinks || t >= L - recent));
    same = competes && t < w1 && k == prefix;
  };
  int n_more = 0, n_same = 0;
  uint32_t mores = 0u, sames = 0u;                     // bit i: the thread's i-th token
  if constexpr (HELD > 0) {
#pragma unroll
    for (int i = 0; i < HELD; ++i) {
      mores |= held[i] > prefix ? 1u << i : 0u;
      sames |= held[i] == prefix ? 1u << i : 0u;
    }
    if (want == 0) mores = sames = 0u;
    mores = (mores & competes) | stays;
    sames &= competes;
    n_more = __reduce_add_sync(0xffffffffu, __popc(mores));
    n_same = __reduce_add_sync(0xffffffffu, __popc(sames));
  } else {
    each([&](int t, uint32_t k) {
      bool more, same;
      classes(t, k, more, same);
      n_more += __popc(__ballot_sync(0xffffffffu, more));
      n_same += __popc(__ballot_sync(0xffffffffu, same));
    });
  }
  if (lane == 0) {
    s_above[warp] = n_more;
    s_equal[warp] = n_same;
  }
  __syncthreads();
  // every warp: the sums over the warps before it, and the block's
  int a = s_above[lane], e = s_equal[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, a, o), y = __shfl_up_sync(0xffffffffu, e, o);
    if (lane >= o) {
      a += x;
      e += y;
    }
  }
  if (tid == kSelWarps - 1) {
    ex.above = a;
    ex.equal = e;
  }
  int before_more = __shfl_sync(0xffffffffu, a, warp) - n_more, before_same = __shfl_sync(0xffffffffu, e, warp) - n_same;
  cluster.sync();
  if (CL > 1) {
    const int va = lane < rank ? cluster.map_shared_rank(&ex, lane)->above : 0, ve = lane < rank ? cluster.map_shared_rank(&ex, lane)->equal : 0;
    before_more += __reduce_add_sync(0xffffffffu, va);
    before_same += __reduce_add_sync(0xffffffffu, ve);
  }
  const uint32_t below = (1u << lane) - 1u;
  if constexpr (HELD > 0) {
    int at = before_more + min(before_same, need);     // the warp's first place
    if (n_same > 0 && before_same < need) {            // the first equals stay as well
#pragma unroll
      for (int i = 0; i < HELD; ++i) {
        const bool same = sames >> i & 1u;
        const uint32_t bs = __ballot_sync(0xffffffffu, same);
        if (same && before_same + __popc(bs & below) < need) mores |= 1u << i;
        before_same += __popc(bs);
      }
    }
    const uint32_t any = __reduce_or_sync(0xffffffffu, mores);
#pragma unroll
    for (int i = 0; i < HELD; ++i) {
      if (!(any >> i & 1u)) continue;
      const uint32_t b = __ballot_sync(0xffffffffu, mores >> i & 1u);
      if (mores >> i & 1u) kept[at + __popc(b & below)] = w0 + 32 * i + lane;
      at += __popc(b);
    }
  } else {
    each([&](int t, uint32_t k) {
      bool more, same;
      classes(t, k, more, same);
      const uint32_t bm = __ballot_sync(0xffffffffu, more), bs = __ballot_sync(0xffffffffu, same);
      const int ties = before_same + __popc(bs & below);             // equals before this one
      if (more || (same && ties < need)) kept[before_more + __popc(bm & below) + min(ties, need)] = t;
      before_more += __popc(bm);
      before_same += __popc(bs);
    });
  }
  for (int64_t i = K + (int64_t)rank * kSelThreads + tid; i < p.max_keep; i += CL * kSelThreads) kept[i] = -1;
  if (rank == 0 && tid == 0) p.kept_lens[b] = K;
  cluster.sync();                                      // no block leaves while its counts may be read
}

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" mla_status mla_select_tokens(const float* mass, int32_t num_pages, const int32_t* block_table,
                                        int32_t max_pages, const int32_t* seq_lens, const int32_t* keep_lens,
                                        int32_t batch, int32_t sinks, int32_t recent, int32_t* kept, int32_t max_keep,
                                        int32_t* kept_lens, int32_t* dev_err, mla_stream_t stream) {
  if (batch < 0 || batch > kMaxBatch || sinks < 0 || recent < 0 || max_keep < 1) return MLA_ERR_INVALID_ARG;
  if (max_pages < 1 || max_pages > kSelMaxPages) return MLA_ERR_INVALID_ARG;
  if (num_pages < 1 || (int64_t)num_pages * kPage > (int64_t)INT32_MAX) return MLA_ERR_INVALID_ARG;
  if (batch == 0) return MLA_OK;
  if (!ok4(mass) || !ok4(block_table) || !ok4(seq_lens) || !ok4(keep_lens) || !ok4(kept) || !ok4(kept_lens) ||
      (dev_err && !ok4(dev_err)))
    return MLA_ERR_INVALID_ARG;
  // the lengths are read by several blocks at any time
  const int64_t per = (int64_t)batch * 4;
  if (overlap({kept_lens, per}, {seq_lens, per}) || overlap({kept_lens, per}, {keep_lens, per})) return MLA_ERR_INVALID_ARG;
  SelectParams p;
  p.mass = mass;
  p.num_pages = num_pages;
  p.table = block_table;
  p.max_pages = max_pages;
  p.seq_lens = seq_lens;
  p.keep_lens = keep_lens;
  p.sinks = sinks;
  p.recent = recent;
  p.kept = kept;
  p.kept_lens = kept_lens;
  p.max_keep = max_keep;
  p.keys = 0;
  p.dev_err = dev_err;
  // The more tokens a thread holds, the fewer blocks a sequence needs: as few
  // tokens as let all sequences run side by side, one block to an SM.
  const int64_t tokens = (int64_t)max_pages * kPage;
  const int sms = device_sm_count();
  int CL = 0;
  void (*kernel)(const SelectParams, int) = nullptr;
  int smem = 0;
  for (int held = 8; held <= 32; held *= 2) {
    CL = 1;
    while (CL < 8 && tokens > (int64_t)CL * kSelThreads * held) CL *= 2;
    if (tokens > (int64_t)CL * kSelThreads * held) continue;
    kernel = held == 8 ? select_kernel<8> : (held == 16 ? select_kernel<16> : select_kernel<32>);
    if (batch * CL <= sms) break;
  }
  if (!kernel) {
    kernel = select_kernel<0>;
    p.keys = kSelKeys;                                 // a block's part is more
    smem = p.keys * 4;
  }
  smem += kSelCopies * kSelPitch * 4;
  const int which = kernel == select_kernel<0> ? 0 : (kernel == select_kernel<8> ? 1 : (kernel == select_kernel<16> ? 2 : 3));
  static int configured[4][64] = {{0}};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !configured[which][dev]) {
    const mla_status st = cuda_status(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                           (which ? 0 : kSelKeys * 4) + kSelCopies * kSelPitch * 4));
    if (st != MLA_OK) return st;
    if (dev >= 0 && dev < 64) configured[which][dev] = 1;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(batch * CL);
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = (cudaStream_t)stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = CL;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cuda_status(cudaLaunchKernelEx(&cfg, kernel, p, CL));
}
