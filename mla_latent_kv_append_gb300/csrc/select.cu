// mla_select_tokens: which tokens of each sequence stay in a smaller cache.
//
// Of a sequence's L tokens K stay: the first S = min(sinks, K), the last R =
// min(recent, K - S) and, of those in between, the M = K - S - R with the most
// weight, ties to the lower index.  Weights are ordered as unsigned integers
// (sign flipped, NaN lowest), so that the M-th largest is found digit by digit:
// three counting passes of 11, 11 and 10 bits fix a threshold and how many of its
// equals stay, and one more lists the tokens in increasing order.
//
// What bounds it: latency.  A cluster of up to 8 blocks takes a sequence; each
// holds its part of the weights in shared memory (read once, through the block
// table), the blocks' counts meet in distributed shared memory.  Many tokens
// have equal weights (never looked at: 0), so a warp adds equal digits up
// before it counts them.
#include <cooperative_groups.h>

#include "mla_internal.cuh"
#include "scan.cuh"

namespace mla {
namespace {

namespace cg = cooperative_groups;

constexpr int kSelThreads = 1024, kSelWarps = kSelThreads / 32;
constexpr int kSelBins = 2048;
constexpr int kSelKeys = 49152;                        // weights that a block holds; those behind are read again
constexpr int kSelMaxPages = 1 << 24;                  // 2^30 tokens: a block's strides past the end stay in 31 bits
constexpr int kSelPart = 32768;                        // tokens per block where the cluster can be larger

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
  uint32_t bins[kSelBins];
  int32_t above, equal;                                // of this block's part, against the threshold
};

__global__ void __launch_bounds__(kSelThreads, 1) select_kernel(const SelectParams p, int CL) {
  extern __shared__ uint32_t s_keys[];
  __shared__ Exchange ex;
  __shared__ int red[kSelWarps];
  __shared__ int s_above[kSelWarps], s_equal[kSelWarps];
  __shared__ int s_digit, s_need;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), b = blockIdx.x / CL;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
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
    for (int i = rank * kSelThreads + tid; i < p.max_keep; i += CL * kSelThreads) kept[i] = i < n ? i : -1;
    if (rank == 0 && tid == 0) {
      p.kept_lens[b] = n;
      if (err) set_err(p.dev_err, err);
    }
    return;
  }
  const int sinks = min(p.sinks, K), recent = min(p.recent, K - sinks), want = K - sinks - recent;
  // this block's tokens: whole pages
  const int pages = (L + kPage - 1) / kPage, per = (pages + CL - 1) / CL * kPage;
  const int t0 = min(rank * per, L), t1 = min(t0 + per, L);
  const int m0 = max(t0, sinks), m1 = min(t1, L - recent);           // those that compete
  const int32_t* table = p.table + (int64_t)b * p.max_pages;
  auto fetch = [&](int t) {
    const int page = __ldcg(table + t / kPage);
    return page >= 0 && page < p.num_pages ? order_key(__ldcg(p.mass + (int64_t)page * kPage + t % kPage)) : 0u;
  };
  for (int t = t0 + tid; t < t1; t += kSelThreads) {
    if (t - t0 < p.keys) s_keys[t - t0] = fetch(t);
    if (t % kPage == 0) {
      const int page = __ldcg(table + t / kPage);
      if (page < 0 || page >= p.num_pages) set_err(p.dev_err, MLA_DEVERR_PAGE);
    }
  }
  auto key = [&](int t) { return t - t0 < p.keys ? s_keys[t - t0] : fetch(t); };

  uint32_t prefix = 0u, mask = 0u;
  int need = want;                                     // how many stay among the keys that share the prefix
  for (int pass = 0; pass < 3 && want > 0; ++pass) {
    const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0), bits = pass == 2 ? 10 : 11;
    const uint32_t digits = (1u << bits) - 1u;
    for (int i = tid; i < kSelBins; i += kSelThreads) ex.bins[i] = 0u;
    __syncthreads();
    for (int base = m0 + warp * 32; base < m1; base += kSelThreads) {
      const int t = base + lane;
      const uint32_t k = t < m1 ? key(t) : 0u;
      const bool in = t < m1 && (k & mask) == prefix;
      const uint32_t d = (k >> shift) & digits;
      const uint32_t peers = __match_any_sync(0xffffffffu, in ? d : 0xFFFFFFFFu);
      if (in && lane == __ffs(peers) - 1) atomicAdd(&ex.bins[d], (uint32_t)__popc(peers));
    }
    cluster.sync();
    // thread i has bins 2046 - 2 i and the next: from the largest digit down
    const int top = kSelBins - 2 - 2 * tid;
    int hi = 0, lo = 0;
    for (int r = 0; r < CL; ++r) {
      const uint2 v = *reinterpret_cast<const uint2*>(&cluster.map_shared_rank(&ex, r)->bins[top]);
      lo += v.x;
      hi += v.y;
    }
    int total;
    const int above = block_scan<kSelThreads>(hi + lo, red, &total);
    if (above < need && need <= above + hi) {
      s_digit = top + 1;
      s_need = need - above;
    } else if (above + hi < need && need <= above + hi + lo) {
      s_digit = top;
      s_need = need - above - hi;
    }
    __syncthreads();
    need = s_need;
    prefix |= (uint32_t)s_digit << shift;
    mask |= digits << shift;
    cluster.sync();                                    // the counts have been read
  }

  // Which tokens stay: a warp takes a run of the part, so that order needs one
  // exchange of counts
  const int run = ((t1 - t0 + kSelThreads - 1) / kSelThreads) * 32, w0 = t0 + warp * run, w1 = min(w0 + run, t1);
  auto classes = [&](int t, bool& more, bool& same) {
    const bool competes = t >= m0 && t < m1 && want > 0;
    const uint32_t k = competes ? key(t) : 0u;
    more = t < w1 && (competes ? k > prefix : (t < sinks || t >= L - recent));
    same = competes && t < w1 && k == prefix;
  };
  int n_more = 0, n_same = 0;
  for (int base = w0; base < w1; base += 32) {
    bool more, same;
    classes(base + lane, more, same);
    n_more += __popc(__ballot_sync(0xffffffffu, more));
    n_same += __popc(__ballot_sync(0xffffffffu, same));
  }
  if (lane == 0) {
    s_above[warp] = n_more;
    s_equal[warp] = n_same;
  }
  __syncthreads();
  if (tid == 0) {
    int a = 0, e = 0;
    for (int w = 0; w < kSelWarps; ++w) {
      const int x = s_above[w], y = s_equal[w];
      s_above[w] = a;
      s_equal[w] = e;
      a += x;
      e += y;
    }
    ex.above = a;
    ex.equal = e;
  }
  cluster.sync();
  int before_more = s_above[warp], before_same = s_equal[warp];
  for (int r = 0; r < rank; ++r) {
    before_more += cluster.map_shared_rank(&ex, r)->above;
    before_same += cluster.map_shared_rank(&ex, r)->equal;
  }
  for (int base = w0; base < w1; base += 32) {
    bool more, same;
    const int t = base + lane;
    classes(t, more, same);
    const uint32_t bm = __ballot_sync(0xffffffffu, more), bs = __ballot_sync(0xffffffffu, same);
    const uint32_t below = (1u << lane) - 1u;
    const int ties = before_same + __popc(bs & below);               // equals before this one
    if (more || (same && ties < need)) kept[before_more + __popc(bm & below) + min(ties, need)] = t;
    before_more += __popc(bm);
    before_same += __popc(bs);
  }
  for (int i = K + rank * kSelThreads + tid; i < p.max_keep; i += CL * kSelThreads) kept[i] = -1;
  if (rank == 0 && tid == 0) p.kept_lens[b] = K;
  cluster.sync();                                      // no block leaves while its counts may be read
}

bool ok4(const void* p) { return p && ((uintptr_t)p & 3) == 0; }

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
  if (kept_lens == seq_lens || kept_lens == keep_lens) return MLA_ERR_INVALID_ARG;      // read by several blocks
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
  p.dev_err = dev_err;
  int CL = 1;
  const int64_t tokens = (int64_t)max_pages * kPage;
  while (CL < 8 && tokens > (int64_t)CL * kSelPart) CL *= 2;
  const int64_t part = ((max_pages + CL - 1) / CL) * (int64_t)kPage;
  p.keys = (int)(part < kSelKeys ? part : kSelKeys);
  const int smem = p.keys * 4;
  static int configured[64] = {0};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !configured[dev]) {
    const mla_status st =
        cuda_status(cudaFuncSetAttribute(select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSelKeys * 4));
    if (st != MLA_OK) return st;
    if (dev >= 0 && dev < 64) configured[dev] = 1;
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
  return cuda_status(cudaLaunchKernelEx(&cfg, select_kernel, p, CL));
}
