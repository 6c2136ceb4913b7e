// mla_plan_chunks: the block tables, slot map, positions and lengths of one
// serving step, built on the GPU from the requests' lengths.
//
// For request b (row req[b] of the persistent page table, ctx cached tokens,
// new new ones):
//   need_b  = ceil((ctx + new) / 64) - ceil(ctx / 64)    pages to allocate
//   first_b = sum of need over earlier requests           (exclusive scan)
//   page p of the request: table[req][p] if p < ceil(ctx / 64), else
//                          free[head + first_b + p - ceil(ctx / 64)]
//   q_start_b = sum of new over earlier requests;  token q_start_b + i sits
//   at position ctx + i, slot 64 page + position % 64.
//
// What bounds it: nothing but latency for a decode step (a few hundred
// words), and the [B][max_pages] table copy for large batches.  So one
// launch: every block scans all B requests itself (three words each, at most
// 4096, from L2) instead of waiting for a scan kernel, and takes its share of
// the tokens and of the table.  No block reads what another writes: the
// tokens' old pages come from columns < ceil(ctx / 64) of the persistent
// table, its new columns are only written, and a table row has one owner
// (requests that name the same row are all refused).
//
// Measured: 1 request 3.5 us, 256 requests x 512 pages 4.8 us, 4096 requests x
// 640 pages (11.9 MB) 13.4 us, each as a captured call's share of many; the
// last was 25 us with one element per thread and 64-bit divisions.
#include "mla_internal.cuh"

namespace mla {
namespace {

// Requests per thread, at most: blocks of 256 threads for up to 1024 requests,
// of 1024 threads beyond (every block scans all requests: at 4096 of them a
// 512-thread block with eight each took 20 us against 13.4; blocks of 1024 take
// 4.6 us for 1 request and 6.1 for 256, blocks of 256 3.5 and 4.9).
constexpr int kPlanPer = 4;
constexpr int kPlanSmall = 256, kPlanLarge = kMaxBatch / kPlanPer;
constexpr int kPlanRowWords = kPlanMaxRows / 32;
constexpr int kPlanAhead = 8;
constexpr int kPlanStatic = 512;             // at least the kernel's static shared memory, which counts toward the same limit

struct PlanParams {
  const int32_t *ctx, *nw, *req;
  int B;
  int32_t* table;
  int rows, max_pages;
  const int32_t* free_pages;
  int free_len;
  const int32_t* free_range;
  int num_pages;
  int32_t* block_table;
  int32_t *q_start, *seq_lens, *positions, *token_req, *slot, *free_head;
  int n;
  int32_t* dev_err;
};

// Exclusive scan over the block of one int64 per thread; *total = the sum.
template <int T>
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* red, int64_t* total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int64_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();                                     // an earlier scan's readers of red are done
  if (lane == 31) red[warp] = x;
  __syncthreads();
  int64_t s = lane < T / 32 ? red[lane] : 0;
#pragma unroll
  for (int o = 1; o < T / 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += y;
  }
  *total = __shfl_sync(0xffffffffu, s, T / 32 - 1);
  const int64_t base = __shfl_sync(0xffffffffu, s, warp > 0 ? warp - 1 : 0);
  return (warp ? base : 0) + x - v;
}

__device__ __forceinline__ int pages_of(int tokens) { return (int)(((int64_t)tokens + kPage - 1) / kPage); }

// Where entry b of a per-request array lies: a thread's requests are contiguous,
// so 32 threads write every 8th entry; shifted like this those fall in 32 banks.
__device__ __forceinline__ int spread(int b) { return b + (b >> 5); }

// Dynamic shared memory (entries spread): q_start [B + 1], first [B] (pages before the
// request's own; -1: refused), ctx [B], pages in use after the step [B], table
// row [B], then two bits per persistent row (seen, seen twice).
template <int T>
__global__ void __launch_bounds__(T) plan_kernel(const PlanParams p) {
  extern __shared__ int32_t plan_smem[];
  __shared__ int64_t red[T / 32];
  __shared__ int taken;
  static_assert(sizeof(red) + sizeof(taken) + 16 <= kPlanStatic, "the static share");
  int32_t* s_start = plan_smem;
  const int room = spread(p.B) + 1;
  int32_t* s_first = s_start + room;
  int32_t* s_ctx = s_first + room;
  int32_t* s_now = s_ctx + room;
  int32_t* s_row = s_now + room;
  uint32_t* s_seen = reinterpret_cast<uint32_t*>(s_row + room);
  const int row_words = (p.rows + 31) / 32;
  uint32_t* s_twice = s_seen + row_words;
  const int tid = threadIdx.x;
  for (int i = tid; i < 2 * row_words; i += T) s_seen[i] = 0u;
  if (tid == 0) taken = 0;
  pdl_launch_dependents();
  pdl_wait();
  __syncthreads();

  // this thread's requests b0 .. b0 + per - 1, contiguous so that one scan
  // of the threads' sums orders them
  const int per = (p.B + T - 1) / T;
  const int b0 = tid * per;
  const int cap = p.max_pages * kPage;                 // fits: the host checks it
  int ctx[kPlanPer], nw[kPlanPer], row[kPlanPer];
  int64_t sum = 0;
  int err = 0;
#pragma unroll
  for (int k = 0; k < kPlanPer; ++k) {                 // all loads first: they are in flight together
    const int b = b0 + k;
    const bool mine = k < per && b < p.B;
    ctx[k] = mine ? __ldcg(p.ctx + b) : 0;
    nw[k] = mine ? __ldcg(p.nw + b) : 0;
    row[k] = mine ? __ldcg(p.req + b) : -1;
  }
#pragma unroll
  for (int k = 0; k < kPlanPer; ++k) {
    const int b = b0 + k;
    if (k < per && b < p.B) {
      if (row[k] < 0 || row[k] >= p.rows) {
        err |= MLA_DEVERR_PAGE;
        row[k] = -1;
      } else {
        const uint32_t bit = 1u << (row[k] & 31);
        if (atomicOr(s_seen + (row[k] >> 5), bit) & bit) atomicOr(s_twice + (row[k] >> 5), bit);
      }
      if (ctx[k] < 0 || nw[k] < 0 || (int64_t)ctx[k] + nw[k] > cap) {
        err |= MLA_DEVERR_SEQLEN;
        row[k] = -1;
        ctx[k] = 0;
        if (nw[k] < 0) nw[k] = 0;
      }
      sum += nw[k];
    }
  }
  int64_t total;
  int64_t at = block_scan<T>(sum, red, &total);           // its barriers also order the seen bits
  int64_t need_sum = 0;
#pragma unroll
  for (int k = 0; k < kPlanPer; ++k) {
    const int b = b0 + k;
    if (k < per && b < p.B) {
      s_start[spread(b)] = (int)(at < p.n ? at : p.n);
      at += nw[k];
      if (row[k] >= 0 && ((s_twice[row[k] >> 5] >> (row[k] & 31)) & 1u)) {
        err |= MLA_DEVERR_PAGE;
        row[k] = -1;
      }
      if (at > p.n) {                                  // its tokens do not fit the step's arrays
        err |= MLA_DEVERR_SEQLEN;
        row[k] = -1;
      }
      if (row[k] >= 0) need_sum += pages_of(ctx[k] + nw[k]) - pages_of(ctx[k]);
    }
  }
  if (tid == 0) s_start[spread(p.B)] = (int)(total < p.n ? total : p.n);
  const int head = __ldcg(p.free_range), tail = __ldcg(p.free_range + 1);
  int avail = 0;
  if (head < 0 || tail < head || tail > p.free_len) {
    err |= MLA_DEVERR_PAGE;
  } else {
    avail = tail - head;                               // not before: with a tail far below 0 it would wrap around
  }
  int64_t first = block_scan<T>(need_sum, red, &total);
#pragma unroll
  for (int k = 0; k < kPlanPer; ++k) {
    const int b = b0 + k;
    if (k < per && b < p.B) {
      int f = -1;
      if (row[k] >= 0) {
        const int need = pages_of(ctx[k] + nw[k]) - pages_of(ctx[k]);
        // with the earlier requests' needs all counted, nobody behind the
        // first refusal takes a page: the pages taken are one run
        if (need == 0 || first + need <= avail) {
          f = need ? (int)first : 0;
          if (need) atomicMax(&taken, f + need);
        } else {
          err |= MLA_DEVERR_NO_PAGES;
        }
        first += need;
      }
      s_first[spread(b)] = f;
      s_ctx[spread(b)] = ctx[k];
      s_now[spread(b)] = f >= 0 ? pages_of(ctx[k] + nw[k]) : 0;
      s_row[spread(b)] = row[k];
      if (blockIdx.x == 0) {
        p.q_start[b] = s_start[spread(b)];
        p.seq_lens[b] = f >= 0 ? ctx[k] + nw[k] : 0;
      }
    }
  }
  __syncthreads();
  if (blockIdx.x == 0) {
    if (err) set_err(p.dev_err, err);
    if (tid == 0) {
      p.q_start[p.B] = s_start[spread(p.B)];
      *p.free_head = head + taken;
    }
  }

  const int64_t threads = (int64_t)gridDim.x * T, me = (int64_t)blockIdx.x * T + tid;
  // ---- tokens
  const int used = s_start[spread(p.B)];
  for (int64_t i = me; i < p.n; i += threads) {
    int b = -1, pos = 0, slot = -1;
    if (i < used) {
      int lo = 0, hi = p.B;                            // last b whose q_start is <= i
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_start[spread(mid)] <= i) lo = mid;
        else hi = mid;
      }
      b = lo;
      if (s_first[spread(b)] >= 0) {
        const int c = s_ctx[spread(b)];
        pos = c + (int)(i - s_start[spread(b)]);
        const int pg = pos / kPage, old = pages_of(c);
        const int id = pg < old ? __ldcg(p.table + (int64_t)s_row[spread(b)] * p.max_pages + pg)
                                : __ldcg(p.free_pages + head + s_first[spread(b)] + pg - old);
        if (id >= 0 && id < p.num_pages) slot = id * kPage + (pos & (kPage - 1));
        else set_err(p.dev_err, MLA_DEVERR_PAGE);
      }
    }
    p.positions[i] = pos;
    p.token_req[i] = b;
    p.slot[i] = slot;
  }
  // ---- tables: a warp per row, or several warps on a row's columns when there
  // are more warps; kPlanAhead pieces of 32 columns with their loads in flight
  const int lane = tid & 31;
  const int64_t warps = threads >> 5, wid = me >> 5;
  const int split = (int)(warps / p.B > 1 ? warps / p.B : 1);
  const int64_t lines = warps / split;                 // rows in work at a time
  if (wid < lines * split) {
    const int part = (int)(wid % split);
    for (int64_t b = wid / split; b < p.B; b += lines) {
      const int first = s_first[spread((int)b)], old = pages_of(s_ctx[spread((int)b)]), now = s_now[spread((int)b)];
      int32_t* mine = p.table + (int64_t)max(s_row[spread((int)b)], 0) * p.max_pages;
      int32_t* out = p.block_table + b * p.max_pages;
      for (int64_t c0 = 32 * part + lane; c0 < p.max_pages; c0 += 32 * split * kPlanAhead) {
        int id[kPlanAhead];
#pragma unroll
        for (int e = 0; e < kPlanAhead; ++e) {
          const int64_t pg = c0 + 32 * split * e;
          id[e] = pg >= now ? -1 : (pg < old ? __ldcg(mine + pg) : __ldcg(p.free_pages + head + first + pg - old));
        }
#pragma unroll
        for (int e = 0; e < kPlanAhead; ++e) {
          const int64_t pg = c0 + 32 * split * e;
          if (pg >= p.max_pages) continue;
          if (pg < now) {
            if (id[e] < 0 || id[e] >= p.num_pages) {
              set_err(p.dev_err, MLA_DEVERR_PAGE);
              id[e] = -1;
            }
            if (pg >= old) mine[pg] = id[e];
          }
          out[pg] = id[e];
        }
      }
    }
  }
}

bool ok4(const void* p) { return p && ((uintptr_t)p & 3) == 0; }

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" mla_status mla_plan_chunks(const int32_t* ctx_lens, const int32_t* new_lens, const int32_t* req,
                                      int32_t batch, int32_t* page_table, int32_t rows, int32_t max_pages,
                                      const int32_t* free_pages, int32_t free_len, const int32_t* free_range,
                                      int32_t num_pages, int32_t n_tokens, int32_t* block_table, int32_t* q_start,
                                      int32_t* seq_lens, int32_t* positions, int32_t* token_req, int32_t* slot,
                                      int32_t* free_head, int32_t* dev_err, mla_stream_t stream) {
  if (batch < 0 || batch > kMaxBatch || n_tokens < 0) return MLA_ERR_INVALID_ARG;
  if (rows < 1 || rows > kPlanMaxRows || max_pages < 1 || (int64_t)max_pages * kPage > (int64_t)INT32_MAX)
    return MLA_ERR_INVALID_ARG;
  // slots are 32-bit
  if (num_pages < 1 || (int64_t)num_pages * kPage > (int64_t)INT32_MAX || free_len < 0) return MLA_ERR_INVALID_ARG;
  if (batch == 0) return MLA_OK;
  if (!ok4(ctx_lens) || !ok4(new_lens) || !ok4(req) || !ok4(page_table) || !ok4(free_range) || !ok4(block_table) ||
      !ok4(q_start) || !ok4(seq_lens) || !ok4(free_head) || (free_len > 0 && !ok4(free_pages)) ||
      (dev_err && !ok4(dev_err)))
    return MLA_ERR_INVALID_ARG;
  if (n_tokens > 0 && (!ok4(positions) || !ok4(token_req) || !ok4(slot))) return MLA_ERR_INVALID_ARG;
  if (free_head >= free_range && free_head < free_range + 2) return MLA_ERR_INVALID_ARG;
  PlanParams p;
  p.ctx = ctx_lens;
  p.nw = new_lens;
  p.req = req;
  p.B = batch;
  p.table = page_table;
  p.rows = rows;
  p.max_pages = max_pages;
  p.free_pages = free_pages;
  p.free_len = free_len;
  p.free_range = free_range;
  p.num_pages = num_pages;
  p.block_table = block_table;
  p.q_start = q_start;
  p.seq_lens = seq_lens;
  p.positions = positions;
  p.token_req = token_req;
  p.slot = slot;
  p.free_head = free_head;
  p.n = n_tokens;
  p.dev_err = dev_err;
  const size_t smem = sizeof(int32_t) * ((size_t)5 * (batch + batch / 32 + 1) + 2 * ((rows + 31) / 32));
  const int sms = device_sm_count();
  const bool large = batch > kPlanSmall * kPlanPer;
  const int block = large ? kPlanLarge : kPlanSmall;
  if (smem + kPlanStatic > 48 * 1024) {    // many rows or requests: past what a launch gets unasked
    static int configured[2][64] = {{0}};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64 || !configured[large][dev]) {
      const int most = (int)sizeof(int32_t) * (5 * (kMaxBatch + kMaxBatch / 32 + 1) + 2 * kPlanRowWords);
      const mla_status st = cuda_status(
          cudaFuncSetAttribute(large ? plan_kernel<kPlanLarge> : plan_kernel<kPlanSmall>,
                               cudaFuncAttributeMaxDynamicSharedMemorySize, most));
      if (st != MLA_OK) return st;
      if (dev >= 0 && dev < 64) configured[large][dev] = 1;
    }
  }
  const int64_t work = (int64_t)n_tokens + (int64_t)batch * max_pages;
  const int64_t want = (work + 4 * block - 1) / (4 * block);
  const int64_t most = sms > 0 ? (large ? sms : 2 * sms) : 1;
  const int grid = (int)(want < 1 ? 1 : (want < most ? want : most));
  if (large) return cuda_status(launch_pdl(plan_kernel<kPlanLarge>, dim3(grid), dim3(block), smem, (cudaStream_t)stream, p));
  return cuda_status(launch_pdl(plan_kernel<kPlanSmall>, dim3(grid), dim3(block), smem, (cudaStream_t)stream, p));
}
