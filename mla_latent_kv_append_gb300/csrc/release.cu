// mla_release_pages: page tables and the free list after requests got shorter.
//
// For request b with was_b = ceil(old / 64) pages and now_b = ceil(new / 64):
//   trim   pages now_b .. was_b - 1 go back, the others stay
//   move   (new < old) pages 0 .. was_b - 1 go back, now_b fresh ones come
// Pages come from the free list's head, as the plan's do, and those given back
// follow in front of what is left:
//   fresh page j of the request    = free[head + take_b + j]
//   new head                       = head + take - back
//   free[new head + back_b + j]    = the request's j-th page given back
// (take_b, back_b: sums over earlier requests, exclusive scans; take, back: of
// all).  What is given back lands on the places of what was taken, so a move
// is two launches: one that reads the list, one that writes it.  A trim takes
// nothing and is one.
//
// What bounds it: latency for a step's few requests, and the [B][max_pages]
// tables for large batches.  As for the step plan, every block scans all B
// requests itself (three words each, from L2) and then takes its share of the
// rows.
//
// Measured: 32 requests x 512 pages trimmed 3.0 us; 4096 x 640 moved 26 us: two
// launches that each scan all requests (8 us), then the tables (6) and the list (4).
#include "checks.cuh"
#include "mla_internal.cuh"
#include "scan.cuh"

namespace mla {
namespace {

constexpr int kRelPer = 4;                             // requests per thread, at most
constexpr int kRelSmall = 256, kRelLarge = kMaxBatch / kRelPer;
constexpr int kRelAhead = 4;                           // columns of a lane with their loads in flight (8: 30 us for 4096 x 640 pages)

struct ReleaseParams {
  const int32_t *old_lens, *new_lens, *req;
  int B;
  const int32_t* table;
  int32_t* page_table;
  int rows, max_pages;
  int32_t* free_pages;
  int free_len;
  const int32_t* free_range;
  int num_pages, move;
  int32_t *out, *lens_out, *range_out;
  int32_t* dev_err;
};

__device__ __forceinline__ int pages_of(int tokens) { return (int)(((int64_t)tokens + kPage - 1) / kPage); }
// Where entry b of a per-request array lies: a thread's requests are contiguous,
// so 32 threads write every 4th entry; shifted like this they fall in 32 banks.
__device__ __forceinline__ int spread(int b) { return b + (b >> 5); }

// kTables: writes the tables, lengths and range.  kList: writes the free list.
enum { kTables = 1, kList = 2 };

// Dynamic shared memory (entries spread): per request the pages that stay
// or come, the pages it had, its first fresh page (-1: none), the first
// place of those given back (-1: none), its row; for `move` two bits per
// persistent row (seen, seen twice).
template <int T>
__global__ void __launch_bounds__(T) release_kernel(const ReleaseParams p, int part_of) {
  extern __shared__ int32_t release_smem[];
  __shared__ int64_t red[T / 32];
  __shared__ int total_take, total_back;
  const int room = spread(p.B) + 1;
  int32_t* s_now = release_smem;
  int32_t* s_was = s_now + room;
  int32_t* s_take = s_was + room;
  int32_t* s_back = s_take + room;
  int32_t* s_row = s_back + room;
  uint32_t* s_seen = reinterpret_cast<uint32_t*>(s_row + room);
  const int row_words = p.move ? (p.rows + 31) / 32 : 0;
  uint32_t* s_twice = s_seen + row_words;
  const int tid = threadIdx.x;
  for (int i = tid; i < 2 * row_words; i += T) s_seen[i] = 0u;
  if (tid == 0) total_take = total_back = 0;
  pdl_launch_dependents();
  pdl_wait();
  __syncthreads();

  const int per = (p.B + T - 1) / T, b0 = tid * per;
  const int cap = p.max_pages * kPage;                 // fits: the host checks it
  int was[kRelPer], now[kRelPer], row[kRelPer];
  int err = 0;
#pragma unroll
  for (int k = 0; k < kRelPer; ++k) {                  // all loads first: they are in flight together
    const bool mine = k < per && b0 + k < p.B;
    was[k] = mine ? __ldcg(p.old_lens + b0 + k) : 0;
    now[k] = mine ? __ldcg(p.new_lens + b0 + k) : 0;
    row[k] = mine && p.move ? __ldcg(p.req + b0 + k) : 0;
  }
#pragma unroll
  for (int k = 0; k < kRelPer; ++k) {
    if (!(k < per && b0 + k < p.B)) continue;
    bool ok = true;
    if (p.move) {
      if (row[k] < 0 || row[k] >= p.rows) {
        err |= MLA_DEVERR_PAGE;
        ok = false;
      } else {
        const uint32_t bit = 1u << (row[k] & 31);
        if (atomicOr(s_seen + (row[k] >> 5), bit) & bit) atomicOr(s_twice + (row[k] >> 5), bit);
      }
    }
    if (was[k] < 0 || was[k] > cap || now[k] < 0 || now[k] > was[k]) {
      err |= MLA_DEVERR_SEQLEN;
      if (was[k] < 0 || was[k] > cap) was[k] = 0;
      ok = false;
    }
    if (!ok) now[k] = was[k];                          // refused: stays as it is
  }
  __syncthreads();                                     // the rows' bits
  int64_t take_sum = 0, back_sum = 0;
  int take[kRelPer], back[kRelPer];
#pragma unroll
  for (int k = 0; k < kRelPer; ++k) {
    take[k] = back[k] = 0;
    if (!(k < per && b0 + k < p.B)) continue;
    if (p.move && row[k] >= 0 && row[k] < p.rows && ((s_twice[row[k] >> 5] >> (row[k] & 31)) & 1u)) {
      err |= MLA_DEVERR_PAGE;
      now[k] = was[k];
    }
    if (now[k] < was[k]) {
      take[k] = p.move ? pages_of(now[k]) : 0;
      back[k] = pages_of(was[k]) - (p.move ? 0 : pages_of(now[k]));
    }
    take_sum += take[k];
    back_sum += back[k];
  }
  const int head = __ldcg(p.free_range), tail = __ldcg(p.free_range + 1);
  int avail = 0, space = 0;
  if (head < 0 || tail < head || tail > p.free_len) {
    err |= MLA_DEVERR_PAGE;
  } else {
    avail = tail - head;
    space = head;
  }
  int64_t unused;
  int64_t first_take = block_scan<T>(take_sum, red, &unused);
  int64_t first_back = block_scan<T>(back_sum, red, &unused);
  int most_take = 0, most_back = 0;
#pragma unroll
  for (int k = 0; k < kRelPer; ++k) {
    const int b = b0 + k;
    if (!(k < per && b < p.B)) continue;
    const bool any = take[k] > 0 || back[k] > 0;
    // the scans count every request, so nobody behind the first one that
    // finds no page or no place gets any: what is taken and given back are runs
    const bool fits = first_take + take[k] <= avail && first_back + back[k] - first_take - take[k] <= space;
    if (any && !fits) {
      err |= MLA_DEVERR_NO_PAGES;
      now[k] = was[k];
    }
    const bool done = any && fits;
    if (done) {                                        // runs: the last one's end
      most_take = (int)first_take + take[k];
      most_back = (int)first_back + back[k];
    }
    s_take[spread(b)] = done && p.move ? (int)first_take : -1;
    s_back[spread(b)] = done && back[k] ? (int)first_back : -1;
    s_now[spread(b)] = pages_of(now[k]);
    s_was[spread(b)] = pages_of(was[k]);
    s_row[spread(b)] = row[k];
    first_take += take[k];
    first_back += back[k];
    if (blockIdx.x == 0 && (part_of & kTables)) p.lens_out[b] = now[k];
  }
  // one atomic a warp (4096 requests: one each, all on one word, 0.5 us more a launch)
  most_take = __reduce_max_sync(0xffffffffu, most_take);
  most_back = __reduce_max_sync(0xffffffffu, most_back);
  if ((tid & 31) == 0) {
    atomicMax(&total_take, most_take);
    atomicMax(&total_back, most_back);
  }
  __syncthreads();
  const int64_t to = (int64_t)head + total_take - total_back;
  if (blockIdx.x == 0 && (part_of & kTables)) {
    if (err) set_err(p.dev_err, err);
    if (tid == 0) {
      p.range_out[0] = (int)to;
      p.range_out[1] = tail;
    }
  }

  // a warp per row, or several warps on a row's columns when there are more warps
  const int lane = tid & 31;
  const int64_t warps = (int64_t)gridDim.x * T >> 5, wid = ((int64_t)blockIdx.x * T + tid) >> 5;
  const int split = (int)(warps / p.B > 1 ? warps / p.B : 1);
  const int64_t lines = warps / split;                 // rows in work at a time
  if (wid < lines * split) {
    const int part = (int)(wid % split);
    for (int64_t b = wid / split; b < p.B; b += lines) {
      const int s = spread((int)b), now_b = s_now[s], was_b = s_was[s], take_b = s_take[s], back_b = s_back[s];
      const int kept = take_b >= 0 ? 0 : now_b;        // columns below keep their pages, those given back begin here
      const int32_t* in = p.table + b * p.max_pages;
      int32_t* out = p.out + b * p.max_pages;
      const int end = part_of & kTables ? p.max_pages : (back_b >= 0 ? was_b : 0);
      for (int64_t c0 = 32 * part + lane; c0 < end; c0 += 32 * split * kRelAhead) {
        int id[kRelAhead], fresh[kRelAhead];
#pragma unroll
        for (int e = 0; e < kRelAhead; ++e) {
          const int64_t pg = c0 + 32 * split * e;
          id[e] = pg < was_b ? __ldcg(in + pg) : -1;
          fresh[e] = take_b >= 0 && pg < now_b && (part_of & kTables) ? __ldcg(p.free_pages + head + take_b + pg) : -1;
        }
#pragma unroll
        for (int e = 0; e < kRelAhead; ++e) {
          const int64_t pg = c0 + 32 * split * e;
          if (pg >= end) continue;
          if (pg < was_b && (id[e] < 0 || id[e] >= p.num_pages)) {
            set_err(p.dev_err, MLA_DEVERR_PAGE);
            id[e] = -1;
          }
          if ((part_of & kList) && back_b >= 0 && pg >= kept && pg < was_b) p.free_pages[to + back_b + pg - kept] = id[e];
          if (!(part_of & kTables)) continue;
          int mine = pg < now_b ? id[e] : -1;
          if (take_b >= 0 && pg < now_b) {
            mine = fresh[e];
            if (mine < 0 || mine >= p.num_pages) {
              set_err(p.dev_err, MLA_DEVERR_PAGE);
              mine = -1;
            }
            p.page_table[(int64_t)s_row[s] * p.max_pages + pg] = mine;
          }
          out[pg] = mine;
        }
      }
    }
  }
}

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" mla_status mla_release_pages(const int32_t* old_lens, const int32_t* new_lens, const int32_t* req,
                                        int32_t batch, const int32_t* block_table, int32_t* page_table, int32_t rows,
                                        int32_t max_pages, int32_t* free_pages, int32_t free_len,
                                        const int32_t* free_range, int32_t num_pages, int32_t move, int32_t* new_table,
                                        int32_t* lens_out, int32_t* free_range_out, int32_t* dev_err,
                                        mla_stream_t stream) {
  if (batch < 0 || batch > kMaxBatch || move < 0 || move > 1) return MLA_ERR_INVALID_ARG;
  if (max_pages < 1 || (int64_t)max_pages * kPage > (int64_t)INT32_MAX) return MLA_ERR_INVALID_ARG;
  if (num_pages < 1 || (int64_t)num_pages * kPage > (int64_t)INT32_MAX || free_len < 0) return MLA_ERR_INVALID_ARG;
  if (move && (rows < 1 || rows > kPlanMaxRows)) return MLA_ERR_INVALID_ARG;
  if (batch == 0) return MLA_OK;
  if (!ok4(old_lens) || !ok4(new_lens) || !ok4(block_table) || !ok4(free_range) || !ok4(new_table) || !ok4(lens_out) ||
      !ok4(free_range_out) || (free_len > 0 && !ok4(free_pages)) || (dev_err && !ok4(dev_err)) ||
      (move && (!ok4(req) || !ok4(page_table))))
    return MLA_ERR_INVALID_ARG;
  // blocks read their inputs at any time: no output may overlap one of them, or another output
  const int64_t words = (int64_t)batch * max_pages * 4, per = (int64_t)batch * 4;
  const Range in[] = {{old_lens, per}, {new_lens, per}, {req, move ? per : 0}, {block_table, words}, {free_range, 8}};
  const Range out[] = {{new_table, words}, {lens_out, per}, {free_range_out, 8}, {free_pages, (int64_t)free_len * 4},
                       {page_table, move ? (int64_t)rows * max_pages * 4 : 0}};
  for (int o = 0; o < 5; ++o) {
    for (int i = 0; i < 5; ++i)
      if (overlap(in[i], out[o])) return MLA_ERR_INVALID_ARG;
    for (int q = 0; q < o; ++q)
      if (overlap(out[q], out[o])) return MLA_ERR_INVALID_ARG;
  }
  ReleaseParams p;
  p.old_lens = old_lens;
  p.new_lens = new_lens;
  p.req = req;
  p.B = batch;
  p.table = block_table;
  p.page_table = page_table;
  p.rows = move ? rows : 0;
  p.max_pages = max_pages;
  p.free_pages = free_pages;
  p.free_len = free_len;
  p.free_range = free_range;
  p.num_pages = num_pages;
  p.move = move;
  p.out = new_table;
  p.lens_out = lens_out;
  p.range_out = free_range_out;
  p.dev_err = dev_err;
  const size_t smem = sizeof(int32_t) * ((size_t)5 * (batch + batch / 32 + 1) + (move ? 2 * ((rows + 31) / 32) : 0));
  const bool large = batch > kRelSmall * kRelPer;
  const int block = large ? kRelLarge : kRelSmall;
  if (smem + 512 > 48 * 1024) {            // 512: at least the kernel's static shared memory
    static int configured[2][64] = {{0}};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64 || !configured[large][dev]) {
      const int most = (int)sizeof(int32_t) * (5 * (kMaxBatch + kMaxBatch / 32 + 1) + 2 * (kPlanMaxRows / 32));
      const mla_status st =
          cuda_status(cudaFuncSetAttribute(large ? release_kernel<kRelLarge> : release_kernel<kRelSmall>,
                                           cudaFuncAttributeMaxDynamicSharedMemorySize, most));
      if (st != MLA_OK) return st;
      if (dev >= 0 && dev < 64) configured[large][dev] = 1;
    }
  }
  const int sms = device_sm_count();
  const int64_t work = (int64_t)batch * max_pages;
  const int64_t want = (work + 4 * block - 1) / (4 * block);
  const int64_t most = sms > 0 ? (large ? sms : 2 * sms) : 1;
  const int grid = (int)(want < 1 ? 1 : (want < most ? want : most));
  auto launch = [&](int part_of) {
    return cuda_status(launch_pdl(large ? release_kernel<kRelLarge> : release_kernel<kRelSmall>, dim3(grid), dim3(block), smem,
                                  (cudaStream_t)stream, p, part_of));
  };
  if (!move) return launch(kTables | kList);
  const mla_status st = launch(kTables);
  return st != MLA_OK ? st : launch(kList);
}
