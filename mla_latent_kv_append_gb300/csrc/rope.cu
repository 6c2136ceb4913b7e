// mla_rope: rotary positions on the RoPE parts of queries and keys, with one
// to four position axes.
//
// Pair i (i < 32) of a 64-channel row turns by t = pos[axis(i)] f_i:
//   y1 = a (x1 cos t - x2 sin t),  y2 = a (x1 sin t + x2 cos t),
// or by -t for the inverse, which is the transposed rotation and so also the
// gradient.  Pairs are channels (2i, 2i + 1) or (i, i + 32).
//
// Angles.  pos f_i reaches 10^6 radians and more, where an fp32 product is
// off by whole tenths of a radian.  The turn count pos f_i / (2 pi) is kept
// as a 64-bit fixed-point fraction instead: G_i = frac(f_i / (2 pi)) 2^64 is
// computed once per lane in fp64, pos * G_i wraps modulo 2^64 = one turn on
// its own, and the top 32 bits are the angle to 2^-31 of a half turn.  The
// fp64 quotient is off by 2^-52 relative (1 / (2 pi) and the product, rounded), so
// an angle is off by 2^-52 |pos f| radians, and by 1e-7 through its conversion to
// fp32: 6e-7 at position 2^31 for f = 1, far below bf16.
//
// What bounds it: reading and writing N (H + 1) rows of 128 bytes.  A warp
// takes a token (or a run of its heads); lane i computes pair i's cosine and
// sine once, the lanes then exchange them by shuffles and every lane turns
// 16-byte pieces, four heads per sweep of the warp.  Warps stride over the
// tokens, so the fp64 constant is paid once per warp.
//
// Measured: 8192 tokens x 128 heads (271 MB) 47 us, 5.8 TB/s or 85% of a plain
// copy's rate; 1999 tokens x 64 heads, pairs in halves (33 MB, which L2 holds), 10.6
// us; 8 tokens x 16 heads 2.7 us, latency.
#include <math.h>

#include "mla_internal.cuh"

namespace mla {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopePairs = kDr / 2;          // 32: one per lane
constexpr int kRopeUnroll = 4;               // sweeps whose loads are in flight together

struct RopeParams {
  const uint16_t* q;
  const uint16_t* k;
  uint16_t* qo;
  uint16_t* ko;
  int64_t q_tok, q_head, k_tok, qo_tok, qo_head, ko_tok;   // strides in elements
  const int32_t* pos;       // [axes][n]
  const float* inv_freq;    // [32]
  uint64_t axis;            // 2 bits per pair
  int n, H;
  int rows;                 // H, plus one when there is a key
  int groups;               // a token's rows are cut into this many runs
  float amp;
  int inverse;
};

__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;\n" : "=r"(r) : "f"(b), "f"(a));
  return r;
}

template <bool INTERLEAVED>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t warps = (int64_t)gridDim.x * (kRopeThreads / 32);
  pdl_launch_dependents();
  pdl_wait();
  const double turns = (double)p.inv_freq[lane] * 0.15915494309189533577;    // f / (2 pi)
  const uint64_t G = (uint64_t)((turns - floor(turns)) * 18446744073709551616.0);
  const int axis = (int)((p.axis >> (2 * lane)) & 3);
  // this lane's 16-byte pieces: interleaved, piece lane % 8 of head lane / 8
  // (4 pairs); halves, pieces lane % 4 and lane % 4 + 4 of head lane / 4 (8
  // pairs, a half of the head's 128 bytes each)
  constexpr int kPer = INTERLEAVED ? 4 : 8;          // pairs per lane, and heads per sweep
  const int piece = lane & (32 / kPer - 1), sub = lane / (32 / kPer);
  for (int64_t w = ((int64_t)blockIdx.x * kRopeThreads + threadIdx.x) >> 5; w < (int64_t)p.n * p.groups; w += warps) {
    const int tok = (int)(w / p.groups), g = (int)(w % p.groups);
    const int r_lo = (int)((int64_t)p.rows * g / p.groups), r_hi = (int)((int64_t)p.rows * (g + 1) / p.groups);
    const int64_t at = __ldcg(p.pos + (int64_t)axis * p.n + tok);
    uint4 a[kRopeUnroll], b[kRopeUnroll];
    auto fetch = [&](int r0) {
#pragma unroll
      for (int u = 0; u < kRopeUnroll; ++u) {
        const int r = r0 + u * kPer + sub;
        if (r < r_hi) {
          const uint16_t* src = r < p.H ? p.q + tok * p.q_tok + r * p.q_head : p.k + tok * p.k_tok;
          a[u] = __ldcg(reinterpret_cast<const uint4*>(src + 8 * piece));
          if (!INTERLEAVED) b[u] = __ldcg(reinterpret_cast<const uint4*>(src + kRopePairs + 8 * piece));
        }
      }
    };
    fetch(r_lo);                           // under way while the angles are computed
    const int32_t half_turns = (int32_t)(uint32_t)(((uint64_t)at * G) >> 32);   // units of 2^-31 half turns
    float sn, cs;
    sincospif((float)half_turns * 0x1p-31f, &sn, &cs);
    cs *= p.amp;
    sn *= p.inverse ? -p.amp : p.amp;
    float c[kPer], s[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      c[i] = __shfl_sync(0xffffffffu, cs, kPer * piece + i);
      s[i] = __shfl_sync(0xffffffffu, sn, kPer * piece + i);
    }
    for (int r0 = r_lo; r0 < r_hi; r0 += kPer * kRopeUnroll) {
      if (r0 > r_lo) fetch(r0);
#pragma unroll
      for (int u = 0; u < kRopeUnroll; ++u) {
        const int r = r0 + u * kPer + sub;
        if (r >= r_hi) continue;
        uint16_t* dst = r < p.H ? p.qo + tok * p.qo_tok + r * p.qo_head : p.ko + tok * p.ko_tok;
        uint32_t x[4] = {a[u].x, a[u].y, a[u].z, a[u].w};
        if (INTERLEAVED) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float x1 = bf16lo(x[i]), x2 = bf16hi(x[i]);
            x[i] = bf16_pair(x1 * c[i] - x2 * s[i], x1 * s[i] + x2 * c[i]);
          }
          *reinterpret_cast<uint4*>(dst + 8 * piece) = make_uint4(x[0], x[1], x[2], x[3]);
        } else {
          uint32_t y[4] = {b[u].x, b[u].y, b[u].z, b[u].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float l1 = bf16lo(x[i]), h1 = bf16hi(x[i]), l2 = bf16lo(y[i]), h2 = bf16hi(y[i]);
            x[i] = bf16_pair(l1 * c[(2 * i) % kPer] - l2 * s[(2 * i) % kPer],
                             h1 * c[(2 * i + 1) % kPer] - h2 * s[(2 * i + 1) % kPer]);
            y[i] = bf16_pair(l1 * s[(2 * i) % kPer] + l2 * c[(2 * i) % kPer],
                             h1 * s[(2 * i + 1) % kPer] + h2 * c[(2 * i + 1) % kPer]);
          }
          *reinterpret_cast<uint4*>(dst + 8 * piece) = make_uint4(x[0], x[1], x[2], x[3]);
          *reinterpret_cast<uint4*>(dst + kRopePairs + 8 * piece) = make_uint4(y[0], y[1], y[2], y[3]);
        }
      }
    }
  }
}

bool ok16(const void* p) { return p && ((uintptr_t)p & 15) == 0; }

// Rows of 64 elements at i s1 + j s2 (i < n1, j < n2) do not overlap.
bool apart(int64_t n1, int64_t s1, int64_t n2, int64_t s2) {
  if (n1 == 1 && n2 == 1) return true;
  if (n1 == 1) return s2 >= kDr;
  if (n2 == 1) return s1 >= kDr;
  const bool one = s1 <= s2;
  const int64_t lo = one ? s1 : s2, nlo = one ? n1 : n2, hi = one ? s2 : s1;
  return lo >= kDr && hi >= (nlo - 1) * lo + kDr;
}

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" mla_status mla_rope(const uint16_t* q_pe, int64_t q_token_stride, int64_t q_head_stride,
                               const uint16_t* k_pe, int64_t k_token_stride, const int32_t* positions, int32_t axes,
                               const uint8_t* pair_axis, const float* inv_freq, int32_t n, int32_t heads,
                               int32_t interleaved, int32_t inverse, float amplitude, uint16_t* q_out,
                               int64_t qo_token_stride, int64_t qo_head_stride, uint16_t* k_out,
                               int64_t ko_token_stride, mla_stream_t stream) {
  if (n < 0 || heads < 0 || heads > 128 || axes < 1 || axes > 4 || !isfinite(amplitude)) return MLA_ERR_INVALID_ARG;
  if ((interleaved & ~1) || (inverse & ~1)) return MLA_ERR_INVALID_ARG;
  if ((k_pe == nullptr) != (k_out == nullptr)) return MLA_ERR_INVALID_ARG;
  uint64_t axis = 0;
  for (int i = 0; i < kRopePairs; ++i) {
    const int a = pair_axis ? pair_axis[i] : 0;
    if (a >= axes) return MLA_ERR_INVALID_ARG;
    axis |= (uint64_t)a << (2 * i);
  }
  const int64_t strides[6] = {q_token_stride, q_head_stride, k_token_stride, qo_token_stride, qo_head_stride,
                              ko_token_stride};
  for (int i = 0; i < 6; ++i)
    if (strides[i] < 0 || strides[i] % 8) return MLA_ERR_INVALID_ARG;
  const int rows = heads + (k_pe ? 1 : 0);
  if (n == 0 || rows == 0) return MLA_OK;
  if (!positions || ((uintptr_t)positions & 3) || !inv_freq || ((uintptr_t)inv_freq & 3)) return MLA_ERR_INVALID_ARG;
  if (heads > 0 && (!ok16(q_pe) || !ok16(q_out) || !apart(n, qo_token_stride, heads, qo_head_stride)))
    return MLA_ERR_INVALID_ARG;
  if (k_pe && (!ok16(k_pe) || !ok16(k_out) || !apart(n, ko_token_stride, 1, kDr))) return MLA_ERR_INVALID_ARG;
  RopeParams p;
  p.q = q_pe;
  p.k = k_pe;
  p.qo = q_out;
  p.ko = k_out;
  p.q_tok = q_token_stride;
  p.q_head = q_head_stride;
  p.k_tok = k_token_stride;
  p.qo_tok = qo_token_stride;
  p.qo_head = qo_head_stride;
  p.ko_tok = ko_token_stride;
  p.pos = positions;
  p.inv_freq = inv_freq;
  p.axis = axis;
  p.n = n;
  p.H = heads;
  p.rows = rows;
  p.amp = amplitude;
  p.inverse = inverse;
  const int sms = device_sm_count() > 0 ? device_sm_count() : 1;
  const int64_t full = (int64_t)sms * 8 * (kRopeThreads / 32);      // warps of a full GPU
  // a token's rows are split over several warps only while warps are idle
  int groups = (int)(full / n);
  const int most = (rows + 15) / 16;
  groups = groups < 1 ? 1 : (groups > most ? most : groups);
  p.groups = groups;
  const int64_t blocks = ((int64_t)n * groups + kRopeThreads / 32 - 1) / (kRopeThreads / 32);
  const int grid = (int)(blocks < (int64_t)sms * 8 ? blocks : (int64_t)sms * 8);
  const cudaStream_t st = (cudaStream_t)stream;
  if (interleaved) return cuda_status(launch_pdl(rope_kernel<true>, dim3(grid), dim3(kRopeThreads), 0, st, p));
  return cuda_status(launch_pdl(rope_kernel<false>, dim3(grid), dim3(kRopeThreads), 0, st, p));
}
