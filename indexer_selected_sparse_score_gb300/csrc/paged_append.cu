// New keys and values into the pages of a paged cache, rotary embedding on the
// way, the queries rotated alongside, and the mean key of every page that fills.
//
// Rotation: pair i turns by p f_i.  The frequency is held as a 64-bit fraction
// of a turn, F = f / (2 pi) 2^64, so p F modulo 2^64 is the angle modulo a turn
// by one integer product (the wrap-around is the reduction), exact to p 2^-53
// of F for any 31-bit position; its upper 32 bits go to fp32 as half turns
// (error below 2^-24 of a half turn) and to sincospif.  A reduction in double
// would be limited by the part's FP64 rate (two operations a clock per SM).
//
// Traffic: every row is read once and written once (2 T (H + 2 H_kv) D values),
// bound by HBM for a prefill and by latency for a decode step.  One CTA per
// token: every thread issues its rows' loads, then a part of the block finds
// the token's page and tables the rotations in shared memory, and 32-byte units
// (two 16-byte chunks, the two halves of their pairs) leave through registers.
// The means are a second kernel that starts in the first one's tail: a page may
// fill from tokens of any CTA, and its rows are still in L2.
//
// Measured, 64 query and 8 KV heads of 128, means included: 64 tokens of a
// decode step 8 to 12 us (two launches and a chain of dependent loads); a ragged
// prefill of 10,907 tokens 90 us, 5.0 TB/s of the 449 MB it must move (the first
// kernel about 5.7 TB/s, the means 11 us).  4096 tokens of 64 + 1 heads: 35 us,
// 4.0 TB/s.  A persistent grid that overlapped the next token's loads with this
// one's stores measured 120 us against 95 on the prefill.
#include <algorithm>
#include <cmath>

#include "internal.h"
#include "paged.cuh"

namespace sa {
namespace {

constexpr int kThreads = 320;     // append, at most: two units a thread at 64 + 2 x 8 heads of dim 128
constexpr int kMeanThreads = 256, kMeanHeads = 2;
constexpr int kMaxPairs = 64;

struct Turns {
  uint64_t f[kMaxPairs];  // turns per position, times 2^64
};

struct AppendParams {
  PagedView pv;
  const uint16_t *k, *v, *q;
  int64_t k_stride, v_stride, q_stride;
  uint16_t *K, *V, *q_out;
  int q_heads;   // H, or 0 without queries
  int D, dim;
  int halves;
  uint32_t *status;
};

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 r = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Four adjacent pairs of one chunk.
__device__ __forceinline__ uint4 rotate_adjacent(uint4 x, const float2 *cs) {
  uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 c = cs[i];
    const float a = lo_f(w[i]), b = hi_f(w[i]);
    w[i] = pack_bf16(a * c.x - b * c.y, a * c.y + b * c.x);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Eight pairs (x[e], y[e]) of two chunks half the rotated span apart.
__device__ __forceinline__ void rotate_halves(uint4 &x, uint4 &y, const float2 *cs) {
  uint32_t u[4] = {x.x, x.y, x.z, x.w}, w[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 c0 = cs[2 * i], c1 = cs[2 * i + 1];
    const float a0 = lo_f(u[i]), a1 = hi_f(u[i]), b0 = lo_f(w[i]), b1 = hi_f(w[i]);
    u[i] = pack_bf16(a0 * c0.x - b0 * c0.y, a1 * c1.x - b1 * c1.y);
    w[i] = pack_bf16(a0 * c0.y + b0 * c0.x, a1 * c1.y + b1 * c1.x);
  }
  x = make_uint4(u[0], u[1], u[2], u[3]);
  y = make_uint4(w[0], w[1], w[2], w[3]);
}

__global__ void __launch_bounds__(kThreads, 4)
paged_append_kernel(const AppendParams p, const __grid_constant__ Turns turns) {
  __shared__ float2 cs[kMaxPairs];
  pdl_trigger();
  const int t = blockIdx.x;
  const int log_upr = p.D == 128 ? 3 : 2;   // of the 32-byte units per row
  const int kept = (p.D - p.dim) >> 4;      // units before the rotated span
  const int span = p.dim >> 3;              // chunks of the rotated span
  const int first = (p.D >> 3) - span;      // first rotated chunk
  const int units = (p.q_heads + 2 * p.pv.H_kv) << log_upr;
  // chunks of unit u within its row: two neighbours, or the two halves of
  // eight pairs
  auto chunks = [&](int u, int &c0, int &c1) {
    const int i = u & ((1 << log_upr) - 1), j = i - kept;
    const bool half = p.halves && j >= 0;
    c0 = half ? first + j : 2 * i;
    c1 = half ? c0 + (span >> 1) : 2 * i + 1;
  };
  // units a thread has in flight (3 of 256 threads and 1 of 640 measured 2 and
  // 12 % slower on a prefill; five blocks of 320 per SM instead of four spill
  // registers: 91 us against 90, three leave too little in flight: 100)
  constexpr int kUnits = 2;
  bool ok = false;
  int page = -1, slot = 0;
  bool tabled = false;
  const int threads = blockDim.x;
  for (int base = 0; base < units; base += kUnits * threads) {
    // the rows' loads need no more than t: they go out before the token's
    // position and page are known
    uint4 x[kUnits], y[kUnits];
#pragma unroll
    for (int e = 0; e < kUnits; ++e) {
      const int u = base + e * threads + threadIdx.x;
      if (u >= units) continue;
      int c0, c1;
      chunks(u, c0, c1);
      const int row = u >> log_upr, h = row - p.q_heads;
      const uint16_t *src = h < 0           ? p.q + t * p.q_stride + static_cast<int64_t>(row) * p.D
                            : h < p.pv.H_kv ? p.k + t * p.k_stride + static_cast<int64_t>(h) * p.D
                                            : p.v + t * p.v_stride + static_cast<int64_t>(h - p.pv.H_kv) * p.D;
      x[e] = *reinterpret_cast<const uint4 *>(src + 8 * c0);
      y[e] = *reinterpret_cast<const uint4 *>(src + 8 * c1);
    }
    if (!tabled) {
      int b, pos;
      ok = load_paged_token(p.pv, t, p.status, threadIdx.x == 0, b, pos);
      if (ok) {
        page = load_page(p.pv, b, pos >> p.pv.logP, p.status, threadIdx.x == 0);
        slot = pos & (p.pv.P - 1);
        if (threadIdx.x < p.dim / 2) {
          const uint64_t ph = static_cast<uint64_t>(pos) * turns.f[threadIdx.x] + (uint64_t{1} << 31);
          float sn, c;
          sincospif(static_cast<float>(static_cast<int32_t>(ph >> 32)) * 0x1p-31f, &sn, &c);
          cs[threadIdx.x] = make_float2(c, sn);
        }
      }
      __syncthreads();
      tabled = true;
    }
    if (!ok) return;  // the whole CTA alike
#pragma unroll
    for (int e = 0; e < kUnits; ++e) {
      const int u = base + e * threads + threadIdx.x;
      if (u >= units) continue;
      int c0, c1;
      chunks(u, c0, c1);
      const int row = u >> log_upr, h = row - p.q_heads;
      uint16_t *dst;
      if (h < 0) {
        dst = p.q_out + (static_cast<int64_t>(t) * p.pv.H + row) * p.D;
      } else {
        if (page < 0) continue;
        const int hk = h < p.pv.H_kv ? h : h - p.pv.H_kv;
        dst = (h < p.pv.H_kv ? p.K : p.V) +
              ((static_cast<int64_t>(page) * p.pv.H_kv + hk) * p.pv.P + slot) * p.D;
      }
      if (h < p.pv.H_kv && c0 >= first) {
        if (p.halves) {
          rotate_halves(x[e], y[e], cs + 8 * (c0 - first));
        } else {
          x[e] = rotate_adjacent(x[e], cs + 4 * (c0 - first));
          y[e] = rotate_adjacent(y[e], cs + 4 * (c1 - first));
        }
      }
      *reinterpret_cast<uint4 *>(dst + 8 * c0) = x[e];
      *reinterpret_cast<uint4 *>(dst + 8 * c1) = y[e];
    }
  }
}

// Adds kLoads loads of 32 chunks each, all in flight at once.
template <int kLoads>
__device__ __forceinline__ void add_rows(const uint4 *src, float (&s)[8]) {
  uint4 x[kLoads];
#pragma unroll
  for (int e = 0; e < kLoads; ++e) x[e] = src[e * 32];
#pragma unroll
  for (int e = 0; e < kLoads; ++e) {
    const uint32_t u[4] = {x[e].x, x[e].y, x[e].z, x[e].w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      s[2 * k] += lo_f(u[k]);
      s[2 * k + 1] += hi_f(u[k]);
    }
  }
}

// Mean of the key rows of every page whose last position is among the tokens.
// CTA (x, y): tokens x * per .. + per - 1 (at most kMeanThreads), KV heads
// y * kMeanHeads .. + kMeanHeads - 1.  Its (page, head) pairs share its warps,
// one to eight of them each.  Sums are fp32, rounded to bf16 once.  It runs
// after the append has written every row, so a page may fill from tokens in any
// order; which pages those are is found before the wait.
template <int kDim>
__global__ void __launch_bounds__(kMeanThreads)
page_mean_kernel(const PagedView pv, const uint16_t *K, uint16_t *k_mean, int per) {
  constexpr int kLanes = kDim / 8, kRows = 32 / kLanes;  // lanes of a row, rows of a load
  constexpr int kWarps = kMeanThreads / 32;
  __shared__ int pages[kMeanThreads], n_s;
  __shared__ float part[kWarps][kDim];
  if (threadIdx.x == 0) n_s = 0;
  __syncthreads();
  const int own = blockIdx.x * per + threadIdx.x;
  if (threadIdx.x < per && own < pv.T) {
    int b, pos;
    if (load_paged_token(pv, own, nullptr, false, b, pos) && ((pos + 1) & (pv.P - 1)) == 0) {
      const int page = load_page(pv, b, pos >> pv.logP, nullptr, false);
      if (page >= 0) pages[atomicAdd(&n_s, 1)] = page;
    }
  }
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = lane % kLanes;
  const int h0 = blockIdx.y * kMeanHeads, heads = min(kMeanHeads, pv.H_kv - h0);
  const int items = n_s * heads, loads = pv.P / kRows;  // loads of a page (both powers of two)
  // warps of an item: a power of two; with more than one every item is in the
  // first round
  int share = 1;
  while (2 * share * items <= kWarps && 2 * share <= loads) share *= 2;
  const int each = loads / share;  // of a warp
  const int w = warp % share;      // this warp's part of the rows
  pdl_wait();
  if (items == 0) return;
  for (int it0 = 0; it0 < items; it0 += kWarps / share) {
    const int it = it0 + warp / share;
    float s[8] = {};
    int64_t tile = 0;
    if (it < items) {
      const int i = it / heads;
      tile = static_cast<int64_t>(pages[i]) * pv.H_kv + h0 + it - i * heads;
      const uint4 *src = reinterpret_cast<const uint4 *>(K + tile * pv.P * kDim) + lane;
      if (each >= 16) {
        for (int r = 0; r < each; r += 16) add_rows<16>(src + (w * each + r) * 32, s);
      } else if (each >= 4) {
        for (int r = 0; r < each; r += 4) add_rows<4>(src + (w * each + r) * 32, s);
      } else {
        for (int r = 0; r < each; ++r) add_rows<1>(src + (w * each + r) * 32, s);
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
#pragma unroll
      for (int o = kLanes; o < 32; o <<= 1) s[e] += __shfl_xor_sync(0xffffffffu, s[e], o);
    if (share > 1) {
      if (lane < kLanes) {
#pragma unroll
        for (int e = 0; e < 8; ++e) part[warp][8 * c + e] = s[e];
      }
      __syncthreads();
      if (w == 0 && lane < kLanes) {
        for (int k = 1; k < share; ++k)
#pragma unroll
          for (int e = 0; e < 8; ++e) s[e] += part[warp + k][8 * c + e];
      }
    }
    if (lane < kLanes && w == 0 && it < items) {
      const float f = 1.f / static_cast<float>(pv.P);  // exact: P is a power of two
      *reinterpret_cast<uint4 *>(k_mean + tile * kDim + 8 * c) =
          make_uint4(pack_bf16(s[0] * f, s[1] * f), pack_bf16(s[2] * f, s[3] * f), pack_bf16(s[4] * f, s[5] * f),
                     pack_bf16(s[6] * f, s[7] * f));
    }
  }
}

}  // namespace

cudaError_t launch_paged_append(const sa_paged_args &pa, const void *k, int64_t k_stride, const void *v,
                                int64_t v_stride, const void *q, int64_t q_stride, void *q_out,
                                const sa_rope_args *rope, bool halves, void *k_mean, uint32_t *status,
                                cudaStream_t stream) {
  if (pa.T == 0) return cudaSuccess;
  AppendParams p;
  p.pv = paged_view(pa);
  p.k = static_cast<const uint16_t *>(k);
  p.v = static_cast<const uint16_t *>(v);
  p.q = static_cast<const uint16_t *>(q);
  p.k_stride = k_stride ? k_stride : static_cast<int64_t>(pa.H_kv) * pa.D;
  p.v_stride = v_stride ? v_stride : static_cast<int64_t>(pa.H_kv) * pa.D;
  p.q_stride = q_stride ? q_stride : static_cast<int64_t>(pa.H) * pa.D;
  p.K = static_cast<uint16_t *>(pa.K);
  p.V = static_cast<uint16_t *>(pa.V);
  p.q_out = static_cast<uint16_t *>(q_out);
  p.q_heads = q ? pa.H : 0;
  p.D = pa.D;
  p.dim = rope ? rope->dim : 0;
  p.halves = halves ? 1 : 0;
  p.status = status;
  Turns turns{};
  const RopeRamp ramp = p.dim > 0 ? rope_ramp(*rope) : RopeRamp{0.0, 0.0};
  for (int i = 0; i < p.dim / 2; ++i) {
    const double f = rope_frequency(*rope, ramp, i) / (2.0 * 3.14159265358979323846);
    turns.f[i] = static_cast<uint64_t>(std::ldexp(f - std::floor(f), 64));
  }
  const int units = (p.q_heads + 2 * pa.H_kv) * (pa.D / 16);
  // when the tokens fill the SMs, blocks of two units a thread (7465 tokens of 40
  // rows of 128: 46 us with blocks of kThreads, 40 so); a few tokens are served by
  // the larger block sooner (8 of 32 rows of 64: 5.4 us, 6.2 with 128 threads)
  const int threads =
      pa.T > 4 * sm_count() ? std::min(std::max((units / 2 + 31) & ~31, kMaxPairs), kThreads) : kThreads;
  cudaError_t e = launch_ex(false, paged_append_kernel, dim3(pa.T), dim3(threads), 0, stream, 1, p, turns);
  if (e != cudaSuccess || !k_mean) return e;
  // one CTA per token while they are few, two CTAs per SM for more (most
  // tokens end no page), for every pair of heads
  const int per = std::min(std::max(1, pa.T / (2 * sm_count())), kMeanThreads);
  const dim3 grid((pa.T + per - 1) / per, (pa.H_kv + kMeanHeads - 1) / kMeanHeads);
  return pa.D == 128 ? launch_ex(true, page_mean_kernel<128>, grid, dim3(kMeanThreads), 0, stream, 1, p.pv,
                                 static_cast<const uint16_t *>(pa.K), static_cast<uint16_t *>(k_mean), per)
                     : launch_ex(true, page_mean_kernel<64>, grid, dim3(kMeanThreads), 0, stream, 1, p.pv,
                                 static_cast<const uint16_t *>(pa.K), static_cast<uint16_t *>(k_mean), per);
}

}  // namespace sa
