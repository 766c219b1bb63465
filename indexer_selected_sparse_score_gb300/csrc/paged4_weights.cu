// The attention weight that every slot of a 4-bit cache gathers in a call: the sum
// over the call's tokens and the heads of a KV head of exp(logit - lse).
//
// Keys stay, queries pass: 32 slots belong to one warp, which takes every token of
// the sequence's run of tokens against them, so a slot's sum has one owner and one
// order, and warps need nothing of each other.  A warp turns the codes of its slots
// into fp16 operands in registers (layout as in paged4_attn.cu) and takes eight
// columns (token, head) at a time:
//   S^T = K Q^T, M = 16 keys, N = 8 columns, K = D;  w = 2^(S cs - lse log2 e)
// Its codes come through a ring of its own by asynchronous copies.  A decode step is
// bound by HBM and issue (72 bytes of codes a slot and KV head at D = 128, and its record
// read and written): 64 sequences of 2 .. 8 K slots and 8 heads 49 us, 4.3 TB/s, 62% of the
// issue slots.  (Sixteen slots a step and the CTA's eight warps in step: 72 us.)
#include <algorithm>

#include "internal.h"
#include "paged4_mma.cuh"
#include "paged4_units.cuh"
#include "paged_umma.cuh"

namespace sa {
namespace {

using namespace umma;

constexpr int kTile = 32;                // slots of a warp's step
constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kCtasPerSm = 2;            // 16 warps of 128 registers (three CTAs spill: 55 us against 49)
constexpr int kStages = 4;               // tiles that a warp has in its ring
// Columns of a unit, on average; more: paged4_weights_umma.cu.  64 sequences of 8 .. 16 K slots
// and one KV head, every call with a cold L2: 16 columns 45 us here and 141 there, 32 74 and 148,
// 64 129 and 162, 96 184 and 100, 128 240 and 102.  16 sequences of 512 .. 1024 slots: 32
// columns 14 and 23 us, 64 18 and 23, 96 23 and 23, 128 27 and 25; one of 100 slots: 64 18 and 21, 96
// 25 and 23, so the border does not move with the slots.
constexpr int kMostColumns = 64;
constexpr int kRunsInSmem = 256;         // tokens whose runs a CTA works out by itself

struct WeightsParams {
  Paged4View c;
  const uint16_t *q;
  const float *lse;
  float *weight;
  int64_t ld;
  Runs runs;  // in global memory (T above kRunsInSmem), planned by plan_kernel
  int *n_runs;
  int group;
  float qk_scale;
  uint32_t *status;
};

template <int kDim>
struct WeightsSmem {
  static constexpr uint32_t kCodes = kTile * kDim / 2, kScales = kTile * kDim / 16;
  static constexpr uint32_t kStage = kCodes + kScales;
  static constexpr size_t scan = static_cast<size_t>(kWarps) * kStages * kStage;
  static constexpr size_t off = scan + 32 * 8;
  static constexpr size_t t0 = off + (kRunsInSmem + 1) * 8;
  static constexpr size_t last = t0 + (kRunsInSmem + 2) * 4;
  static constexpr size_t total = last + kRunsInSmem * 4;
  static_assert(t0 % 8 == 0 && (total + 1024) * kCtasPerSm <= 228 * 1024, "layout");
};

__global__ void __launch_bounds__(1024) plan_kernel(const PagedView v, const Runs r, int *n_runs, uint32_t *status) {
  __shared__ long long warp_s[32];
  const int n = plan_runs(v, kTile, warp_s, r, status);
  if (threadIdx.x == 0) *n_runs = n;
}

template <int kDim>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
weights4_kernel(const WeightsParams p) {
  using L = WeightsSmem<kDim>;
  constexpr int kFr = kDim / 32;
  extern __shared__ __align__(128) uint8_t smem[];
  const PagedView &pv = p.c.v;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  Runs r = p.runs;
  int runs;
  if (pv.T <= kRunsInSmem) {
    r = Runs{reinterpret_cast<int *>(smem + L::t0), reinterpret_cast<int *>(smem + L::last),
             reinterpret_cast<long long *>(smem + L::off)};
    runs = plan_runs(pv, kTile, reinterpret_cast<long long *>(smem + L::scan), r, blockIdx.x == 0 ? p.status : nullptr);
  } else {
    runs = *p.n_runs;
  }
  const long long total = r.off[runs];
  // warp w of all takes the tiles total * w / warps ..: a CTA's are far apart, so that
  // the warps of an SM do not end together
  const int workers = gridDim.x * kWarps, me = warp * gridDim.x + blockIdx.x;
  long long x = total * me / workers;
  const long long x1 = total * (me + 1) / workers;
  if (x >= x1) return;

  const int g = lane >> 2, tq = lane & 3;
  uint8_t *ring = smem + warp * kStages * L::kStage;
  const uint32_t ring_s = smem_u32(ring);
  uint4 qr[kFr];
  float cs[2], ls[2];
  int lim[2];
  // Columns 8 c .. 8 c + 7 of a unit: fragments of the column g, and the factor,
  // logarithm and limit of columns 2 t and 2 t + 1.
  auto load_columns = [&](int t0, int ncols, int hk, int c) {
    const int col = 8 * c + g;
    const bool in = col < ncols;
    const int i = in ? col / p.group : 0, h = in ? hk * p.group + col - i * p.group : 0;
    const uint4 *src =
        reinterpret_cast<const uint4 *>(p.q + (static_cast<int64_t>(t0 + i) * pv.H + h) * kDim + kDim / 4 * tq);
    float l = 0.f, top = 0.f;
    int pos = -1;
    if (in) {
      l = p.lse[static_cast<int64_t>(t0 + i) * pv.H + h] * kLog2e;
      pos = pv.q_pos[t0 + i];
    }
#pragma unroll
    for (int j = 0; j < kFr; ++j) qr[j] = in ? src[j] : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int j = 0; j < kFr; ++j) {
      const uint32_t u[4] = {qr[j].x, qr[j].y, qr[j].z, qr[j].w};
#pragma unroll
      for (int e = 0; e < 4; ++e)
        top = fmaxf(top, fmaxf(fabsf(__uint_as_float(u[e] << 16)), fabsf(__uint_as_float(u[e] & 0xFFFF0000u))));
    }
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const float f = to_half_factor(top), own = p.qk_scale / f;
#pragma unroll
    for (int j = 0; j < kFr; ++j) {
      uint32_t u[4] = {qr[j].x, qr[j].y, qr[j].z, qr[j].w};
#pragma unroll
      for (int e = 0; e < 4; ++e)
        u[e] = as_u32(__floats2half2_rn(__uint_as_float(u[e] << 16) * f, __uint_as_float(u[e] & 0xFFFF0000u) * f));
      qr[j] = make_uint4(u[0], u[1], u[2], u[3]);
    }
    // (column g's factor and row are in the lanes of group g; a row whose lse is -inf
    // adds nothing)
    if (pos < 0 || (pos >> pv.logP) >= pv.max_pages || l == -INFINITY) pos = -1;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int from = 4 * (2 * tq + e);
      cs[e] = __shfl_sync(0xffffffffu, own, from);
      ls[e] = __shfl_sync(0xffffffffu, l, from);
      lim[e] = __shfl_sync(0xffffffffu, pos, from);
    }
  };
  for (int run = run_of_tile(r.off, runs, x); x < x1; ++run) {
    const int last = r.last[run], cost = (last + kTile) / kTile;
    if (cost == 0) continue;
    const int t0 = r.t0[run], n = r.t0[run + 1] - t0, seq = pv.q_seq[t0];
    const int ncols = n * p.group, groups = (ncols + 7) / 8;
    const TilePlace place = tile_place(x - r.off[run], cost);
    int hk = place.head, kt0 = place.tile;
    for (; hk < pv.H_kv && x < x1; ++hk, kt0 = 0) {
      const int count = static_cast<int>(min(static_cast<long long>(cost - kt0), x1 - x));
      x += count;
      // lane l: the page of the l-th 16 slots from here on, two of each tile
      auto load_ids = [&](int i) {
        const int slot = kTile * (kt0 + i + (lane >> 1)) + 16 * (lane & 1);
        if (i + (lane >> 1) >= count || slot > last) return -1;
        return load_page(pv, seq, slot >> pv.logP, p.status, true);
      };
      int ids = load_ids(0), ids_next = -1;
      uint32_t held = __ballot_sync(0xffffffffu, ids >= 0), held_now = held;
      auto copy = [&](int i) {
        if (i < count) {
          const int id0 = __shfl_sync(0xffffffffu, ids, (2 * i) & 31), id1 = __shfl_sync(0xffffffffu, ids, (2 * i + 1) & 31);
          const uint32_t st = ring_s + (i % kStages) * L::kStage;
          const int slot = kTile * (kt0 + i);
          const int64_t row0 = (static_cast<int64_t>(max(id0, 0) * pv.H_kv + hk) << pv.logP) + (slot & (pv.P - 1));
          const int64_t row1 = (static_cast<int64_t>(max(id1, 0) * pv.H_kv + hk) << pv.logP) + ((slot + 16) & (pv.P - 1));
          const uint32_t b0 = id0 >= 0 ? 16u : 0u, b1 = id1 >= 0 ? 16u : 0u;
          const uint8_t *s0 = p.c.K + row0 * (kDim / 2) + 16 * lane, *s1 = p.c.K + row1 * (kDim / 2) + 16 * lane;
#pragma unroll
          for (int e = 0; e < kDim / 64; ++e) {
            cp_async16_or_zero(st + 16 * lane + 512 * e, s0 + 512 * e, b0);
            cp_async16_or_zero(st + 16 * lane + 8 * kDim + 512 * e, s1 + 512 * e, b1);
          }
          constexpr int kSc = kDim / 16;  // chunks of the scales of 16 rows
          if (lane < 2 * kSc)
            cp_async16_or_zero(st + L::kCodes + 16 * lane,
                               p.c.Ks + (lane < kSc ? row0 : row1) * (kDim / 16) + 16 * (lane % kSc), lane < kSc ? b0 : b1);
        }
        cp_async_commit();
      };
#pragma unroll
      for (int i = 0; i < kStages - 1; ++i) copy(i);
      if (groups == 1) load_columns(t0, ncols, hk, 0);
      float *weight = p.weight + (static_cast<int64_t>(seq) * pv.H_kv + hk) * p.ld;
#pragma unroll 1
      for (int i = 0; i < count; ++i) {
        const int ahead = i + kStages - 1;
        if ((ahead & 15) == 0) {
          ids = ids_next;
          held = __ballot_sync(0xffffffffu, ids >= 0);
        }
        if ((i & 15) == 0) held_now = held;  // (ahead is among the same)
        cp_async_wait<kStages - 2>();
        __syncwarp();
        copy(ahead);
        if ((ahead & 15) == 4) ids_next = load_ids(ahead - 4 + 16);
        const int base = kTile * (kt0 + i);
        const uint32_t halves = (held_now >> (2 * (i & 15))) & 3u;
        if (!halves) continue;
        const uint8_t *st = ring + (i % kStages) * L::kStage;
        KeyRows<kDim> rows[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) rows[h].load(st + h * (8 * kDim), st + L::kCodes + h * kDim, g, tq);
        float sum[4] = {};  // of rows g, g + 8, g + 16, g + 24
        for (int c = 0; c < groups; ++c) {
          if (groups > 1) load_columns(t0, ncols, hk, c);
          float acc[2][4] = {};
#pragma unroll
          for (int j = 0; j < kFr; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              __half2 a[4], b[4];
              rows[h].values(0, j, a);
              rows[h].values(1, j, b);
              mma_16816(acc[h], as_u32(a[0]), as_u32(b[0]), as_u32(a[1]), as_u32(b[1]), qr[j].x, qr[j].y);
              mma_16816(acc[h], as_u32(a[2]), as_u32(b[2]), as_u32(a[3]), as_u32(b[3]), qr[j].z, qr[j].w);
            }
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float w = exp2_fast(fmaf(acc[h][e], cs[e & 1], -ls[e & 1]));
              if (base + 16 * h + g + 4 * (e & 2) <= lim[e & 1]) sum[2 * h + (e >> 1)] += w;
            }
        }
        // over the columns; lane (g, t) gets row g + 8 t
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], 1);
          sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], 2);
        }
        const float own = tq == 0 ? sum[0] : tq == 1 ? sum[1] : tq == 2 ? sum[2] : sum[3];
        const int slot = base + g + 8 * tq;
        // one addition a slot and run (a sequence in several runs adds in any order)
        if (slot <= last && ((halves >> (tq >> 1)) & 1u)) atomicAdd(weight + slot, own);
      }
      cp_async_wait<0>();
      __syncwarp();
    }
  }
}

size_t round_up(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

template <int kDim>
cudaError_t launch(const WeightsParams &p, cudaStream_t stream) {
  auto kern = weights4_kernel<kDim>;
  static bool done[64] = {};
  const cudaError_t e = set_smem_once(reinterpret_cast<const void *>(kern), WeightsSmem<kDim>::total, done);
  if (e != cudaSuccess) return e;
  return launch_ex(false, kern, dim3(kCtasPerSm * sm_count()), dim3(kThreads), WeightsSmem<kDim>::total, stream, 1, p);
}

}  // namespace

size_t weights4_scratch(const sa_paged4_args &pa) {
  if (columns_of(pa) > kMostColumns) return weights4_umma_scratch(pa);
  return round_up((static_cast<size_t>(pa.p.T) + 2) * 8) + 2 * round_up((static_cast<size_t>(pa.p.T) + 2) * 4) + 256;
}

cudaError_t launch_weights4(const sa_paged4_args &pa, const void *q, const float *lse, float *weight, int64_t ld,
                            void *scratch, uint32_t *status, cudaStream_t stream) {
  if (pa.p.T == 0) return cudaSuccess;
  if (columns_of(pa) > kMostColumns) return launch_weights4_umma(pa, q, lse, weight, ld, scratch, status, stream);
  WeightsParams p;
  p.c = paged4_view(pa);
  p.q = static_cast<const uint16_t *>(q);
  p.lse = lse;
  p.weight = weight;
  p.ld = ld;
  char *w = static_cast<char *>(scratch);
  const size_t n8 = round_up((static_cast<size_t>(pa.p.T) + 2) * 8), n4 = round_up((static_cast<size_t>(pa.p.T) + 2) * 4);
  p.runs = Runs{reinterpret_cast<int *>(w + n8), reinterpret_cast<int *>(w + n8 + n4), reinterpret_cast<long long *>(w)};
  p.n_runs = reinterpret_cast<int *>(w + n8 + 2 * n4);
  p.group = pa.p.H / pa.p.H_kv;
  p.qk_scale = pa.p.scale * pa.k_gain * kLog2e;
  p.status = status;
  if (pa.p.T > kRunsInSmem) {
    const cudaError_t e = launch_ex(false, plan_kernel, dim3(1), dim3(1024), 0, stream, 1, p.c.v, p.runs, p.n_runs, status);
    if (e != cudaSuccess) return e;
  }
  return pa.p.D == 128 ? launch<128>(p, stream) : launch<64>(p, stream);
}

}  // namespace sa
