// The attention weight that every slot of a 4-bit cache gathers in a call: the sum
// over the call's tokens and the heads of a KV head of exp(logit - lse).
//
// Keys stay, queries pass: a tile of 128 slots belongs to one CTA, which takes
// every token of the sequence's run of tokens against it, so a slot's sum has one
// owner and one order.  A warp holds 16 keys as fp16 operands in registers
// (layout as in paged4_attn.cu) and takes eight columns (token, head) at a time:
//   S^T = K Q^T, M = 16 keys, N = 8 columns, K = D;  w = 2^(S cs - lse log2 e)
// A decode step is bound by HBM (72 bytes of codes a slot and KV head at D = 128,
// and its record read and written); a chunk by the products.
#include <algorithm>

#include "internal.h"
#include "paged4_mma.cuh"
#include "paged4_units.cuh"
#include "umma.cuh"

namespace sa {
namespace {

using namespace umma;

constexpr int kTile = 128;
constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps + 32;
constexpr int kRunsInSmem = 1024;  // tokens whose runs a CTA works out by itself

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

struct TileInfo {
  int t0, n, hk, b, base, last;
  uint32_t have;
  int first;
};

template <int kDim>
struct WeightsSmem {
  static constexpr int kStages = kDim == 128 ? 6 : 8;
  static constexpr uint32_t kCodes = kTile * kDim / 2, kScales = kTile * kDim / 16;
  static constexpr uint32_t kStage = kCodes + kScales;
  static constexpr size_t info = static_cast<size_t>(kStages) * kStage;
  static constexpr size_t bars = info + kStages * sizeof(TileInfo);
  static constexpr size_t scan = bars + 2 * kStages * 8;
  static constexpr size_t off = scan + 32 * 8;
  static constexpr size_t t0 = off + (kRunsInSmem + 1) * 8;
  static constexpr size_t last = t0 + (kRunsInSmem + 2) * 4;
  static constexpr size_t flag = last + kRunsInSmem * 4;
  static constexpr size_t total = flag + 16;
  static_assert(sizeof(TileInfo) % 8 == 0 && t0 % 8 == 0, "alignment");
};

__global__ void __launch_bounds__(1024) plan_kernel(const PagedView v, const Runs r, int *n_runs, uint32_t *status) {
  __shared__ long long warp_s[32];
  const int n = plan_runs(v, kTile, warp_s, r, status);
  if (threadIdx.x == 0) *n_runs = n;
}

template <int kDim>
__global__ void __launch_bounds__(kThreads, 2)
weights4_kernel(const WeightsParams p) {
  using L = WeightsSmem<kDim>;
  constexpr int kStages = L::kStages, kFr = kDim / 32;
  extern __shared__ __align__(128) uint8_t smem[];
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + L::bars), *empty = full + kStages;
  TileInfo *infos = reinterpret_cast<TileInfo *>(smem + L::info);
  volatile int *flags = reinterpret_cast<volatile int *>(smem + L::flag);
  const PagedView &pv = p.c.v;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], kWarps);
    }
    flags[0] = 0;
    fence_barrier_init();
  }
  Runs r = p.runs;
  int runs;
  if (pv.T <= kRunsInSmem) {
    r = Runs{reinterpret_cast<int *>(smem + L::t0), reinterpret_cast<int *>(smem + L::last),
             reinterpret_cast<long long *>(smem + L::off)};
    runs = plan_runs(pv, kTile, reinterpret_cast<long long *>(smem + L::scan), r, blockIdx.x == 0 ? p.status : nullptr);
  } else {
    runs = *p.n_runs;
    __syncthreads();
  }
  const long long total = r.off[runs];
  const long long x0 = total * blockIdx.x / gridDim.x, x1 = total * (blockIdx.x + 1) / gridDim.x;

  if (warp == kWarps) {
    int issued = 0;
    bool ok = true;
    if (x0 < x1) {
      int run = run_of_tile(r.off, runs, x0);
      long long x = x0;
      for (; x < x1 && ok; ++run) {
        const int last = r.last[run], cost = (last + kTile) / kTile;
        if (cost == 0) continue;
        const int t0 = r.t0[run], n = r.t0[run + 1] - t0, seq = pv.q_seq[t0];
        int rest = static_cast<int>(x - r.off[run]);
        int hk = rest / cost, kt = rest - hk * cost;
        bool fresh = true;
        for (; hk < pv.H_kv && x < x1; ++x) {
          const int s = issued % kStages;
          // lane 2 q + kind copies page q's part: codes, scales
          const int base = kt * kTile, q = lane >> 1, kind = lane & 1, from = base + (q << pv.logP);
          const int rows = min(pv.P, ((min(last - from, kTile) + 16) & ~15));
          int page = -1;
          if (q < (kTile >> pv.logP) && from <= last) page = load_page(pv, seq, from >> pv.logP, p.status, kind == 0);
          const uint32_t pages = __ballot_sync(0xffffffffu, page >= 0 && kind == 0);
          uint32_t have = 0;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) have |= ((pages >> (2 * ((16 * w) >> pv.logP))) & 1u) << w;
          const uint32_t row_bytes = kind ? kDim / 16 : kDim / 2;
          const uint32_t bytes = page >= 0 ? rows * row_bytes : 0u;
          const uint32_t sum = __reduce_add_sync(0xffffffffu, bytes);
          if (!mbar_wait_warp(&empty[s], ((issued / kStages) & 1) ^ 1) || flags[0]) {
            ok = false;
            break;
          }
          if (lane == 0) {
            infos[s] = TileInfo{t0, n, hk, seq, base, last, have, fresh};
            mbar_expect_tx(&full[s], sum);
          }
          __syncwarp();
          ++issued;
          if (bytes) {
            const int64_t at = (static_cast<int64_t>(page) * pv.H_kv + hk) * pv.P * row_bytes;
            bulk_load(smem + s * L::kStage + (kind ? L::kCodes : 0) + (q << pv.logP) * row_bytes,
                      (kind ? p.c.Ks : p.c.K) + at, bytes, &full[s]);
          }
          fresh = false;
          if (++kt == cost) {
            kt = 0;
            ++hk;
            fresh = true;
          }
        }
      }
    }
    if (lane == 0) {
      if (!ok) {
        raise_flag(p.status, kFlagTimeout);
        flags[0] = 1;
      }
      for (int m = max(0, issued - kStages); m < issued; ++m) mbar_wait(&full[m % kStages], (m / kStages) & 1);
    }
    __syncwarp();
    return;
  }

  // --------------------------------------------------------- product warps
  const int g = lane >> 2, tq = lane & 3;
  long long left = x1 - x0;
  uint4 qr[kFr] = {};
  float cs[2] = {}, ls[2] = {};
  int lim[2] = {-1, -1};
  // Columns 8 c .. 8 c + 7 of a unit: fragments of the column g, and the factor,
  // logarithm and limit of columns 2 t and 2 t + 1.
  auto load_columns = [&](int t0, int ncols, int hk, int c) {
    const int col = 8 * c + g;
    float x[kDim / 4], top = 0.f;
    const bool in = col < ncols;
    const int i = in ? col / p.group : 0, h = in ? hk * p.group + col - i * p.group : 0;
    const uint4 *src =
        reinterpret_cast<const uint4 *>(p.q + (static_cast<int64_t>(t0 + i) * pv.H + h) * kDim + kDim / 4 * tq);
#pragma unroll
    for (int j = 0; j < kFr; ++j) {
      const uint4 w = in ? src[j] : make_uint4(0, 0, 0, 0);
      const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[8 * j + 2 * e] = __uint_as_float(u[e] << 16);
        x[8 * j + 2 * e + 1] = __uint_as_float(u[e] & 0xFFFF0000u);
      }
    }
#pragma unroll
    for (int e = 0; e < kDim / 4; ++e) top = fmaxf(top, fabsf(x[e]));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const float f = to_half_factor(top), own = p.qk_scale / f;
#pragma unroll
    for (int j = 0; j < kFr; ++j) {
      uint32_t u[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) u[e] = as_u32(__floats2half2_rn(x[8 * j + 2 * e] * f, x[8 * j + 2 * e + 1] * f));
      qr[j] = make_uint4(u[0], u[1], u[2], u[3]);
    }
    // (column g's factor and row are in the lanes of group g)
    float l = 0.f;
    int pos = -1;
    if (in) {
      const int t = t0 + i;
      l = p.lse[static_cast<int64_t>(t) * pv.H + h] * kLog2e;
      const int at = pv.q_pos[t];
      if (l != -INFINITY && at >= 0 && (at >> pv.logP) < pv.max_pages) pos = at;
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int from = 4 * (2 * tq + e);
      cs[e] = __shfl_sync(0xffffffffu, own, from);
      ls[e] = __shfl_sync(0xffffffffu, l, from);
      lim[e] = __shfl_sync(0xffffffffu, pos, from);
    }
  };
  bool ok = true;
  for (int n = 0; left > 0; ++n, --left) {
    const int s = n % kStages;
    if (!mbar_wait_warp(&full[s], (n / kStages) & 1)) {
      ok = false;
      break;
    }
    const TileInfo ti = infos[s];
    const int ncols = ti.n * p.group, groups = (ncols + 7) / 8;
    if (ti.first && groups == 1) load_columns(ti.t0, ncols, ti.hk, 0);
    const int base = ti.base + 16 * warp;
    const bool live = ((ti.have >> warp) & 1u) && base <= ti.last;
    __half2 a[2][kFr][4];
    if (live) {
      const uint8_t *k = smem + s * L::kStage + 16 * warp * (kDim / 2);
      KeyRows<kDim> rows;
      rows.load(k, smem + s * L::kStage + L::kCodes + 16 * warp * (kDim / 16), g, tq);
#pragma unroll
      for (int i = 0; i < kFr; ++i) {
        rows.values(0, i, a[0][i]);
        rows.values(1, i, a[1][i]);
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[s]);
    if (!live) continue;
    float sum[2] = {};
    for (int c = 0; c < groups; ++c) {
      if (groups > 1) load_columns(ti.t0, ncols, ti.hk, c);
      float acc[2][4] = {};
#pragma unroll
      for (int i = 0; i < kFr; ++i) {
        mma_16816(acc[0], as_u32(a[0][i][0]), as_u32(a[1][i][0]), as_u32(a[0][i][1]), as_u32(a[1][i][1]), qr[i].x, qr[i].y);
        mma_16816(acc[1], as_u32(a[0][i][2]), as_u32(a[1][i][2]), as_u32(a[0][i][3]), as_u32(a[1][i][3]), qr[i].z, qr[i].w);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float w = exp2_fast(fmaf(acc[0][e] + acc[1][e], cs[e & 1], -ls[e & 1]));
        if (base + g + 4 * (e & 2) <= lim[e & 1]) sum[e >> 1] += w;
      }
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], 1);
      sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], 2);
    }
    // one addition a slot and run (a sequence in several runs adds in any order)
    if (tq < 2) {
      const int slot = base + g + 8 * tq;
      if (slot <= ti.last)
        atomicAdd(p.weight + (static_cast<int64_t>(ti.b) * pv.H_kv + ti.hk) * p.ld + slot, tq ? sum[1] : sum[0]);
    }
  }
  if (!ok && lane == 0) {
    raise_flag(p.status, kFlagTimeout);
    flags[0] = 1;
  }
}

size_t round_up(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

template <int kDim>
cudaError_t launch(const WeightsParams &p, cudaStream_t stream) {
  auto kern = weights4_kernel<kDim>;
  static bool done[64] = {};
  const cudaError_t e = set_smem_once(reinterpret_cast<const void *>(kern), WeightsSmem<kDim>::total, done);
  if (e != cudaSuccess) return e;
  return launch_ex(false, kern, dim3(2 * sm_count()), dim3(kThreads), WeightsSmem<kDim>::total, stream, 1, p);
}

}  // namespace

size_t weights4_scratch(const sa_paged4_args &pa) {
  return round_up((static_cast<size_t>(pa.p.T) + 2) * 8) + 2 * round_up((static_cast<size_t>(pa.p.T) + 2) * 4) + 256;
}

cudaError_t launch_weights4(const sa_paged4_args &pa, const void *q, const float *lse, float *weight, int64_t ld,
                            void *scratch, uint32_t *status, cudaStream_t stream) {
  if (pa.p.T == 0) return cudaSuccess;
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
