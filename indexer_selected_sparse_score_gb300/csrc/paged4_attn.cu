// Attention of a few query columns (tokens x heads of a KV head, up to 16) over a
// cache held in 4 bits: one pass over the codes.
//
// For D = 128 a row of keys and of values is 144 bytes, so the cache streams at
// 2.3 x the rows of a 16-bit one, and what bounds the kernel next to HBM is the
// conversion: 256 values a row, at a rate of 64 pairs a clock and SM for the
// conversion instruction alone against the 20 pairs a clock that 6.7 TB/s brings.
// So codes are turned into fp16 operands in registers, where the warp-level
// product wants them, and touch shared memory only as codes:
//   S^T = K Q^T   M = 16 keys, N = 8 columns, K = D.  The contraction may take D in
//                 any order: lane (g, t) takes values D/4 t .. of keys g and g + 8,
//                 one 16-byte load of each
//   O^T += V^T P^T  M = 16 of D, N = 8 columns, K = 16 keys.  Lane (g, t) takes block
//                 g's values of keys 2t, 2t + 1, 2t + 8, 2t + 9; code pairs of two keys
//                 are joined before the conversion (four operations for eight pairs)
//   P^T           two 8 x 8 transposes in registers (movmatrix)
// A warp owns 16 of a tile's 128 keys with sums and O of its own, so nothing is
// exchanged until the CTA's part of a unit ends.  (The 5th-generation tensor cores
// would need the fp16 operands in shared memory, four times the codes' bytes there
// and back, for products that fill an eighth of their rows; the warp-level
// product's rate, measured 1018 multiply-adds a clock and SM, serves 8 columns at
// three times HBM's pace and 16 at one and a half.  More columns: paged4_umma.cu.)
//
// A column's logits are taken relative to a reference that is raised (and O
// rescaled) only when one passes it by 2^14; weights are then at most 2^14 and
// enter the product as fp16, normal down to 2^-28 of the largest.
//
// Work: paged4_units.cuh.  A copy warp keeps a ring of tiles in flight (bulk
// copies; a page's rows of one KV head are contiguous).  A unit that is cut leaves
// parts in scratch; the CTA that adds the last of them (a counter) merges them in
// order.
#include <algorithm>

#include "internal.h"
#include "paged4_mma.cuh"
#include "paged4_units.cuh"
#include "umma.cuh"

namespace sa {
namespace {

using namespace umma;

constexpr int kTile = 128;               // slots per tile, 16 per warp
constexpr int kWarps = 8;                // and a copy warp
constexpr int kThreads = 32 * kWarps + 32;
constexpr int kCtasPerSm = 2;
constexpr int kLeast = 2;                // tiles of a CTA, at least

// What the copy warp tells of a tile.
struct TileInfo {
  int t0, n, h0, g;      // unit: first token, tokens, first query head, heads of a token
  int base;              // first slot
  int low, last;         // lowest and highest slot of the unit's valid tokens
  uint32_t have;         // bit w: slots 16 w .. of the tile are in a page
  int first, end;        // first, last tile of this CTA's part of the unit
  int c0, c1;            // CTAs that share the unit
  int pos[16];           // slots of the tokens, -1 for one to be skipped
};

template <int kDim, int NT>
struct AttnSmem {
  static constexpr int kStages = kDim == 128 ? 3 : 6;
  static constexpr uint32_t kCodes = kTile * kDim / 2, kScales = kTile * kDim / 16;
  static constexpr uint32_t kQ = 8 * NT * kDim * 2;  // queries as they come
  static constexpr uint32_t kStage = 2 * (kCodes + kScales) + kQ;
  static constexpr size_t red = static_cast<size_t>(kStages) * kStage;      // [warp][D / 4][32] fp32
  static constexpr size_t qf = red + kWarps * (kDim / 4) * 32 * 4;  // [NT][D / 32][32] 16 B: fragments
  static constexpr size_t info = qf + kQ;
  static constexpr size_t cols = info + kStages * sizeof(TileInfo);         // factor, limit of a column
  static constexpr size_t stat = cols + 16 * 8;                             // [warp][16] reference, sum
  static constexpr size_t poison = stat + kWarps * 16 * 8;                  // [8] lowest slot with a NaN block
  static constexpr size_t bars = poison + 32;
  static constexpr size_t scan = bars + (2 * kStages + 1) * 8;
  static constexpr size_t start = scan + 32 * 8;
  static constexpr size_t flag = start + sizeof(UnitStart);
  static constexpr size_t total = flag + 16;
  static_assert(sizeof(TileInfo) % 8 == 0 && sizeof(UnitStart) % 8 == 0 && kQ % 16 == 0, "alignment");
  static_assert(total <= 113 * 1024, "two CTAs per SM");
};

struct Attn4Params {
  Paged4View c;
  const uint16_t *q;
  __nv_bfloat16 *out;
  float *lse;
  float *part;         // [2 grid][NT][D / 4][32]
  float2 *ml;          // [2 grid][16]: reference (log2 units), sum
  uint32_t *counters;  // [grid], 0 between calls
  int group, gb, nt;   // query heads of a KV head, their parts, tokens of a block
  float qk_scale, v_gain;
  uint32_t *status;
};

// Columns col0 and col0 + 1 of a unit: values d and d + 1 of the output rows (o: [d
// + 0, 1][column]) and, with write_lse, the rows' logarithms.
template <int kDim>
__device__ __forceinline__ void store_columns(const float (&o)[4], const float (&m)[2], const float (&sum)[2], int col0,
                                              int ncols, const int (&lim)[2], const Attn4Params &p, int t0, int h0, int ng,
                                              int d, bool write_lse) {
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int col = col0 + e;
    if (col >= ncols || lim[e] < 0) continue;
    const int i = col / ng;
    const int64_t row = static_cast<int64_t>(t0 + i) * p.c.v.H + h0 + col - i * ng;
    const float inv = sum[e] != 0.f ? p.v_gain / sum[e] : 0.f;
    *reinterpret_cast<__nv_bfloat162 *>(p.out + row * kDim + d) = __floats2bfloat162_rn(o[e] * inv, o[2 + e] * inv);
    if (write_lse && p.lse) p.lse[row] = sum[e] == 0.f ? -INFINITY : (m[e] + log2f(sum[e])) * 0.69314718055994531f;
  }
}

// Joins the parts of a unit shared by CTAs c0 .. c1, in their order.
template <int kDim, int NT>
__device__ __forceinline__ void merge_parts(const float *part, const float2 *ml, int c0, int c1, int nt, int mt, int lane,
                                            float (&o)[4], float (&m)[2], float (&sum)[2]) {
  constexpr int kBatch = 8;  // parts whose loads go out together
  for (int k0 = c0; k0 <= c1; k0 += kBatch) {
    float x[kBatch][4];
    float4 s[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int k = min(k0 + i, c1);
      const int64_t slot = 2 * static_cast<int64_t>(k) + (k == c0);
      s[i] = __ldcg(reinterpret_cast<const float4 *>(ml + slot * 16 + 8 * nt + 2 * (lane & 3)));
#pragma unroll
      for (int e = 0; e < 4; ++e) x[i][e] = __ldcg(part + ((slot * NT + nt) * (kDim / 4) + 4 * mt + e) * 32 + lane);
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float top = m[e];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) top = fmaxf(top, e ? s[i].z : s[i].x);
      if (top == -INFINITY) continue;
      const float f = m[e] == top ? 1.f : exp2f(m[e] - top);
      m[e] = top;
      sum[e] *= f;
      o[e] *= f;
      o[2 + e] *= f;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        if (k0 + i > c1) continue;
        const float r = e ? s[i].z : s[i].x;
        const float w = r == top ? 1.f : exp2f(r - top);
        sum[e] = fmaf(w, e ? s[i].w : s[i].y, sum[e]);
        o[e] = fmaf(w, x[i][e], o[e]);
        o[2 + e] = fmaf(w, x[i][2 + e], o[2 + e]);
      }
    }
  }
}

template <int kDim, int NT>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
attn4_kernel(const Attn4Params p) {
  using L = AttnSmem<kDim, NT>;
  constexpr int kStages = L::kStages;
  extern __shared__ __align__(128) uint8_t smem[];
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + L::bars), *empty = full + kStages, *meet = empty + kStages;
  TileInfo *infos = reinterpret_cast<TileInfo *>(smem + L::info);
  UnitStart *start = reinterpret_cast<UnitStart *>(smem + L::start);
  volatile int *flags = reinterpret_cast<volatile int *>(smem + L::flag);  // [0] abort, [1] last of a unit's parts
  const PagedView &pv = p.c.v;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], kWarps);
    }
    mbar_init(meet, kWarps);
    flags[0] = 0;
    fence_barrier_init();
  }
  long long x0, x1;
  int ctas;
  const int heads = pv.H_kv * p.gb;
  find_units(pv, p.nt, heads, kTile, kLeast, reinterpret_cast<long long *>(smem + L::scan), start, p.status, x0, x1, ctas);
  __syncthreads();

  if (warp == kWarps) {
    // ------------------------------------------------------------ copy warp
    int issued = 0;
    bool ok = true;
    if (x0 < x1) {
      const long long total = start->total;
      int block = start->block, hv = start->head, kt = start->tile;
      int skip_to = start->t0;  // units of the block before this token are not of this CTA
      long long x = x0;
      while (x < x1 && ok && static_cast<int64_t>(block) * p.nt < pv.T) {
        // the units of one block: lane l holds token block * nt + l
        const int t = block * p.nt + lane;
        const bool in = lane < p.nt && t < pv.T;
        const int b = in ? pv.q_seq[t] : -1, pos = in ? pv.q_pos[t] : -1;
        const bool valid = in && b >= 0 && b < pv.B && pos >= 0 && (pos >> pv.logP) < pv.max_pages;
        const int b_prev = __shfl_up_sync(0xffffffffu, b, 1);
        uint32_t starts = __ballot_sync(0xffffffffu, in && (lane == 0 || b != b_prev));
        const int count = __popc(__ballot_sync(0xffffffffu, in));
        while (starts && x < x1 && ok) {
          const int l0 = __ffs(starts) - 1;
          starts &= starts - 1;
          const int l1 = starts ? __ffs(starts) - 1 : count;
          const int t0 = block * p.nt + l0;
          if (t0 < skip_to) continue;
          const bool member = lane >= l0 && lane < l1 && valid;
          const int last = static_cast<int>(__reduce_max_sync(0xffffffffu, member ? pos : -1));
          const int low = static_cast<int>(__reduce_min_sync(0xffffffffu, member ? pos : 0x7FFFFFFF));
          const int cost = (last + kTile) / kTile;
          if (cost == 0) continue;
          const int seq = __shfl_sync(0xffffffffu, b, l0);
          const int mypos = __shfl_sync(0xffffffffu, valid ? pos : -1, min(l0 + lane, 31));
          for (; hv < heads && x < x1 && ok; ++hv) {
            const int hk = hv / p.gb, g0 = 16 * (hv - hk * p.gb), ng = min(16, p.group - g0), h0 = hk * p.group + g0;
            const long long u0 = x - kt, u1 = u0 + cost;
            const int c0 = u0 < x0 ? cta_of_tile(u0, total, ctas) : blockIdx.x;
            const int c1 = u1 > x1 ? cta_of_tile(u1 - 1, total, ctas) : blockIdx.x;
            bool fresh = true;
            for (; kt < cost && x < x1; ++kt, ++x) {
              const int s = issued % kStages;
              // lane 4 q + kind copies page q's part: codes and scales of K and V
              const int base = kt * kTile, q = lane >> 2, kind = lane & 3;
              const int from = base + (q << pv.logP);
              const int rows = min(pv.P, ((min(last - from, kTile) + 16) & ~15));  // this page's, by sixteens
              int page = -1;
              if (q < (kTile >> pv.logP) && from <= last)
                page = load_page(pv, seq, from >> pv.logP, p.status, kind == 0);
              uint32_t have = 0;
              const uint32_t pages = __ballot_sync(0xffffffffu, page >= 0 && kind == 0);
#pragma unroll
              for (int w = 0; w < kWarps; ++w) have |= ((pages >> (4 * ((16 * w) >> pv.logP))) & 1u) << w;
              const uint32_t row_bytes = kind < 2 ? kDim / 2 : kDim / 16;
              const uint32_t bytes = page >= 0 ? rows * row_bytes : 0u;
              const uint32_t sum = __reduce_add_sync(0xffffffffu, bytes);
              if (!mbar_wait_warp(&empty[s], ((issued / kStages) & 1) ^ 1) || flags[0]) {
                ok = false;
                break;
              }
              uint8_t *stage = smem + s * L::kStage;
              TileInfo *in_s = &infos[s];
              const uint32_t q_bytes = fresh ? static_cast<uint32_t>(l1 - l0) * ng * kDim * 2 : 0u;
              if (lane < 16) in_s->pos[lane] = l0 + lane < l1 ? mypos : -1;
              if (lane == 0) {
                in_s->t0 = t0;
                in_s->n = l1 - l0;
                in_s->h0 = h0;
                in_s->g = ng;
                in_s->base = base;
                in_s->low = low;
                in_s->last = last;
                in_s->have = have;
                in_s->first = fresh;
                in_s->end = kt + 1 == cost || x + 1 == x1;
                in_s->c0 = c0;
                in_s->c1 = c1;
              }
              __syncwarp();
              if (lane == 0) mbar_expect_tx(&full[s], sum + q_bytes);
              __syncwarp();
              ++issued;
              if (bytes) {
                const int64_t at = (static_cast<int64_t>(page) * pv.H_kv + hk) * pv.P * row_bytes;
                const uint8_t *src = (kind == 0 ? p.c.K : kind == 1 ? p.c.V : kind == 2 ? p.c.Ks : p.c.Vs) + at;
                uint8_t *dst = stage + (kind == 0   ? 0
                                        : kind == 1 ? L::kCodes
                                        : kind == 2 ? 2 * L::kCodes
                                                    : 2 * L::kCodes + L::kScales) + (q << pv.logP) * row_bytes;
                bulk_load(dst, src, bytes, &full[s]);
              }
              if (fresh && lane < l1 - l0)
                bulk_load(stage + 2 * (L::kCodes + L::kScales) + lane * ng * kDim * 2,
                          p.q + (static_cast<int64_t>(t0 + lane) * pv.H + h0) * kDim, ng * kDim * 2,
                          &full[s]);
              fresh = false;
            }
            if (kt < cost) break;  // the range ends inside the unit
            kt = 0;
          }
          if (hv == heads) hv = 0;
        }
        ++block;
      }
    }
    if (lane == 0) {
      if (!ok) {
        raise_flag(p.status, kFlagTimeout);
        flags[0] = 1;
      }
      // every copy lands before the CTA exits
      for (int m = max(0, issued - kStages); m < issued; ++m) mbar_wait(&full[m % kStages], (m / kStages) & 1);
    }
    __syncwarp();
    return;
  }

  // --------------------------------------------------------- product warps
  const int g = lane >> 2, tq = lane & 3;
  uint4 *qf = reinterpret_cast<uint4 *>(smem + L::qf);
  float2 *cols = reinterpret_cast<float2 *>(smem + L::cols);  // factor of the logits, limit (as an int)
  float2 *stat = reinterpret_cast<float2 *>(smem + L::stat);
  int *poison = reinterpret_cast<int *>(smem + L::poison);
  float *red = reinterpret_cast<float *>(smem + L::red);
  int met = 0;
  bool ok = true;
  // the product warps meet (a bounded wait: a warp that gave up must not hold the others)
  auto sync = [&]() {
    __syncwarp();
    if (lane == 0) mbar_arrive(meet);
    ok = mbar_wait_warp(meet, (met++) & 1) && ok;
  };
  Columns<kDim, NT> a;
  long long left = x1 - x0;
  for (int n = 0; left > 0; ++n, --left) {
    const int s = n % kStages;
    if (!mbar_wait_warp(&full[s], (n / kStages) & 1)) {
      ok = false;
      break;
    }
    const uint8_t *stage = smem + s * L::kStage;
    const TileInfo &ti = infos[s];
    if (ti.first) {
      // queries as fp16 fragments, a column per warp
      if (tid < 8) poison[tid] = 0x7FFFFFFF;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        stage_column<kDim>(reinterpret_cast<const uint16_t *>(stage + 2 * (L::kCodes + L::kScales)), 8 * nt + warp,
                           ti.n * ti.g, lane, qf, [&](int col, float inv) {
                             cols[col] = make_float2(p.qk_scale * inv,
                                                     __int_as_float(col < ti.n * ti.g ? ti.pos[col / ti.g] : -1));
                           });
      sync();
      if (!ok) break;
      a.begin(qf, cols, lane);
    }
    const int base = ti.base + 16 * warp;
    if (((ti.have >> warp) & 1u) && base <= ti.last) {
      const uint8_t *k = stage + 16 * warp * (kDim / 2), *v = k + L::kCodes;
      const uint8_t *ks = stage + 2 * L::kCodes + 16 * warp * (kDim / 16), *vs = ks + L::kScales;
      const bool edge = base + 15 > ti.low;
      a.step(k, ks, v, vs, base, edge, ti.low, ti.last, qf, poison, lane);
    }
    if (!ti.end) {
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[s]);
      continue;
    }
    // ------------------------------------------ the part of a unit is done
    const int t0 = ti.t0, ng = ti.g, ncols = ti.n * ng, h0 = ti.h0, c0 = ti.c0, c1 = ti.c1;
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[s]);
    a.sum_up();
    if (g == 0) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) stat[warp * 16 + 8 * nt + 2 * tq + e] = make_float2(a.ref[nt][e], a.l[nt][e]);
    }
    sync();
    if (!ok) break;
    const int d = kDim / 8 * g + 2 * warp;  // of the O values that this thread finishes: d, d + 1 of two columns
    const int bad = warp < kDim / 16 ? poison[d >> 4] : 0;
    const bool cut = c0 != c1;
    const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (c0 == static_cast<int>(blockIdx.x) ? 1 : 0);
    constexpr int kMt = kDim / 16;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      // the column's reference over the warps, its sum, and this warp's factor
      float m[2], sum[2], fac[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int col = 8 * nt + 2 * tq + e;
        m[e] = -INFINITY;
        for (int w = 0; w < kWarps; ++w) m[e] = fmaxf(m[e], stat[w * 16 + col].x);
        sum[e] = 0.f;
        const float mm = m[e] == -INFINITY ? 0.f : m[e];
        for (int w = 0; w < kWarps; ++w) {
          const float2 x = stat[w * 16 + col];
          sum[e] += x.y * (x.x == -INFINITY ? 0.f : exp2f(x.x - mm));
        }
        fac[e] = a.ref[nt][e] == -INFINITY ? 0.f : exp2f(a.ref[nt][e] - mm);
      }
      float *mine = red + warp * (kDim / 4) * 32 + lane;
#pragma unroll
      for (int mt = 0; mt < kMt; ++mt)
#pragma unroll
        for (int e = 0; e < 4; ++e) mine[(4 * mt + e) * 32] = a.o[nt][mt][e] * fac[e & 1];
      sync();
      if (!ok) break;
      if (warp < kMt) {
        float o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          o[e] = 0.f;
          for (int w = 0; w < kWarps; ++w) o[e] += red[(w * (kDim / 4) + 4 * warp + e) * 32 + lane];
        }
        // a NaN block of V that the column's token attends
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (a.lim[nt][e & 1] >= bad) o[e] = NAN;
        if (cut) {
#pragma unroll
          for (int e = 0; e < 4; ++e) p.part[((slot * NT + nt) * (kDim / 4) + 4 * warp + e) * 32 + lane] = o[e];
          if (warp == 0 && g == 0)
#pragma unroll
            for (int e = 0; e < 2; ++e) p.ml[slot * 16 + 8 * nt + 2 * tq + e] = make_float2(m[e], sum[e]);
        } else {
          store_columns<kDim>(o, m, sum, 8 * nt + 2 * tq, ncols, a.lim[nt], p, t0, h0, ng, d, warp == 0 && g == 0);
        }
      }
      if (NT > 1) sync();
      if (!ok) break;
    }
    if (!ok) break;
    if (cut) {
      __threadfence();
      sync();
      if (!ok) break;
      if (tid == 0) {
        const uint32_t before = atomicAdd(&p.counters[c0], 1u);
        flags[1] = before == static_cast<uint32_t>(c1 - c0);
        if (flags[1]) p.counters[c0] = 0;  // for the next call
        __threadfence();
      }
      sync();
      if (!ok) break;
      if (flags[1] && warp < kMt) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float o[4] = {}, m[2] = {-INFINITY, -INFINITY}, sum[2] = {};
          merge_parts<kDim, NT>(p.part, p.ml, c0, c1, nt, warp, lane, o, m, sum);
          store_columns<kDim>(o, m, sum, 8 * nt + 2 * tq, ncols, a.lim[nt], p, t0, h0, ng, d, warp == 0 && g == 0);
        }
      }
    }
    // (the next part's first write to what is read here comes after its first meeting)
  }
  if (!ok && lane == 0) {
    raise_flag(p.status, kFlagTimeout);
    flags[0] = 1;
  }
}

int grid_of() { return std::min(kCtasPerSm * sm_count(), kAttn4Counters); }

template <int kDim, int NT>
cudaError_t launch(const Attn4Params &p, cudaStream_t stream) {
  auto kern = attn4_kernel<kDim, NT>;
  static bool done[64] = {};
  const cudaError_t e = set_smem_once(reinterpret_cast<const void *>(kern), AttnSmem<kDim, NT>::total, done);
  if (e != cudaSuccess) return e;
  return launch_ex(false, kern, dim3(grid_of()), dim3(kThreads), AttnSmem<kDim, NT>::total, stream, 1, p);
}

size_t round_up(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

}  // namespace

size_t attn4_scratch(const sa_paged4_args &pa) {
  return round_up(2 * sizeof(float) * grid_of() * 16 * pa.p.D) + round_up(2 * sizeof(float2) * grid_of() * 16);
}

cudaError_t launch_attn4(const sa_paged4_args &pa, const void *q, void *out, float *lse, void *scratch,
                         uint32_t *counters, uint32_t *status, cudaStream_t stream) {
  if (pa.p.T == 0) return cudaSuccess;
  Attn4Params p;
  p.c = paged4_view(pa);
  p.q = static_cast<const uint16_t *>(q);
  p.out = static_cast<__nv_bfloat16 *>(out);
  p.lse = lse;
  p.part = static_cast<float *>(scratch);
  p.ml = reinterpret_cast<float2 *>(static_cast<char *>(scratch) + round_up(2 * sizeof(float) * grid_of() * 16 * pa.p.D));
  p.counters = counters;
  p.group = pa.p.H / pa.p.H_kv;
  p.qk_scale = pa.p.scale * pa.k_gain * kLog2e;
  p.v_gain = pa.v_gain;
  p.status = status;
  // tokens of a block: one as long as the call can be a token per sequence
  p.gb = (p.group + 15) / 16;
  p.nt = pa.p.T <= pa.p.B ? 1 : std::max(1, 16 / p.group);
  if (p.nt * p.group <= 8) return pa.p.D == 128 ? launch<128, 1>(p, stream) : launch<64, 1>(p, stream);
  return pa.p.D == 128 ? launch<128, 2>(p, stream) : launch<64, 2>(p, stream);
}

}  // namespace sa
