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
// A warp takes every 8th (or 6th) group of 32 keys, with a ring of copies, sums and O
// of its own, so that nothing is exchanged until the CTA's part of a unit ends.  (The
// 5th-generation tensor cores would need the fp16 operands in shared memory, four
// times the codes' bytes there and back, for products that fill an eighth of their
// rows; the warp-level product's rate, measured 1018 multiply-adds a clock and SM,
// serves 8 columns at three times HBM's pace and 16 at one and a half.  More columns:
// paged4_umma.cu.)
//
// What bounds it is issue: about 310 instructions for 16 keys and 8 columns (counters:
// the ALU pipe, which the conversion shares with the masks and selects, is the fullest).
// 64 sequences of 8 .. 16 K slots, 64 heads over 8 of 128: 163 us, 5.4 TB/s; 32 sequences
// of 4 tokens at 2 .. 8 K (16 columns, O of 64 registers, three warps a scheduler): 72 us;
// one token of 16 over 2 heads at 40 K slots: 16 us, a chain of loads, joins and merges.
// Measured against: a copy warp with barriers for all (219 us: a wait that is already
// over still costs a warp 150 to 200 clocks), 7 or 5 warps for 16 columns (79, 84 us).
//
// A column's logits are taken relative to a reference that is raised (and O
// rescaled) only when one passes it by 2^14; weights are then at most 2^14 and
// enter the product as fp16, normal down to 2^-28 of the largest.
//
// Work: paged4_units.cuh.  A warp's copies are 16 bytes a lane, three groups in flight;
// a page's rows of one KV head are contiguous, and a page that is not there reads as
// zeros.  A unit that is cut leaves parts in scratch; the CTA that adds the last of
// them (a counter) merges them in order, in two steps where they are many.
#include <cfloat>
#include <climits>

#include <algorithm>
#include <type_traits>

#include "internal.h"
#include "paged4_mma.cuh"
#include "paged4_units.cuh"
#include "paged_umma.cuh"

namespace sa {
namespace {

using namespace umma;

constexpr int kTile = 128;               // slots per tile: the grain of the work's division
// Warps of a CTA: with two CTAs per SM, 128 registers each for 8 of them and 168 for 6
// (O of 16 columns of 128 alone is 64)
template <int kDim, int NT>
constexpr int warps_of() {
  return kDim == 128 && NT == 2 ? 6 : 8;
}
constexpr int kCtasPerSm = 2;
constexpr int kGroup = 32;               // slots of a warp's step
constexpr int kStages = 3;               // groups that a warp has in its ring
constexpr int kLeast = 2;                // tiles of a CTA, at least
constexpr int kFan = 16;                 // parts that a CTA merges; a unit of more is merged in two steps
constexpr int kMostCtas = 400;           // counters: one a CTA, then one per kFan CTAs
static_assert(kMostCtas + kMostCtas / kFan <= kAttn4Counters, "counters");

template <int kDim, int NT>
struct AttnSmem {
  static constexpr int kWarps = warps_of<kDim, NT>();
  static constexpr uint32_t kCodes = kGroup * kDim / 2, kScales = kGroup * kDim / 16;  // of a group
  static constexpr uint32_t kStage = 2 * (kCodes + kScales);
  static constexpr uint32_t kRing = kStages * kStage;  // of a warp; at a part's end it holds its O, [D / 4][32] fp32
  static constexpr size_t qf = static_cast<size_t>(kWarps) * kRing;               // [NT][D / 32][32] 16 B: fragments
  static constexpr size_t cols = qf + 8 * NT * kDim * 2;                         // factor, limit of a column
  static constexpr size_t poison = cols + 16 * 8;                                // [8] lowest slot with a NaN block
  static constexpr uint32_t stat = kDim / 4 * 32 * 4;  // within a warp's ring at a part's end: [16] reference, sum
  static constexpr size_t scan = poison + 32;
  static constexpr size_t start = scan + 32 * 8;
  static constexpr size_t flag = start + sizeof(UnitStart);
  static constexpr size_t total = flag + 16;
  static_assert(sizeof(UnitStart) % 8 == 0 && kRing >= stat + 16 * 8, "layout");
  static_assert((total + 1024) * kCtasPerSm <= 228 * 1024, "shared memory of an SM");
};

struct Attn4Params {
  Paged4View c;
  const uint16_t *q;
  __nv_bfloat16 *out;
  float *lse;
  float *part;         // [2 grid][NT][D / 4][32]
  float2 *ml;          // [2 grid][16]: reference (log2 units), sum
  uint32_t *counters;  // [kAttn4Counters], 0 between calls
  int group, nt;       // query heads of a KV head, tokens of a block (group * nt <= 16)
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

template <int kDim, int NT, bool kSmall>
__global__ void __launch_bounds__(32 * warps_of<kDim, NT>(), kCtasPerSm)
attn4_kernel(const Attn4Params p) {
  using L = AttnSmem<kDim, NT>;
  constexpr int kWarps = L::kWarps;
  extern __shared__ __align__(128) uint8_t smem[];
  UnitStart *start = reinterpret_cast<UnitStart *>(smem + L::start);
  volatile int *last_s = reinterpret_cast<volatile int *>(smem + L::flag);  // whether this CTA merges a unit's parts
  const PagedView &pv = p.c.v;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  long long x0, x1;
  int ctas;
  find_units<true>(pv, p.nt, pv.H_kv, kTile, kLeast, reinterpret_cast<long long *>(smem + L::scan), start, p.status, x0, x1, ctas,
                   reinterpret_cast<int *>(smem));
  __syncthreads();
  if (x0 >= x1) return;
  const long long total = start->total;
  const int round = start->round;

  const int g = lane >> 2, tq = lane & 3;
  uint4 *qf = reinterpret_cast<uint4 *>(smem + L::qf);
  float2 *cols = reinterpret_cast<float2 *>(smem + L::cols);  // factor of the logits, limit (as an int)
  int *poison = reinterpret_cast<int *>(smem + L::poison);
  uint8_t *ring = smem + warp * L::kRing;
  const uint32_t ring_s = smem_u32(ring);
  constexpr int kCols = (8 * NT + kWarps - 1) / kWarps;                   // columns that a warp stages
  constexpr int kMt = kDim / 16, kEach = (kMt + kWarps - 1) / kWarps;  // pairs of O's rows, of a warp
  Columns<kDim, NT> a;

  // Every warp walks the CTA's units by itself: lane l holds token l of a block.
  int block = start->block, hk = start->head, kt0 = start->tile;
  const int skip_to = start->t0;  // units of the first block before this token are not of this CTA
  long long x = x0;
  int t_seq = -1, t_pos = -1, n_seq = -1, n_pos = -1;
  auto load_block = [&](int i, int &seq, int &pos) {
    const int64_t t = static_cast<int64_t>(i) * p.nt + lane;
    const bool in = lane < p.nt && t < pv.T;
    seq = in ? pv.q_seq[t] : -1;
    pos = in ? pv.q_pos[t] : -1;
  };
  load_block(block, n_seq, n_pos);
  for (; x < x1 && static_cast<int64_t>(block) * p.nt < pv.T; ++block) {
    t_seq = n_seq;
    t_pos = n_pos;
    load_block(block + 1, n_seq, n_pos);
    const int count = static_cast<int>(min(static_cast<int64_t>(p.nt), pv.T - static_cast<int64_t>(block) * p.nt));
    const bool in = lane < count;
    const bool valid = in && t_seq >= 0 && t_seq < pv.B && t_pos >= 0 && (t_pos >> pv.logP) < pv.max_pages;
    const int prev = __shfl_up_sync(0xffffffffu, t_seq, 1);
    uint32_t starts = __ballot_sync(0xffffffffu, in && (lane == 0 || t_seq != prev));
    while (starts && x < x1) {
      const int l0 = __ffs(starts) - 1;
      starts &= starts - 1;
      const int l1 = starts ? __ffs(starts) - 1 : count;
      const int t0 = block * p.nt + l0;
      if (t0 < skip_to) continue;
      const bool member = lane >= l0 && lane < l1 && valid;
      const int last = __reduce_max_sync(0xffffffffu, member ? t_pos : -1);
      const int low = __reduce_min_sync(0xffffffffu, member ? t_pos : INT_MAX);
      const int cost = (last + kTile) / kTile;
      if (cost == 0) continue;
      const int counted = (cost + round - 1) / round * round;
      const int seq = __shfl_sync(0xffffffffu, t_seq, l0);
      for (; hk < pv.H_kv && x < x1; ++hk, kt0 = 0) {
        const int ng = p.group, h0 = hk * ng;
        const int ncols = (l1 - l0) * ng;
        const long long u0 = x - kt0, u1 = u0 + counted;
        const int c0 = u0 < x0 ? cta_of_tile(u0, total, ctas) : blockIdx.x;
        const int c1 = u1 > x1 ? cta_of_tile(u1 - 1, total, ctas) : blockIdx.x;
        const int end = static_cast<int>(min(static_cast<long long>(counted), kt0 + (x1 - x))), kt1 = min(cost, end);
        x += end - kt0;
        // ------------------------------- this CTA's part of a unit: tiles kt0 .. kt1 - 1
        // groups of 32 slots: warp w takes first + w, + 8, ..; lane l holds the page of
        // the l-th of each 32 (pages of 16: of the halves of each 16 groups)
        constexpr int kPer = kTile / kGroup;       // groups of a tile
        constexpr int kIds = kSmall ? 16 : 32;     // groups whose pages the lanes hold
        const int n_groups = min(kt1 * kPer, last / kGroup + 1) - kt0 * kPer - warp;
        const int mine = n_groups > 0 ? (n_groups + kWarps - 1) / kWarps : 0;
        const int first = kt0 * kPer + warp;
        uint32_t qw[kCols][kDim / 64];
#pragma unroll
        for (int j = 0; j < kCols; ++j) {
          const int col = warp + j * kWarps, i = min(col, ncols - 1) / ng;
          load_column<kDim>(p.q + (static_cast<int64_t>(t0 + i) * pv.H + h0 + col - i * ng) * kDim, col < ncols, lane, qw[j]);
        }
        auto load_ids = [&](int i) {
          const int j = i + (kSmall ? lane >> 1 : lane);
          const int slot = kGroup * (first + kWarps * j) + (kSmall ? 16 * (lane & 1) : 0);
          if (j >= mine || slot > last) return -1;
          return load_page(pv, seq, slot >> pv.logP, p.status, true);
        };
        int ids = load_ids(0), ids_next = -1;
        uint32_t held = __ballot_sync(0xffffffffu, ids >= 0), held_now = held;  // which of them are pages
        auto copy = [&](int i) {
          if (i < mine) {
            const uint32_t st = ring_s + (i % kStages) * L::kStage;
            const int slot = kGroup * (first + kWarps * i);
            constexpr int kS = kDim / 16;     // 16-byte chunks of the scales of 16 rows
            // rows of a page from `in` on, into the ring from row `at` on; where there is
            // no page nothing is read
            auto rows = [&](int id, int in, uint32_t at, auto n_tag) {
              constexpr int n = decltype(n_tag)::value;
              const uint32_t bytes = id >= 0 ? 16u : 0u;
              const int64_t row = (static_cast<int64_t>(max(id, 0) * pv.H_kv + hk) << pv.logP) + in;
              const uint8_t *k = p.c.K + row * (kDim / 2) + 16 * lane, *v = p.c.V + row * (kDim / 2) + 16 * lane;
#pragma unroll
              for (int e = 0; e < n * kDim / 2; e += 512) {
                cp_async16_or_zero(st + at * (kDim / 2) + e + 16 * lane, k + e, bytes);
                cp_async16_or_zero(st + L::kCodes + at * (kDim / 2) + e + 16 * lane, v + e, bytes);
              }
              constexpr int kC = n / 16 * kS;  // chunks of scales, of K and of V
              const int c = lane % kC;
              if (2 * kC == 32 || lane < 2 * kC)
                cp_async16_or_zero(st + 2 * L::kCodes + (lane < kC ? 0 : L::kScales) + at * (kDim / 16) + 16 * c,
                                   (lane < kC ? p.c.Ks : p.c.Vs) + row * (kDim / 16) + 16 * c, bytes);
            };
            if constexpr (kSmall) {
#pragma unroll
              for (int h = 0; h < 2; ++h)
                rows(__shfl_sync(0xffffffffu, ids, (2 * i + h) & 31), 0, 16 * h, std::integral_constant<int, 16>());
            } else {
              rows(__shfl_sync(0xffffffffu, ids, i & 31), slot & (pv.P - 1), 0, std::integral_constant<int, 32>());
            }
          }
          cp_async_commit();
        };
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i) copy(i);
        if (tid < 8) poison[tid] = INT_MAX;
        // queries as fp16 fragments, a column per warp
#pragma unroll
        for (int j = 0; j < kCols; ++j) {
          const int col = warp + j * kWarps, i = min(col / ng, l1 - l0 - 1);
          const int pos = __shfl_sync(0xffffffffu, valid ? t_pos : -1, l0 + i);
          if (col >= 8 * NT) continue;
          const float inv = stage_column<kDim>(qw[j], col, lane, qf);
          if (lane == 0) cols[col] = make_float2(p.qk_scale * inv, __int_as_float(col < ncols ? pos : -1));
        }
        __syncthreads();
        a.begin(cols, lane);
#pragma unroll 1
        for (int i = 0; i < mine; ++i) {
          const int ahead = i + kStages - 1;
          if (ahead % kIds == 0) {
            ids = ids_next;
            held = __ballot_sync(0xffffffffu, ids >= 0);
          }
          if (i % kIds == 0) held_now = held;  // (ahead is among the same)
          cp_async_wait<kStages - 2>();
          __syncwarp();
          copy(ahead);
          if (ahead % kIds == 4) ids_next = load_ids(ahead - 4 + kIds);
          const int base = kGroup * (first + kWarps * i);
          const uint32_t halves = kSmall ? (held_now >> (2 * (i % kIds))) & 3u : ((held_now >> (i % kIds)) & 1u) * 3u;
          if (halves) {
            const uint8_t *st = ring + (i % kStages) * L::kStage;
            a.step(st, st + 2 * L::kCodes, st + L::kCodes, st + 2 * L::kCodes + L::kScales, base,
                   base + kGroup - 1 > low || halves != 3u, halves, low, last, qf, poison, lane);
          }
        }
        cp_async_wait<0>();
        a.sum_up();
        const bool cut = c0 != c1;
        int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (c0 == static_cast<int>(blockIdx.x) ? 1 : 0);
        // The warps' sums and O joined: into scratch (to_part) or the output.
        auto join = [&](bool to_part) {
          if (g == 0) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 2; ++e) reinterpret_cast<float2 *>(ring + L::stat)[8 * nt + 2 * tq + e] = make_float2(a.ref[nt][e], a.l[nt][e]);
          }
          __syncthreads();
          int bad[kEach];
#pragma unroll
          for (int i = 0; i < kEach; ++i) bad[i] = poison[(kDim / 8 * g + 2 * ((warp + i * kWarps) % kMt)) >> 4];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            // the columns' references over the warps, their sums, this warp's factors
            float m[2] = {-FLT_MAX, -FLT_MAX}, sum[2] = {}, fac[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              auto stat = [&](int w) {
                return reinterpret_cast<const float2 *>(smem + w * L::kRing + L::stat)[8 * nt + 2 * tq + e];
              };
              for (int w = 0; w < kWarps; ++w) m[e] = fmaxf(m[e], stat(w).x);
              for (int w = 0; w < kWarps; ++w) sum[e] += stat(w).y * exp2_fast(stat(w).x - m[e]);
              fac[e] = exp2_fast(a.ref[nt][e] - m[e]);
            }
            float *mine_s = reinterpret_cast<float *>(ring) + lane;
#pragma unroll
            for (int mt = 0; mt < kMt; ++mt)
#pragma unroll
              for (int e = 0; e < 4; ++e) mine_s[(4 * mt + e) * 32] = a.o[nt][mt][e] * fac[e & 1];
            __syncthreads();
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
              const int mt = warp + i * kWarps, d = kDim / 8 * g + 2 * mt;
              if (mt >= kMt) break;
              float o[4] = {};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
#pragma unroll
                for (int w = 0; w < kWarps; ++w) o[e] += reinterpret_cast<const float *>(smem + w * L::kRing)[(4 * mt + e) * 32 + lane];
                // a NaN block of V that the column's token attends
                if (a.lim[nt][e & 1] >= bad[i]) o[e] = NAN;
              }
              if (to_part) {
#pragma unroll
                for (int e = 0; e < 4; ++e) __stcg(p.part + ((slot * NT + nt) * (kDim / 4) + 4 * mt + e) * 32 + lane, o[e]);
                if (mt == 0 && g == 0)
                  __stcg(reinterpret_cast<float4 *>(p.ml + slot * 16 + 8 * nt + 2 * tq), make_float4(m[0], sum[0], m[1], sum[1]));
              } else {
                store_columns<kDim>(o, m, sum, 8 * nt + 2 * tq, ncols, a.lim[nt], p, t0, h0, ng, d, mt == 0 && g == 0);
              }
            }
            if (NT > 1) __syncthreads();
          }
        };
        join(cut);
        if (cut) {
          // The last CTA to add a part merges them.  Of more than kFan, it merges its group's
          // into the first one's place, and the last group to be done merges the groups' (a
          // CTA reads 4 KB of 8 columns a part at 30 bytes a clock: one token over 304 CTAs
          // 19.1 us by one CTA a unit).
          const int me = static_cast<int>(blockIdx.x);
          bool groups = c1 - c0 >= kFan;
          int lo = groups ? c0 + (me - c0) / kFan * kFan : c0, hi = groups ? min(lo + kFan - 1, c1) : c1;
          int span = 1, counter = lo;
          for (;;) {
            if (groups && lo == hi) {
              // (a group of one has its part in place; its counter is the next unit's)
            } else {
              __syncthreads();
              if (tid == 0) {
                const bool last_one = count_part(p.counters + counter) == static_cast<uint32_t>((hi - lo) / span);
                if (last_one) p.counters[counter] = 0;  // for the next call
                *last_s = last_one;
              }
              __syncthreads();
              if (!*last_s) break;
              // every warp takes a part in turn
              a.begin(cols, lane);
              for (int k = lo + warp * span; k <= hi; k += kWarps * span) {
                const int64_t from = 2 * static_cast<int64_t>(k) + (k == c0);
  #pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                  float x[kMt][4];
                  const float4 s = __ldcg(reinterpret_cast<const float4 *>(p.ml + from * 16 + 8 * nt + 2 * tq));
  #pragma unroll
                  for (int mt = 0; mt < kMt; ++mt)
  #pragma unroll
                    for (int e = 0; e < 4; ++e) x[mt][e] = __ldcg(p.part + ((from * NT + nt) * (kDim / 4) + 4 * mt + e) * 32 + lane);
  #pragma unroll
                  for (int e = 0; e < 2; ++e) {
                    const float r = e ? s.z : s.x, m = fmaxf(a.ref[nt][e], r);
                    const float f0 = exp2_fast(a.ref[nt][e] - m), f1 = exp2_fast(r - m);
                    a.ref[nt][e] = m;
                    a.l[nt][e] = a.l[nt][e] * f0 + (e ? s.w : s.y) * f1;
  #pragma unroll
                    for (int mt = 0; mt < kMt; ++mt) {
                      a.o[nt][mt][e] = a.o[nt][mt][e] * f0 + x[mt][e] * f1;
                      a.o[nt][mt][e + 2] = a.o[nt][mt][e + 2] * f0 + x[mt][e + 2] * f1;
                    }
                  }
                }
              }
              slot = 2 * static_cast<int64_t>(lo) + (lo == c0);
              join(groups);
              if (!groups) break;
            }
            groups = false;
            lo = c0;
            hi = c0 + (c1 - c0) / kFan * kFan;
            span = kFan;
            counter = kMostCtas + c0 / kFan;
          }
        }
        __syncthreads();  // (the next part's copies land where O was)
      }
      if (hk == pv.H_kv) hk = 0;
    }
  }
}

int grid_of() { return std::min(kCtasPerSm * sm_count(), kMostCtas); }

template <int kDim, int NT, bool kSmall>
cudaError_t launch(const Attn4Params &p, cudaStream_t stream) {
  auto kern = attn4_kernel<kDim, NT, kSmall>;
  static bool done[64] = {};
  const cudaError_t e = set_smem_once(reinterpret_cast<const void *>(kern), AttnSmem<kDim, NT>::total, done);
  if (e != cudaSuccess) return e;
  return launch_ex(false, kern, dim3(grid_of()), dim3(32 * warps_of<kDim, NT>()), AttnSmem<kDim, NT>::total, stream, 1, p);
}

size_t most_parts() { return 2 * static_cast<size_t>(grid_of()); }
size_t round_up(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

}  // namespace

int columns_of(const sa_paged4_args &pa) {
  const int64_t each = (pa.p.T + static_cast<int64_t>(pa.p.B) - 1) / pa.p.B;
  return static_cast<int>(std::min<int64_t>(std::max<int64_t>(each, 1) * (pa.p.H / pa.p.H_kv), 1 << 20));
}

size_t attn4_scratch(const sa_paged4_args &pa) {
  if (columns_of(pa) > 16) return attn4_umma_scratch(pa);
  return round_up(sizeof(float) * most_parts() * 16 * pa.p.D) + round_up(sizeof(float2) * most_parts() * 16);
}

cudaError_t launch_attn4(const sa_paged4_args &pa, const void *q, void *out, float *lse, void *scratch,
                         uint32_t *counters, uint32_t *status, cudaStream_t stream) {
  if (pa.p.T == 0) return cudaSuccess;
  // Up to 16 columns here (O of more is more than a warp's registers hold), where 16 of them take
  // half of the time that they take on the 5th-generation tensor cores (every call with a cold
  // L2: 64 sequences of 128 over 8 heads at 8 .. 16 K slots 238 us here and 449 there, 32
  // sequences of 4 drafted tokens of 32 over 8 heads 74 and 141, one token of 100 slots 14 and
  // 33).  More columns there: up to 128 with one row tile (64 sequences of 64 heads over one
  // KV head 223 us, with two 345; 4 tokens of 32 heads over one 72 and 90), above with two
  // (1270 prompt tokens of 32 over 4 heads without their join 201 us, with one 263).
  const int columns = columns_of(pa);
  if (columns > 16)
    return launch_attn4_umma(pa, q, out, lse, columns > 128 ? 256 : 128, scratch, status, stream);
  Attn4Params p;
  p.c = paged4_view(pa);
  p.q = static_cast<const uint16_t *>(q);
  p.out = static_cast<__nv_bfloat16 *>(out);
  p.lse = lse;
  p.part = static_cast<float *>(scratch);
  p.ml = reinterpret_cast<float2 *>(static_cast<char *>(scratch) + round_up(sizeof(float) * most_parts() * 16 * pa.p.D));
  p.counters = counters;
  p.group = pa.p.H / pa.p.H_kv;
  p.qk_scale = pa.p.scale * pa.k_gain * kLog2e;
  p.v_gain = pa.v_gain;
  p.status = status;
  // tokens of a block: one as long as the call can be a token per sequence
  p.nt = pa.p.T <= pa.p.B ? 1 : 16 / p.group;
  auto of_pages = [&](auto dim, auto nt) {
    constexpr int kDim = decltype(dim)::value, NT = decltype(nt)::value;
    return pa.p.P == 16 ? launch<kDim, NT, true>(p, stream) : launch<kDim, NT, false>(p, stream);
  };
  auto of_columns = [&](auto dim) {
    return p.nt * p.group <= 8 ? of_pages(dim, std::integral_constant<int, 1>())
                               : of_pages(dim, std::integral_constant<int, 2>());
  };
  return pa.p.D == 128 ? of_columns(std::integral_constant<int, 128>()) : of_columns(std::integral_constant<int, 64>());
}

}  // namespace sa
