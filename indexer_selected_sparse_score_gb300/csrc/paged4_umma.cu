// Attention of many query columns (tokens x heads of a KV head, up to 256) over a
// cache held in 4 bits, on the 5th-generation tensor cores.
//
//   S = Q K^T   M = 128 rows, N = 128 keys, K = D; a softmax thread owns a row
//   P           fp16, written over S in tensor memory (the A operand of P V)
//   O += P V    M = 128 rows, N = D, K = 128 keys, V read MN-major
// Eight warps turn codes into fp16 tiles in the 128-byte swizzle: they copy the codes
// of the next tiles asynchronously (a warp the rows that it converts, so copies need
// no barrier), multiply by the blocks' scales and store.  The products take 512
// clocks each for 128 rows; the conversion hides behind those of 256 rows (with four
// converting warps it did not: 300 us against 250 for 64 tokens of 64 heads over one
// KV head).
//
// Two streams of products take turns on the tensor cores, each with a softmax
// warpgroup and an issuing warp:
//   two row tiles (units of up to 256 rows: chunks of a prompt): both meet every key
//   tile, so a tile is converted once for 256 rows;
//   one row tile (up to 128: a few tokens or one, of many heads): both hold the same
//   rows, and key tiles go to them in turn; their sums and O are joined at the end.
//   Up to 64 rows lie in the tile twice, each copy with half of a tile's keys, so that
//   every softmax thread has keys to take.
// A row's logits are taken relative to a reference, 2^6 below its first ones' largest.
// Where the weights of 64 keys add up to more than 2^15, it is raised by a power of two
// that brings the largest back to 2^6, and O is rescaled; so weights stay below fp16's
// largest and are normal down to 2^-19 of the row's largest, or more.
//
// Bound by a stream's chain: a tile's logits, softmax (2900 clocks for 128 keys beside
// the other stream's products: loads from tensor memory wait behind them), weights,
// product: about 5000 clocks, in which the tensor cores work 1024 for each of the streams.  1270 prompt tokens of
// 32 over 4 heads at 6 .. 12 K slots: 238 us, 0.84 PFLOP/s; 64 tokens of 64 heads over one
// KV head at 32 .. 65 K: 225 us; a call of one short unit: 24 us, of which a part's queries,
// chain and stores are 15.
//
// Work: paged4_units.cuh, units cut evenly over one CTA per SM, or few of them into pieces
// of one length; what has to be joined goes to scratch, and a second kernel joins the
// units that were cut, in order.
#include <cfloat>
#include <climits>

#include <algorithm>

#include "internal.h"
#include "paged4_mma.cuh"
#include "paged4_units.cuh"
#include "paged_list.h"
#include "paged_umma.cuh"

namespace sa {
namespace {

using namespace umma;

constexpr int kTile = 128;
constexpr int kThreads = 640;
constexpr int kWarpConv = 8;   // .. 11 convert keys, 12 .. 15 values (rows 32 i .. 32 i + 31 of a tile each)
constexpr int kWarpMma = 16;   // and 17: the issuers
constexpr int kWarpInfo = 18;  // describes the tiles (19 only joins the block barriers)
constexpr int kLeast = 2;      // tiles of a CTA, at least
constexpr int kInfos = 8, kParts = 4;
// Registers per thread: 640 threads start with 96 each; the softmax warpgroups raise
// their limit, the last one lowers its own: 2 * 120 + 2 * 96 + 48 = 5 * 96.
constexpr int kLaunchRegs = 96, kSoftmaxRegs = 120, kOtherRegs = 48;
static_assert(2 * kSoftmaxRegs + 2 * kLaunchRegs + kOtherRegs <= 5 * kLaunchRegs, "register split exceeds the launch allocation");

struct TileInfo {
  int t0, n, hk;     // unit: first token, tokens, KV head
  int base;          // first slot
  int low, last;     // lowest and highest slot of the unit's valid tokens
  uint32_t have;     // bit j: slots 16 j .. of the tile are in a page
  int first, end;    // first, last tile of this CTA's part of the unit
  int c0, c1;        // CTAs that share the unit
  int tiles;         // of the part
  int part;          // parts of this CTA before
  int pad;
};

template <int kDim, bool kTwo>
struct UmmaSmem {
  static constexpr int kRowTiles = kTwo ? 2 : 1;
  static constexpr int kSlots = kDim == 128 ? 4 : 6;                  // fp16 tiles: K(0), V(0), K(1), ..
  static constexpr int kStages = kDim == 128 ? (kTwo ? 1 : 3) : 4;    // tiles of codes
  static constexpr uint32_t kBlock = kTile * 128;
  static constexpr uint32_t kKv = kBlock * (kDim / 64);
  static constexpr uint32_t kCodes = 32 * kDim / 2, kScales = 32 * kDim / 16;  // of a warp's rows
  static constexpr uint32_t kStage = kCodes + kScales;
  static constexpr size_t q = 0;                                      // [row tile][D / 64][128 rows][128 B]
  static constexpr size_t kv = q + kRowTiles * kKv;
  static constexpr size_t codes = kv + kSlots * kKv;                  // [converting warp][stage]
  static constexpr size_t info = codes + 8 * kStages * kStage;
  static constexpr size_t parts = info + kInfos * sizeof(TileInfo);   // [kParts] tiles, rows of a part
  static constexpr size_t factor = parts + kParts * 8;  // [row tile][128] of the logits
  static constexpr size_t poison = factor + kRowTiles * 512;          // [kInfos][4 warps][8]
  static constexpr size_t bars = poison + kInfos * 4 * 8 * 4;
  static constexpr int kBars = 2 * kSlots + 2 * kInfos + 2 * kParts + 2 + 2 + 4 + 2 + 2 + 2 + 2 + 1;
  static constexpr size_t scan = bars + kBars * 8;
  static constexpr size_t start = scan + 32 * 8;
  static constexpr size_t misc = start + sizeof(UnitStart);
  static constexpr size_t total = misc + 16;
  static_assert(total + 1024 <= 232448, "shared memory budget");
  static_assert(sizeof(TileInfo) % 8 == 0 && bars % 8 == 0 && start % 8 == 0, "alignment");
};

struct UmmaParams {
  Paged4View c;
  const uint16_t *q;
  __nv_bfloat16 *out;
  float *lse;
  float *part;         // [slot][stream][128][D]
  float2 *ml;          // [slot][stream][128]: reference (log2 units, -inf: nothing), sum
  int4 *cuts;          // [grid] unit whose first part is the CTA's: first token, rows, KV head, last CTA; rows 0: none
  int group, nt;
  float qk_scale, v_gain;
  uint32_t *status;
};

__device__ __forceinline__ constexpr uint32_t idesc_f16(int M, int N) {
  return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// mbar_wait_warp with a first look that costs a vote: most phases are complete by
// the time they are asked for.
__device__ __forceinline__ bool wait_warp(uint64_t *bar, uint32_t parity) {
  return __all_sync(0xffffffffu, mbar_test_wait(bar, parity)) || mbar_wait_warp(bar, parity);
}

// One warp: row rr of a unit, its pieces (the parts of CTAs c0 .. c1, of two streams, each
// with two copies of up to 64 rows) joined in order, into the output.
template <int kDim, bool kTwo>
__device__ __forceinline__ void join_row(const UmmaParams &p, int rr, int rows, int t0, int hk, int c0, int c1, int lane) {
  constexpr int V = kDim / 32;
  const PagedView &pv = p.c.v;
  const int i = rr / p.group, pos = pv.q_pos[t0 + i];
  const int log_subs = kTwo ? 0 : rows <= 64 ? 2 : 1, count = (c1 - c0 + 1) << log_subs;
  auto piece = [&](int k) {  // its index among the rows of scratch
    const int c = c0 + (k >> log_subs), sub = k & ((1 << log_subs) - 1);
    return ((3 * c + (c0 == c1 ? 2 : c == c0 ? 1 : 0)) * 2 + (rr >> 7) + (sub & 1)) * 128 + (rr & 127) + 64 * (sub >> 1);
  };
  // loads that go out together: rows of two row tiles are many and have few pieces (8: 5 us
  // more for a chunk; 4 of the others: 8 us more for 64 heads over one)
  constexpr int kBatch = kTwo ? 4 : 8;
  float y[kBatch][V];
  auto load = [&](int k) {
#pragma unroll
    for (int e = 0; e < kBatch; ++e) {
      if (k + e >= count) continue;
      const float *src = p.part + static_cast<int64_t>(piece(k + e)) * kDim + V * lane;
      if constexpr (V == 4)
        *reinterpret_cast<float4 *>(y[e]) = __ldcg(reinterpret_cast<const float4 *>(src));
      else
        *reinterpret_cast<float2 *>(y[e]) = __ldcg(reinterpret_cast<const float2 *>(src));
    }
  };
  load(0);  // (needs nothing of the references)
  float M = -INFINITY;
  for (int k = lane; k < count; k += 32) M = max_nan(M, __ldcg(&p.ml[piece(k)].x));
  if (pos < 0 || (pos >> pv.logP) >= pv.max_pages) return;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = max_nan(M, __shfl_xor_sync(0xffffffffu, M, o));
  float sum = 0.f, acc[V] = {};
  for (int k0 = 0; k0 < count; k0 += 32) {
    // lane l: the factor of piece k0 + l, below 0 where it has nothing (what lies there may be anything)
    float f = -1.f;
    if (k0 + lane < count) {
      const float2 v = __ldcg(p.ml + piece(k0 + lane));
      if (v.x != -INFINITY) {
        f = v.x == M ? 1.f : exp2_hw(v.x - M);
        sum += v.y * f;
      }
    }
    for (int k1 = k0; k1 < min(count, k0 + 32); k1 += kBatch) {
      if (k1 > 0) load(k1);
#pragma unroll
      for (int e = 0; e < kBatch; ++e) {
        const float fk = __shfl_sync(0xffffffffu, f, (k1 + e) & 31);
        if (k1 + e >= count || fk < 0.f) continue;
#pragma unroll
        for (int j = 0; j < V; ++j) acc[j] = fmaf(y[e][j], fk, acc[j]);
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  const int64_t out_row = static_cast<int64_t>(t0 + i) * pv.H + hk * p.group + rr - i * p.group;
  const float inv = sum != 0.f ? p.v_gain / sum : 0.f;
#pragma unroll
  for (int e = 0; e < V; e += 2)
    *reinterpret_cast<__nv_bfloat162 *>(p.out + out_row * kDim + V * lane + e) =
        __floats2bfloat162_rn(acc[e] * inv, acc[e + 1] * inv);
  if (lane == 0 && p.lse) p.lse[out_row] = sum == 0.f ? -INFINITY : (M + log2f(sum)) * 0.69314718055994531f;
}

// Joins the units that were cut: CTA (x: eight rows, y: CTA of the first part), a warp a row.
// (Many SMs at once: by the CTA that added the last part, 11 tokens of 32 over 2 heads at 8 K
// slots took 128 us, in two steps 75.)
template <int kDim, bool kTwo>
__global__ void __launch_bounds__(256, kTwo ? 6 : 4) join4_kernel(const UmmaParams p) {
  pdl_wait();
  const int4 u = p.cuts[blockIdx.y];
  const int rr = 8 * blockIdx.x + (threadIdx.x >> 5);
  if (rr < u.y) join_row<kDim, kTwo>(p, rr, u.y, u.x, u.z, blockIdx.y, u.w, threadIdx.x & 31);
}

template <int kDim, bool kTwo>
__global__ void __launch_bounds__(kThreads, 1)
umma4_kernel(const UmmaParams p) {
  using L = UmmaSmem<kDim, kTwo>;
  constexpr int kSlots = L::kSlots;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t *qs = smem + L::q, *kvs = smem + L::kv;
  TileInfo *infos = reinterpret_cast<TileInfo *>(smem + L::info);
  int2 *parts = reinterpret_cast<int2 *>(smem + L::parts);
  float *factor = reinterpret_cast<float *>(smem + L::factor);
  int *poison = reinterpret_cast<int *>(smem + L::poison);
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::bars);
  uint64_t *full = bars, *empty = full + kSlots;
  uint64_t *ifull = empty + kSlots, *iempty = ifull + kInfos, *gfull = iempty + kInfos, *gempty = gfull + kParts;
  uint64_t *qfull = gempty + kParts, *sfull = qfull + 2;
  uint64_t *pfull = sfull + 2, *opv = pfull + 4, *ofull = opv + 2, *turn = ofull + 2, *done = turn + 2, *meet = done + 2;
  UnitStart *start = reinterpret_cast<UnitStart *>(smem + L::start);
  uint32_t *tmem_base_s = reinterpret_cast<uint32_t *>(smem + L::misc);
  volatile int *abort_s = reinterpret_cast<volatile int *>(smem + L::misc + 4);
  const PagedView &pv = p.c.v;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_trigger();
  if (tid == 0) {
    p.cuts[blockIdx.x] = make_int4(0, 0, 0, 0);
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&full[i], 4);
      mbar_init(&empty[i], kTwo ? 2 : 1);
    }
    for (int i = 0; i < kInfos; ++i) {
      mbar_init(&ifull[i], 1);
      mbar_init(&iempty[i], 8);  // softmax warps
    }
    for (int i = 0; i < kParts; ++i) {
      mbar_init(&gfull[i], 1);
      mbar_init(&gempty[i], 2);  // issuers
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&qfull[i], kTwo ? 4 : 8);  // the warps that stage queries
      mbar_init(&sfull[i], 1);
      mbar_init(&pfull[2 * i], 4);
      mbar_init(&pfull[2 * i + 1], 4);
      mbar_init(&opv[i], 1);
      mbar_init(&ofull[i], 1);
      mbar_init(&turn[i], 1);
      mbar_init(&done[i], 1);
    }
    mbar_init(meet, 8);
    *abort_s = 0;
    fence_barrier_init();
  }
  if (warp == kWarpMma) {
    tmem_alloc(tmem_base_s, 512);
    tmem_relinquish();
  }
  long long x0, x1;
  int ctas;
  find_units<true>(pv, p.nt, pv.H_kv, kTile, kLeast, reinterpret_cast<long long *>(smem + L::scan), start, p.status, x0, x1, ctas,
                   reinterpret_cast<int *>(kvs));
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_base_s;
  const long long total = start->total;
  const int round = start->round;
  const long long tiles = x0 < x1 && round > 1 ? start->tiles : x1 - x0;
  auto fail = [&]() {
    raise_flag(p.status, kFlagTimeout);
    *abort_s = 1;
  };

  // Calls use(seq, t0, len, low, last, hv, kt0, count, c0, c1) for the parts of units
  // that this CTA has, in order; stops when it returns false.  (A whole warp.)
  auto walk = [&](const auto &use) {
    int block = start->block, hv = start->head, kt0 = start->tile;
    long long x = x0;
    // first token of the block that is not yet in a unit (before `start` they are other CTAs')
    int i0 = x0 < x1 ? static_cast<int>(start->t0 - static_cast<int64_t>(block) * p.nt) : 0;
    while (x < x1 && static_cast<int64_t>(block) * p.nt < pv.T) {
      const int in_block = static_cast<int>(min(static_cast<int64_t>(p.nt), pv.T - static_cast<int64_t>(block) * p.nt));
      while (x < x1 && i0 < in_block) {
        // the unit that begins at token i0
        const int t0 = block * p.nt + i0;
        const int seq = pv.q_seq[t0];
        int last = -1, low = INT_MAX, len = 0;
        for (bool more = true; more;) {
          const int l = i0 + len + lane;
          const bool in = l < in_block;
          const int b = in ? pv.q_seq[block * p.nt + l] : 0, pos = in ? pv.q_pos[block * p.nt + l] : -1;
          const uint32_t other = __ballot_sync(0xffffffffu, !in || b != seq);
          const int take = other ? __ffs(other) - 1 : 32;
          const bool valid = lane < take && b >= 0 && b < pv.B && pos >= 0 && (pos >> pv.logP) < pv.max_pages;
          last = max(last, __reduce_max_sync(0xffffffffu, valid ? pos : -1));
          low = min(low, __reduce_min_sync(0xffffffffu, valid ? pos : INT_MAX));
          len += take;
          more = take == 32;
        }
        i0 += len;
        const int cost = (last + kTile) / kTile;
        if (cost == 0) continue;
        for (; hv < pv.H_kv && x < x1; ++hv, kt0 = 0) {
          const int counted = (cost + round - 1) / round * round;
          const long long u0 = x - kt0, u1 = u0 + counted;
          const int c0 = u0 < x0 ? cta_of_tile(u0, total, ctas) : blockIdx.x;
          const int c1 = u1 > x1 ? cta_of_tile(u1 - 1, total, ctas) : blockIdx.x;
          const int taken = static_cast<int>(min(static_cast<long long>(counted - kt0), x1 - x)), count = min(taken, cost - kt0);
          x += taken;
          if (!use(seq, t0, len, low, last, hv, kt0, count, c0, c1)) return;
        }
        if (hv == pv.H_kv) hv = 0;
      }
      ++block;
      i0 = 0;
    }
  };

  if (warp >= kWarpMma) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp < kWarpMma + 2) {
      // ---------------------------------------------- issuer of one stream
      const int w = warp - kWarpMma;
      const bool leader = elect_one();
      constexpr uint32_t idesc_s = idesc_f16(128, kTile);
      constexpr uint32_t idesc_o = idesc_f16(128, kDim) | (1u << 16);  // V is MN-major
      const uint32_t ts = tmem + 128 * w, to = tmem + 256 + 128 * w;
      const uint64_t dq = desc_sw128_kmajor(smem_u32(qs + (kTwo ? w : 0) * L::kKv));
      const uint32_t kv0 = smem_u32(kvs);
      bool ok = true, two = false;
      int qn = 0, ln = 0, turns = 0;
      // Two row tiles: the issuers take turns, O_A(n), S_A(n + 1), then O_B(n), S_B(n + 1),
      // so that the softmax of one runs while the products of the other do.
      auto take_turn = [&]() -> bool {
        if (!two) return true;
        const int k = turns++;
        return w == 0 ? k == 0 || wait_warp(&turn[1], (k - 1) & 1) : wait_warp(&turn[0], k & 1);
      };
      auto wait_full = [&](int m) { return wait_warp(&full[m % kSlots], (m / kSlots) & 1); };
      // (the address once for the warp, so that the descriptors are uniform values)
      auto slot_of = [&](int m) { return __reduce_or_sync(0xffffffffu, kv0 + (m % kSlots) * L::kKv); };
      auto issue_s = [&](int m) {
        const uint32_t at = slot_of(m);
        if (leader) {
          const uint64_t db = desc_sw128_kmajor(at);
#pragma unroll
          for (int kk = 0; kk < kDim / 16; ++kk) {
            const uint64_t o = ((kk >> 2) * L::kBlock + (kk & 3) * 32) >> 4;
            mma_f16(ts, dq + o, db + o, idesc_s, kk > 0);
          }
          mma_commit(&sfull[w]);
          mma_commit(&empty[m % kSlots]);
        }
        __syncwarp();
      };
      auto issue_o = [&](int m, int half, bool fresh, bool end) {
        const uint32_t at = slot_of(m);
        if (leader) {
          const uint64_t dv = desc_mn(at, L::kBlock);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_f16_tmem_a(to, ts + 32 * half + 8 * kk, dv + (((4 * half + kk) * 2048) >> 4), idesc_o, !(fresh && kk == 0));
          if (!half) mma_commit(&opv[w]);
          if (half && end) mma_commit(&ofull[w]);
          if (half) mma_commit(&empty[m % kSlots]);
        }
        __syncwarp();
      };
      int n = 0;
      for (int part = 0; n < tiles && ok; ++part) {
        ok = wait_warp(&gfull[part % kParts], (part / kParts) & 1) && !*abort_s;
        if (!ok) break;
        const int count = parts[part % kParts].x, rows = parts[part % kParts].y;
        __syncwarp();
        if (lane == 0) mbar_arrive(&gempty[part % kParts]);
        if constexpr (kTwo) {
          two = rows > 128;
          if (w == 1 && !two) {  // only frees the ring
            for (int m = 2 * n; m < 2 * (n + count) && ok; ++m) {
              ok = wait_full(m);
              if (ok && leader) mbar_arrive(&empty[m % kSlots]);
              __syncwarp();
            }
            n += count;
            continue;
          }
          ok = wait_full(2 * n) && wait_warp(&qfull[w], (qn++) & 1) && take_turn();
          if (!ok) break;
          tc_fence_after();
          issue_s(2 * n);
          if (leader && two) mbar_arrive(&turn[w]);
        } else {
          if (w < count) ok = wait_warp(&qfull[w], (qn++) & 1);
        }
        // own tiles of the part: every one, or every second
        constexpr int kStep = kTwo ? 1 : 2;
        for (int j = kTwo ? 0 : w; j < count; j += kStep) {
          const int mk = 2 * (n + j), mv = mk + 1;
          const bool end = j + kStep >= count;
          if constexpr (kTwo) {
            ok = wait_full(mv) && (end || wait_full(mk + 2)) && wait_warp(&pfull[2 * w], ln & 1) &&
                 wait_warp(&pfull[2 * w + 1], ln & 1) && take_turn();
            if (!ok) break;
            tc_fence_after();
            issue_o(mv, 0, j == 0, end);
            issue_o(mv, 1, false, end);
            if (!end) issue_s(mk + 2);
            if (leader && two) mbar_arrive(&turn[w]);
          } else {
            ok = ok && wait_full(mk);
            if (!ok) break;
            tc_fence_after();
            issue_s(mk);
            ok = wait_full(mv) && wait_warp(&pfull[2 * w], ln & 1);
            if (!ok) break;
            tc_fence_after();
            issue_o(mv, 0, j == w, end);
            ok = wait_warp(&pfull[2 * w + 1], ln & 1);
            if (!ok) break;
            tc_fence_after();
            issue_o(mv, 1, false, end);
          }
          ++ln;
        }
        n += count;
      }
      if (!ok && lane == 0) fail();
      if (leader && tiles > 0) {
        mma_commit(&done[w]);
        if (!mbar_wait(&done[w], 0)) raise_flag(p.status, kFlagTimeout);
      }
      __syncwarp();
    }
    if (warp == kWarpInfo) {
      // ------------------------------------------------ descriptions of tiles
      int n = 0, part = 0;
      bool ok = true;
      walk([&](int seq, int t0, int len, int low, int last, int hv, int kt0, int count, int c0, int c1) {
        // lane j: the page of 16 slots j of a tile, loaded a tile ahead
        auto entry = [&](int i) {
          const int slot = kTile * (kt0 + i) + 16 * lane;
          return i < count && lane < 8 && slot <= last ? load_page(pv, seq, slot >> pv.logP, p.status, true) : -1;
        };
        ok = wait_warp(&gempty[part % kParts], ((part / kParts) & 1) ^ 1) && !*abort_s;
        if (!ok) return false;
        if (lane == 0) {
          parts[part % kParts] = make_int2(count, len * p.group);
          mbar_arrive(&gfull[part % kParts]);
        }
        int next = entry(0);
        for (int i = 0; i < count; ++i, ++n) {
          const uint32_t have = __ballot_sync(0xffffffffu, next >= 0);
          next = entry(i + 1);
          ok = wait_warp(&iempty[n % kInfos], ((n / kInfos) & 1) ^ 1) && !*abort_s;
          if (!ok) return false;
          if (lane == 0) {
            infos[n % kInfos] =
                TileInfo{t0, len, hv, kTile * (kt0 + i), low, last, have, i == 0, i + 1 == count, c0, c1, count, part, 0};
            mbar_arrive(&ifull[n % kInfos]);
          }
        }
        ++part;
        return true;
      });
      if (!ok && lane == 0) fail();
    }
  } else if (warp >= kWarpConv) {
    // ---------------------------- codes to fp16 tiles: 32 rows of keys or of values
    const int kv = (warp - kWarpConv) >> 2, cw = warp & 3;
    uint8_t *ring = smem + L::codes + (warp - kWarpConv) * L::kStages * L::kStage;
    const uint32_t ring_s = smem_u32(ring);
    const uint8_t *codes = kv ? p.c.V : p.c.K, *scales = kv ? p.c.Vs : p.c.Ks;
    constexpr int kItems = kDim / 32, kRows = 32 / kItems;
    // Copies: chunk ch (16 bytes) of row kRows e + of a warp's 32, the chunks of a row
    // swapped by bits of the row so that the reads below meet no bank twice
    const int ch = lane % (kDim / 32), cr = lane / (kDim / 32);
    // Item e of a lane: the 32 values from 32 seg on of row kRows e + of (eight lanes in
    // a row store two neighbouring 64-byte pieces of four rows)
    const int seg = kDim == 128 ? (lane & 1) + 2 * (lane >> 4) : lane & 1;
    const int of = kDim == 128 ? (lane >> 1) & 7 : lane >> 1;
    auto swapped = [](int row, int c) { return kDim == 128 ? c ^ ((row & 2) ? 2 : 0) : c; };
    bool ok = true;
    int n = 0, part = 0;
    walk([&](int seq, int t0, int len, int low, int last, int hv, int kt0, int count, int c0, int c1) {
      // lane l: the page of the l-th 16 slots of this warp's rows, two of each tile
      auto load_ids = [&](int i) {
        const int slot = kTile * (kt0 + i + (lane >> 1)) + 32 * cw + 16 * (lane & 1);
        if (i + (lane >> 1) >= count || slot > last) return -1;
        return load_page(pv, seq, slot >> pv.logP, nullptr, false);
      };
      int ids = load_ids(0), ids_next = -1;
      auto copy = [&](int i) {
        if (i < count) {
          const int id0 = __shfl_sync(0xffffffffu, ids, (2 * i) & 31), id1 = __shfl_sync(0xffffffffu, ids, (2 * i + 1) & 31);
          const uint32_t st = ring_s + (i % L::kStages) * L::kStage;
          const int slot = kTile * (kt0 + i) + 32 * cw;
          // (where there is no page, zeros)
          const int64_t row0 = (static_cast<int64_t>(max(id0, 0) * pv.H_kv + hv) << pv.logP) + (slot & (pv.P - 1));
          const int64_t row1 = (static_cast<int64_t>(max(id1, 0) * pv.H_kv + hv) << pv.logP) + ((slot + 16) & (pv.P - 1));
          const uint32_t b0 = id0 >= 0 ? 16u : 0u, b1 = id1 >= 0 ? 16u : 0u;
          const uint8_t *s0 = codes + row0 * (kDim / 2) + 16 * lane, *s1 = codes + row1 * (kDim / 2) + 16 * lane;
          const uint32_t to = st + cr * (kDim / 2) + 16 * swapped(cr, ch);
#pragma unroll
          for (int e = 0; e < kItems / 2; ++e) {
            cp_async16_or_zero(to + 512 * e, s0 + 512 * e, b0);
            cp_async16_or_zero(to + 8 * kDim + 512 * e, s1 + 512 * e, b1);
          }
          constexpr int kSc = kDim / 16;  // chunks of the scales of 16 rows
          if (lane < 2 * kSc)
            cp_async16_or_zero(st + L::kCodes + 16 * lane,
                               scales + (lane < kSc ? row0 : row1) * (kDim / 16) + 16 * (lane % kSc), lane < kSc ? b0 : b1);
        }
        cp_async_commit();
      };
#pragma unroll
      for (int i = 0; i < L::kStages; ++i) copy(i);
      int *bad = poison + ((part % kInfos) * 4 + cw) * 8;
      if (kv == 1 && lane < 8) bad[lane] = INT_MAX;
      __syncwarp();
      for (int i = 0; i < count; ++i, ++n) {
        const int ahead = i + L::kStages;
        if ((ahead & 15) == 0) ids = ids_next;
        cp_async_wait<L::kStages - 1>();
        __syncwarp();
        const uint8_t *st = ring + (i % L::kStages) * L::kStage;
        const int base = kTile * (kt0 + i) + 32 * cw;
        uint4 c[kItems];
        uint32_t sc[kItems];
#pragma unroll
        for (int e = 0; e < kItems; ++e) {
          const int row = of + kRows * e;
          c[e] = *reinterpret_cast<const uint4 *>(st + row * (kDim / 2) + 16 * swapped(row, seg));
          sc[e] = reinterpret_cast<const uint16_t *>(st + L::kCodes + row * (kDim / 16))[seg];
        }
        __syncwarp();
        copy(ahead);  // (into the stage just read)
        if ((ahead & 15) == 5) ids_next = load_ids(ahead - 5 + 16);
        if (base + 31 > (kv ? low : last)) {
          // rows past the last slot become zeros; a NaN block of values that not every row
          // of queries attends is left out and noted
#pragma unroll
          for (int e = 0; e < kItems; ++e) {
            const int slot = base + of + kRows * e;
            if (slot > last) {
              sc[e] = 0;
            } else if (kv == 1 && slot > low) {
#pragma unroll
              for (int b = 0; b < 2; ++b)
                if (e4m3_is_nan((sc[e] >> (8 * b)) & 0xFFu)) {
                  sc[e] &= 0xFFu << (8 * (1 - b));
                  atomicMin(&bad[2 * seg + b], slot);
                }
            }
          }
        }
        const int m = 2 * n + kv;
        ok = wait_warp(&empty[m % kSlots], ((m / kSlots) & 1) ^ 1) && !*abort_s;
        if (!ok) return false;
        uint8_t *dst = kvs + (m % kSlots) * L::kKv + (seg >> 1) * L::kBlock;
#pragma unroll
        for (int e = 0; e < kItems; ++e) {
          const int row = 32 * cw + of + kRows * e;
          const __half2 two = e4m3x2_to_half2(sc[e]);
          const uint32_t words[4] = {c[e].x, c[e].y, c[e].z, c[e].w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const __half2 s2 = j < 2 ? __low2half2(two) : __high2half2(two);
            __half2 d[4];
            e2m1x8_to_half2(words[j], d);
            *reinterpret_cast<uint4 *>(dst + sw128_offset(row, 64 * (seg & 1) + 16 * j)) =
                make_uint4(as_u32(__hmul2(d[0], s2)), as_u32(__hmul2(d[1], s2)), as_u32(__hmul2(d[2], s2)),
                           as_u32(__hmul2(d[3], s2)));
          }
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[m % kSlots]);
      }
      ++part;
      cp_async_wait<0>();
      __syncwarp();
      return true;
    });
    cp_async_wait<0>();
    if (!ok && lane == 0) fail();
  } else {
    // ------------------------------------------------- softmax of one stream
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    const int w = warp >> 2, row = tid & 127;
    const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const uint32_t ts = tmem + lanes + 128 * w, to = tmem + lanes + 256 + 128 * w;
    uint8_t *qt = qs + (kTwo ? w : 0) * L::kKv;
    float *fac = factor + (kTwo ? w : 0) * 128;
    float ref = 0.f, l = 0.f, cs = 0.f;
    int ln = 0, pieces = 0, in_part = 0, met = 0, lim = -1, r = 0, reps = 1;
    bool ok = true, live = true, idle = false;
    auto sync = [&]() {  // of the softmax warps
      __syncwarp();
      if (lane == 0) mbar_arrive(meet);
      ok = mbar_wait_warp(meet, (met++) & 1) && ok;
    };
    int qn = 0;
    TileInfo ti;
    for (int n = 0; n < tiles; ++n) {
      ok = wait_warp(&ifull[n % kInfos], (n / kInfos) & 1);
      if (!ok || *abort_s) break;
      const TileInfo &info = infos[n % kInfos];
      const int base = info.base, part_first = info.first, part_end = info.end;
      const uint32_t tile_have = info.have;
      if (part_first) ti = info;  // (what is the same for all tiles of a part)
      __syncwarp();
      if (lane == 0) mbar_arrive(&iempty[n % kInfos]);
      const int rows = ti.n * p.group;
      bool mine = true;  // this stream has the tile
      if (part_first) {
        in_part = 0;
        l = 0.f;
        ref = 0.f;
        live = kTwo ? w == 0 || rows > 128 : w == 0 || ti.tiles > 1;
        // (up to 64 rows lie in the tile twice, each copy with half of the keys)
        reps = !kTwo && rows <= 64 ? 2 : 1;
        r = kTwo ? 128 * w + row : row & (128 / reps - 1);
        if (!kTwo || live) {
          // the row's token and limit
          const int i = r / p.group;
          lim = -1;
          if (r < rows) {
            const int pos = pv.q_pos[ti.t0 + i];
            if (pos >= 0 && (pos >> pv.logP) < pv.max_pages) lim = pos;
          }
          {
            // the warp's 32 query rows (of one row tile: 16) as fp16, each scaled by a power of
            // two, into the K-major swizzled layout; a load covers whole rows
            constexpr int kLanes = kDim / 8, kPer = 32 / kLanes;
            const int ch = lane % kLanes;
            uint8_t *dst = qt + (ch >> 3) * L::kBlock;
            constexpr int kRows = kTwo ? 32 : 16;
            constexpr int kBatch = kRows / kPer < 8 ? kRows / kPer : 8;  // loads that go out together
            const int first_row = 32 * (warp & 3) + (kTwo ? 0 : 16 * w);
#pragma unroll 1
            for (int e0 = 0; e0 < kRows; e0 += kBatch * kPer) {
              uint4 v[kBatch];
#pragma unroll
              for (int e = 0; e < kBatch; ++e) {
                const int to_row = first_row + e0 + e * kPer + lane / kLanes;
                const int rr = kTwo ? 128 * w + to_row : to_row & (128 / reps - 1), tt = rr / p.group;
                v[e] = make_uint4(0, 0, 0, 0);
                if (rr < rows)
                  v[e] = reinterpret_cast<const uint4 *>(
                      p.q + (static_cast<int64_t>(ti.t0 + tt) * pv.H + ti.hk * p.group + rr - tt * p.group) * kDim)[ch];
              }
#pragma unroll
              for (int e = 0; e < kBatch; ++e) {
                const int to_row = first_row + e0 + e * kPer + lane / kLanes;
                uint32_t u[4] = {v[e].x, v[e].y, v[e].z, v[e].w};
                float top = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                  top = fmaxf(top, fmaxf(fabsf(__uint_as_float(u[j] << 16)), fabsf(__uint_as_float(u[j] & 0xFFFF0000u))));
#pragma unroll
                for (int o = 1; o < kLanes; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                const float f = to_half_factor(top);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                  u[j] = as_u32(__floats2half2_rn(__uint_as_float(u[j] << 16) * f, __uint_as_float(u[j] & 0xFFFF0000u) * f));
                *reinterpret_cast<uint4 *>(dst + sw128_offset(to_row, 16u * (ch & 7))) = make_uint4(u[0], u[1], u[2], u[3]);
                if (ch == 0) fac[to_row] = p.qk_scale / f;
              }
            }
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(&qfull[kTwo ? w : 0]);
              if (!kTwo && ti.tiles > 1) mbar_arrive(&qfull[1]);
            }
          }
          if (!kTwo && live) {
            // (the other stream's warps stage half of the rows that both hold)
            ok = mbar_wait_warp(&qfull[w], (qn++) & 1);
            if (!ok) break;
          }
          cs = fac[row];
          idle = !__any_sync(0xffffffffu, lim >= 0);
        }
      }
      if constexpr (!kTwo) mine = (in_part & 1) == w;
      ++in_part;
      if (live && mine) {
        const bool first = kTwo ? part_first : in_part <= 2;
        const bool mine_end = kTwo ? part_end : in_part + 2 > ti.tiles;
        const bool masked = tile_have != 0xFFu || base + kTile - 1 > ti.low;
        for (int half = 0; half < 2; ++half) {
          if (half == 0) {
            ok = wait_warp(&sfull[w], ln & 1);
            if (!ok || *abort_s) break;
            tc_fence_after();
          }
          const uint32_t th = ts + 64 * half, tp = ts + 32 * half;  // logits, weights
          if (idle) {  // (its rows' weights and O may be anything)
          } else if (reps == 2 && half != (warp >> 1 & 1)) {
            // the other copy of the rows has these keys
            const uint32_t zero[16] = {};
            tmem_store(tp, zero);
            tmem_store(tp + 16, zero);
            if (half) {
              tmem_wait_st();
              tc_fence_before();
            }
          } else {
            // the half's logits relative to the reference, in v
            float v[64];
            float2 *v2 = reinterpret_cast<float2 *>(v);
            auto logits = [&]() {
              tmem_load(th, reinterpret_cast<uint32_t(&)[32]>(v[0]));
              tmem_load(th + 32, reinterpret_cast<uint32_t(&)[32]>(v[32]));
              tmem_ld_wait();
              const float2 cs2 = make_float2(cs, cs), nref2 = make_float2(-ref, -ref);
#pragma unroll
              for (int e = 0; e < 32; ++e) v2[e] = fma2(v2[e], cs2, nref2);
              if (masked) {
                const int d = lim - base - 64 * half;  // the row's last slot in the half
                const uint32_t have = tile_have >> (4 * half);
#pragma unroll
                for (int e = 0; e < 64; ++e)
                  if (e > d || !((have >> (e >> 4)) & 1u)) v[e] = -INFINITY;
              }
            };
            uint32_t pk[32];
            float sum;
            auto weights = [&]() {
              float2 t[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                const float2 w2 = make_float2(exp2_hw(v2[e].x), exp2_hw(v2[e].y));
                t[e & 1] = add2(t[e & 1], w2);
                pk[e] = as_u32(__floats2half2_rn(w2.x, w2.y));
              }
              t[0] = add2(t[0], t[1]);
              sum = t[0].x + t[0].y;
            };
            logits();
            const bool fresh = l == 0.f && lim >= 0;
            // The weights are taken as they come; only where their sum tells that one may
            // be past 2^9 (all are below 2^15 otherwise), or the row has met no key yet, the
            // reference is looked at.
            bool again = __any_sync(0xffffffffu, fresh);
            if (!again) {
              weights();
              again = __any_sync(0xffffffffu, sum > 32768.f);
              if (again) logits();
            }
            if (again) {
              float top;
              {
                float t4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int e = 0; e < 32; ++e) t4[e & 3] = max3(t4[e & 3], v2[e].x, v2[e].y);
                top = fmaxf(max3(t4[0], t4[1], t4[2]), t4[3]);
              }
              // the row's first keys, or a logit 2^8 above its reference: set or raise it;
              // the sum and O shrink in step, and the first half's weights, or O once their
              // product has been added.  By a power of two, which rounds nothing.
              const float up = top == -INFINITY ? 0.f : fresh || top > 8.f ? rintf(top - kRefHead) : 0.f;
              const float2 nup2 = make_float2(-up, -up);
              ref += up;
#pragma unroll
              for (int e = 0; e < 32; ++e) v2[e] = add2(v2[e], nup2);
              if (!(first && half == 0)) {
                if (!kTwo && half && reps == 1) {
                  ok = wait_warp(&opv[w], ln & 1);
                  if (!ok) break;
                  tc_fence_after();
                }
                const float f = exp2f(fminf(-up, 0.f));
                l *= f;
                if (kTwo && half) {
                  const __half2 f2 = __float2half2_rn(f);
#pragma unroll
                  for (int i = 0; i < 2; ++i) {
                    uint32_t o[16];
                    tmem_load(ts + 16 * i, o);
                    tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 16; ++e) o[e] = as_u32(__hmul2(*reinterpret_cast<__half2 *>(&o[e]), f2));
                    tmem_store(ts + 16 * i, o);
                  }
                }
#pragma unroll 1
                for (int i = 0; i < kDim / 16; ++i) {
                  uint32_t o[16];
                  tmem_load(to + 16 * i, o);
                  tmem_ld_wait();
#pragma unroll
                  for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                  tmem_store(to + 16 * i, o);
                }
                tmem_wait_st();
              }
              weights();
            }
            tmem_store(tp, pk);
            tmem_store(tp + 16, pk + 16);
            tmem_wait_st();
            tc_fence_before();
            l += sum;
          }
          __syncwarp();
          // (copies of rows hand over both halves together)
          if (lane == 0 && (reps == 1 || half)) mbar_arrive(&pfull[2 * w + half]);
          if (lane == 0 && reps == 2 && half) mbar_arrive(&pfull[2 * w]);
        }
        if (!ok || *abort_s) break;
        ++ln;
        if (mine_end) {
          ok = mbar_wait_warp(&ofull[w], pieces & 1);
          if (!ok) break;
          ++pieces;
          tc_fence_after();
        }
      }
      if (!part_end) continue;
      // ------------------------------------------------- the part is done
      const bool cut = ti.c0 != ti.c1, joined = cut || !kTwo;
      const int64_t slot = 3 * static_cast<int64_t>(blockIdx.x) +
                           (!cut ? 2 : ti.c0 == static_cast<int>(blockIdx.x) ? 1 : 0);
      const int64_t at = (slot * 2 + w) * 128 + row;
      const int *bad = poison + (ti.part % kInfos) * 32;
      auto poisoned = [&](int blk) {
        return lim >= min(min(bad[blk], bad[8 + blk]), min(bad[16 + blk], bad[24 + blk]));
      };
      const bool stored = live && r < rows && lim >= 0;
      if (joined) __stcg(p.ml + at, live ? make_float2(l == 0.f ? -INFINITY : ref, l) : make_float2(-INFINITY, 0.f));
      if (live) {
        const float inv = l != 0.f ? p.v_gain / l : 0.f;
        const int i = r / p.group;
        const int64_t out_row = static_cast<int64_t>(ti.t0 + i) * pv.H + ti.hk * p.group + r - i * p.group;
#pragma unroll 1
        for (int blk = 0; blk < kDim / 16; ++blk) {
          uint32_t o[16];
          tmem_load(to + 16 * blk, o);
          tmem_ld_wait();
          if (stored) {
            if (poisoned(blk)) {
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = 0x7FFFFFFFu;
            }
            if (joined) {
#pragma unroll
              for (int e = 0; e < 16; e += 4)
                __stcg(reinterpret_cast<float4 *>(p.part + at * kDim + 16 * blk + e),
                       make_float4(__uint_as_float(o[e]), __uint_as_float(o[e + 1]), __uint_as_float(o[e + 2]),
                                   __uint_as_float(o[e + 3])));
            } else {
              uint32_t b[8];
#pragma unroll
              for (int e = 0; e < 8; ++e)
                b[e] = pack_bf16x2(__uint_as_float(o[2 * e]) * inv, __uint_as_float(o[2 * e + 1]) * inv);
              uint4 *dst = reinterpret_cast<uint4 *>(p.out + out_row * kDim + 16 * blk);
              dst[0] = make_uint4(b[0], b[1], b[2], b[3]);
              dst[1] = make_uint4(b[4], b[5], b[6], b[7]);
            }
          }
        }
        if (!joined && stored && p.lse)
          p.lse[out_row] = l == 0.f ? -INFINITY : (ref + log2f(l)) * 0.69314718055994531f;
        tc_fence_before();
      }
      if (!joined) continue;
      if (cut) {  // (joined by the next kernel)
        if (!kTwo) sync();  // (the streams share the queries)
        if (!ok) break;
        if (ti.c0 == static_cast<int>(blockIdx.x) && tid == 0)
          p.cuts[blockIdx.x] = make_int4(ti.t0, rows, ti.hk, ti.c1);
        continue;
      }
      sync();
      if (!ok) break;
      for (int rr = warp; rr < rows; rr += 8) join_row<kDim, kTwo>(p, rr, rows, ti.t0, ti.hk, blockIdx.x, blockIdx.x, lane);
      sync();  // (the next part writes its own rows where these are read)
      if (!ok) break;
    }
    if (!ok && lane == 0) fail();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

size_t round_up(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }
int grid_of() { return sm_count(); }

template <int kDim, bool kTwo>
cudaError_t launch(const UmmaParams &p, cudaStream_t stream) {
  auto kern = umma4_kernel<kDim, kTwo>;
  // the register split assumes kLaunchRegs registers per thread at launch; anything
  // else could leave a raise waiting forever
  static int regs = -1;
  if (regs < 0) {
    cudaFuncAttributes fa;
    const cudaError_t e = cudaFuncGetAttributes(&fa, reinterpret_cast<const void *>(kern));
    if (e != cudaSuccess) return e;
    regs = fa.numRegs;
  }
  if (regs != kLaunchRegs) return cudaErrorInvalidConfiguration;
  const size_t smem = UmmaSmem<kDim, kTwo>::total + 1024;
  static bool done[64] = {};
  const cudaError_t e = set_smem_once(reinterpret_cast<const void *>(kern), smem, done);
  if (e != cudaSuccess) return e;
  const cudaError_t l = launch_ex(false, kern, dim3(grid_of()), dim3(kThreads), smem, stream, 1, p);
  if (l != cudaSuccess) return l;
  return launch_ex(true, join4_kernel<kDim, kTwo>, dim3(kTwo ? 32 : 16, grid_of()), dim3(256), 0, stream, 1, p);
}

}  // namespace

size_t attn4_umma_scratch(const sa_paged4_args &pa) {
  const size_t rows = static_cast<size_t>(grid_of()) * 3 * 2 * 128;
  return round_up(rows * pa.p.D * sizeof(float)) + round_up(rows * sizeof(float2)) + grid_of() * sizeof(int4);
}

cudaError_t launch_attn4_umma(const sa_paged4_args &pa, const void *q, void *out, float *lse, int rows, void *scratch,
                              uint32_t *status, cudaStream_t stream) {
  const size_t scratch_rows = static_cast<size_t>(grid_of()) * 3 * 2 * 128;
  UmmaParams p;
  p.c = paged4_view(pa);
  p.q = static_cast<const uint16_t *>(q);
  p.out = static_cast<__nv_bfloat16 *>(out);
  p.lse = lse;
  char *w = static_cast<char *>(scratch);
  p.part = reinterpret_cast<float *>(w);
  w += round_up(scratch_rows * pa.p.D * sizeof(float));
  p.ml = reinterpret_cast<float2 *>(w);
  p.cuts = reinterpret_cast<int4 *>(w + round_up(scratch_rows * sizeof(float2)));
  p.group = pa.p.H / pa.p.H_kv;
  p.nt = std::max(1, rows / p.group);
  p.qk_scale = pa.p.scale * pa.k_gain * kLog2e;
  p.v_gain = pa.v_gain;
  p.status = status;
  if (rows > 128) return pa.p.D == 128 ? launch<128, true>(p, stream) : launch<64, true>(p, stream);
  return pa.p.D == 128 ? launch<128, false>(p, stream) : launch<64, false>(p, stream);
}

}  // namespace sa
