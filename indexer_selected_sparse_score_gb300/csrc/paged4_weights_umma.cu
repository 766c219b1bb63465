// Slot weights of many query columns, on the 5th-generation tensor cores.
//
//   S^T = K Q^T   M = 128 keys, N = 128 columns (token, head), K = D
//   sum_c 2^(S^T cs_c - lse_c log2 e): a thread owns a key, so the sum over the columns
//                 needs no exchange; the columns' factors come from shared memory
// A first kernel turns the queries into fp16 (each column scaled by a power of two)
// in the swizzled layout of the product's operand, 128 columns of a KV head to a
// tile that the second one copies whole, with the columns' factors, logarithms and
// limits; a last CTA of it finds the call's runs of tokens.
//
// An item is (run, KV head, 128 slots): its keys are converted once, and the tiles of
// the run's tokens pass them; an item is one CTA's, so a slot's sum has one owner and
// one order.  Tiles' logits go to four buffers of tensor memory that four warpgroups
// empty in turn.  The exponentials (32 a clock and SM) and the products take 512 clocks a
// tile each; measured 1130, which are the issuing warp's (waits 300, issue 640) and, with
// a second one, the query tiles' on their way from L2: 1024 prompt tokens of 32 over 4
// heads at 8 K slots 99 us, 10 of them the first kernel's.
#include <climits>

#include <algorithm>

#include "internal.h"
#include "paged4_mma.cuh"
#include "paged4_units.cuh"
#include "paged_umma.cuh"

namespace sa {
namespace {

using namespace umma;

constexpr int kTile = 128;
constexpr int kGroups = 4;         // warpgroups that sum (with two 139 us for a chunk that takes 99, three 101)
constexpr int kWarpConv = 4 * kGroups;    // and the next three
constexpr int kWarpMma = kWarpConv + 4;
constexpr int kWarpCopy = kWarpMma + 1;
constexpr int kWarpInfo = kWarpMma + 2;   // (the last one only joins the block barriers)
constexpr int kThreads = 32 * (kWarpMma + 4);
constexpr int kInfos = 4, kBufs = 4;
constexpr int kConsts = 8;      // tiles whose factors and limits are held (longer than their queries)

// A tile of columns as the first kernel leaves it.
template <int kDim>
struct ColumnTile {
  static constexpr uint32_t kBlock = kTile * 128;
  static constexpr uint32_t q = 0;                           // [D / 64][128 columns][128 B], swizzled
  static constexpr uint32_t factor = kBlock * (kDim / 64);   // [64]: factors of two columns, their -lse log2 e
  static constexpr uint32_t limit = factor + 64 * 16;        // [128]: the column's last slot, -1: it adds nothing
  static constexpr uint32_t low = limit + 128 * 4;           // lowest limit of the tile's columns; highest
  static constexpr uint32_t total = low + 64;
  static constexpr uint32_t consts = total - factor;
};

struct ItemInfo {
  int t0, t1, seq, hk;   // run: tokens t0 .. t1 - 1
  int base, last;        // first slot, last slot of the run
  uint32_t have;         // bit j: slots 16 j .. are in a page
  int b0, b1;            // tiles of columns: token blocks b0 .. b1 (none: b0 > b1)
  int pad[3];
};

template <int kDim>
struct WSmem {
  using Q = ColumnTile<kDim>;
  static constexpr int kSlots = 3;                          // tiles of columns
  static constexpr uint32_t kKeys = Q::kBlock * (kDim / 64);
  static constexpr uint32_t kQ = Q::factor;
  static constexpr size_t keys = 0;                         // [2]
  static constexpr size_t q = keys + 2 * kKeys;
  static constexpr size_t consts = q + kSlots * kQ;         // [kConsts]
  static constexpr size_t info = consts + kConsts * Q::consts;
  static constexpr size_t sums = info + kInfos * sizeof(ItemInfo);  // [128] of each further warpgroup
  static constexpr size_t bars = sums + (kGroups - 1) * 512;
  static constexpr int kBars = 2 * 2 + 2 * kSlots + 2 * kConsts + 2 * kBufs + 2 * kInfos + 2 + 1;
  static constexpr size_t misc = bars + kBars * 8;
  static constexpr size_t total = misc + 16;
  static_assert(total + 1024 <= 232448 && sizeof(ItemInfo) % 16 == 0, "shared memory budget");
};

struct WParams {
  Paged4View c;
  const uint16_t *q;
  const float *lse;
  float *weight;
  int64_t ld;
  Runs runs;
  int *n_runs;
  uint8_t *tiles;     // [H_kv][blocks] ColumnTile
  int group, nt, blocks;
  float qk_scale;
  uint32_t *status;
};

// CTA (block, KV head): one tile of columns.  The last CTA plans the runs.
template <int kDim>
__global__ void __launch_bounds__(1024) columns_kernel(const WParams p) {
  using Q = ColumnTile<kDim>;
  __shared__ long long scan[32];
  __shared__ int lowest, highest;
  const PagedView &pv = p.c.v;
  pdl_trigger();
  if (blockIdx.x == static_cast<unsigned>(p.blocks) * pv.H_kv) {
    const int n = plan_runs(pv, kTile, scan, p.runs, p.status);
    if (threadIdx.x == 0) *p.n_runs = n;
    return;
  }
  const int hk = blockIdx.x / p.blocks, block = blockIdx.x - hk * p.blocks;
  uint8_t *tile = p.tiles + static_cast<size_t>(blockIdx.x) * Q::total;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    lowest = INT_MAX;
    highest = -1;
  }
  __syncthreads();
  constexpr int kLanes = kDim / 8, kPer = 32 / kLanes;  // lanes of a column, columns of a load
  const int ch = lane % kLanes;
#pragma unroll
  for (int e = 0; e < 4; e += kPer) {
    const int col = 4 * warp + e + lane / kLanes, i = col / p.group, t = block * p.nt + i;
    const bool in = i < p.nt && t < pv.T;
    const int h = hk * p.group + col - i * p.group;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (in) v = reinterpret_cast<const uint4 *>(p.q + (static_cast<int64_t>(t) * pv.H + h) * kDim)[ch];
    uint32_t u[4] = {v.x, v.y, v.z, v.w};
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
    *reinterpret_cast<uint4 *>(tile + Q::q + (ch >> 3) * Q::kBlock + sw128_offset(col, 16u * (ch & 7))) =
        make_uint4(u[0], u[1], u[2], u[3]);
    if (ch == 0) {
      // padding columns add 2^-inf whatever the key (their queries are zeros)
      float cs = 0.f, ls = -INFINITY;
      int limit = -1;
      if (in) {
        const float l = p.lse[static_cast<int64_t>(t) * pv.H + h];
        const int pos = pv.q_pos[t], b = pv.q_seq[t];
        cs = p.qk_scale / f;
        ls = -l * kLog2e;
        if (b >= 0 && b < pv.B && pos >= 0 && (pos >> pv.logP) < pv.max_pages && l != -INFINITY) limit = pos;
        atomicMin(&lowest, limit);
        atomicMax(&highest, limit);
      }
      float *fc = reinterpret_cast<float *>(tile + Q::factor) + (col >> 1) * 4 + (col & 1);
      fc[0] = cs;
      fc[2] = ls;
      reinterpret_cast<int *>(tile + Q::limit)[col] = limit;
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) *reinterpret_cast<int2 *>(tile + Q::low) = make_int2(lowest, highest);
}

__device__ __forceinline__ bool wait_warp(uint64_t *bar, uint32_t parity) {
  return __all_sync(0xffffffffu, mbar_test_wait(bar, parity)) || mbar_wait_warp(bar, parity);
}

template <int kDim>
__global__ void __launch_bounds__(kThreads, 1) weights_umma_kernel(const WParams p) {
  using L = WSmem<kDim>;
  using Q = ColumnTile<kDim>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  ItemInfo *infos = reinterpret_cast<ItemInfo *>(smem + L::info);
  float *sums = reinterpret_cast<float *>(smem + L::sums);
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::bars);
  uint64_t *kfull = bars, *kempty = kfull + 2, *qfull = kempty + 2, *qempty = qfull + L::kSlots, *cfull = qempty + L::kSlots;
  uint64_t *cempty = cfull + kConsts, *sfull = cempty + kConsts;
  uint64_t *sempty = sfull + kBufs, *ifull = sempty + kBufs, *iempty = ifull + kInfos, *meet = iempty + kInfos, *done = meet + 2;
  uint32_t *tmem_base_s = reinterpret_cast<uint32_t *>(smem + L::misc);
  volatile int *abort_s = reinterpret_cast<volatile int *>(smem + L::misc + 4);
  const PagedView &pv = p.c.v;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&kfull[i], 4);
      mbar_init(&kempty[i], 1);
      mbar_init(&meet[i], i == 0 ? 4 * (kGroups - 1) : 4);  // [0]: the further warpgroups' sums are there; [1]: they have been read
    }
    for (int i = 0; i < L::kSlots; ++i) {
      mbar_init(&qfull[i], 1);
      mbar_init(&qempty[i], 1);
    }
    for (int i = 0; i < kConsts; ++i) {
      mbar_init(&cfull[i], 1);
      mbar_init(&cempty[i], 4);
    }
    for (int i = 0; i < kBufs; ++i) {
      mbar_init(&sfull[i], 1);
      mbar_init(&sempty[i], 4);
    }
    for (int i = 0; i < kInfos; ++i) {
      mbar_init(&ifull[i], 1);
      mbar_init(&iempty[i], 4 * kGroups + 6);  // softmax, converting, issuing and copying warps
    }
    mbar_init(done, 1);
    *abort_s = 0;
    fence_barrier_init();
  }
  if (warp == kWarpMma) {
    tmem_alloc(tmem_base_s, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_base_s;
  pdl_wait();
  const int runs = *p.n_runs;
  const long long total = p.runs.off[runs];
  // CTA c takes the items c, c + grid, ..
  const int items = blockIdx.x < total ? static_cast<int>((total - blockIdx.x + gridDim.x - 1) / gridDim.x) : 0;
  auto fail = [&]() {
    raise_flag(p.status, kFlagTimeout);
    *abort_s = 1;
  };
  bool ok = true;
  // Reads item n's description; every warp that calls it does so once per item.
  auto item_of = [&](int n, ItemInfo &it) {
    ok = wait_warp(&ifull[n % kInfos], (n / kInfos) & 1) && !*abort_s;
    if (!ok) return false;
    it = infos[n % kInfos];
    __syncwarp();
    if (lane == 0) mbar_arrive(&iempty[n % kInfos]);
    return true;
  };

  if (warp == kWarpInfo) {
    for (int n = 0; n < items && ok; ++n) {
      const long long x = blockIdx.x + static_cast<long long>(n) * gridDim.x;
      const int run = run_of_tile(p.runs.off, runs, x);
      const int last = p.runs.last[run], cost = (last + kTile) / kTile;
      const int t0 = p.runs.t0[run], t1 = p.runs.t0[run + 1], seq = pv.q_seq[t0];
      const TilePlace place = tile_place(x - p.runs.off[run], cost);
      const int hk = place.head, base = place.tile * kTile;
      const int slot = base + 16 * lane;
      int id = -1;
      if (lane < 8 && slot <= last) id = load_page(pv, seq, slot >> pv.logP, p.status, true);
      const uint32_t have = __ballot_sync(0xffffffffu, id >= 0);
      // the first token block with a column that sees a slot of the item (a prompt's
      // tokens ascend, so those before it see none)
      int b0 = t0 / p.nt, b1 = (t1 - 1) / p.nt;
      for (; b0 <= b1; b0 += 32) {
        int hi = -1;
        if (b0 + lane <= b1)
          hi = reinterpret_cast<const int2 *>(p.tiles + (static_cast<size_t>(hk) * p.blocks + b0 + lane) * Q::total + Q::low)->y;
        const uint32_t sees = __ballot_sync(0xffffffffu, hi >= base);
        if (sees) {
          b0 += __ffs(sees) - 1;
          break;
        }
      }
      if (have == 0) b0 = b1 + 1;
      ok = wait_warp(&iempty[n % kInfos], ((n / kInfos) & 1) ^ 1) && !*abort_s;
      if (!ok) break;
      if (lane == 0) {
        infos[n % kInfos] = ItemInfo{t0, t1, seq, hk, base, last, have, b0, b1, {}};
        mbar_arrive(&ifull[n % kInfos]);
      }
    }
    if (!ok && lane == 0) fail();
  } else if (warp == kWarpCopy) {
    // -------------------------------------------------- tiles of columns
    const bool leader = elect_one();
    int m = 0;
    for (int n = 0; n < items && ok; ++n) {
      ItemInfo it;
      if (!item_of(n, it)) break;
      for (int b = it.b0; b <= it.b1; ++b, ++m) {
        const int s = m % L::kSlots;
        const int cslot = m % kConsts;
        ok = wait_warp(&qempty[s], ((m / L::kSlots) & 1) ^ 1) && wait_warp(&cempty[cslot], ((m / kConsts) & 1) ^ 1) &&
             !*abort_s;
        if (!ok) break;
        if (leader) {
          const uint8_t *src = p.tiles + (static_cast<size_t>(it.hk) * p.blocks + b) * Q::total;
          mbar_expect_tx(&qfull[s], L::kQ);
          bulk_load(smem + L::q + s * L::kQ, src, L::kQ, &qfull[s]);
          mbar_expect_tx(&cfull[cslot], Q::consts);
          bulk_load(smem + L::consts + cslot * Q::consts, src + Q::factor, Q::consts, &cfull[cslot]);
        }
        __syncwarp();
      }
    }
    if (lane == 0) {
      if (!ok) fail();
      // every copy lands before the CTA exits
      for (int k = max(0, m - L::kSlots); k < m; ++k) mbar_wait(&qfull[k % L::kSlots], (k / L::kSlots) & 1);
      for (int k = max(0, m - kConsts); k < m; ++k) mbar_wait(&cfull[k % kConsts], (k / kConsts) & 1);
    }
    __syncwarp();
  } else if (warp == kWarpMma) {
    const bool leader = elect_one();
    constexpr uint32_t idesc = (1u << 4) | (static_cast<uint32_t>(kTile >> 3) << 17) | (static_cast<uint32_t>(128 >> 4) << 24);
    int m = 0, live = 0;
    for (int n = 0; n < items && ok; ++n) {
      ItemInfo it;
      if (!item_of(n, it)) break;
      if (it.b0 > it.b1) continue;
      const int ks = live % 2;
      ok = wait_warp(&kfull[ks], (live / 2) & 1);
      if (!ok) break;
      tc_fence_after();
      const uint32_t ka = __reduce_or_sync(0xffffffffu, smem_u32(smem + L::keys + ks * L::kKeys));
      for (int b = it.b0; b <= it.b1; ++b, ++m) {
        const int s = m % L::kSlots, buf = m % kBufs;
        ok = wait_warp(&qfull[s], (m / L::kSlots) & 1) && wait_warp(&sempty[buf], ((m / kBufs) & 1) ^ 1) && !*abort_s;
        if (!ok) break;
        tc_fence_after();
        const uint32_t qa = __reduce_or_sync(0xffffffffu, smem_u32(smem + L::q + s * L::kQ));
        if (leader) {
          const uint64_t da = desc_sw128_kmajor(ka), db = desc_sw128_kmajor(qa);
#pragma unroll
          for (int kk = 0; kk < kDim / 16; ++kk) {
            const uint64_t o = ((kk >> 2) * Q::kBlock + (kk & 3) * 32) >> 4;
            mma_f16(tmem + 128 * buf, da + o, db + o, idesc, kk > 0);
          }
          mma_commit(&sfull[buf]);
          mma_commit(&qempty[s]);
          if (b == it.b1) mma_commit(&kempty[ks]);
        }
        __syncwarp();
      }
      ++live;
    }
    if (!ok && lane == 0) fail();
    if (leader && items > 0) {
      mma_commit(done);
      if (!mbar_wait(done, 0)) raise_flag(p.status, kFlagTimeout);
    }
    __syncwarp();
  } else if (warp >= kWarpConv && warp < kWarpMma) {
    // ---------------------------- codes to an fp16 tile: 32 rows of keys each
    const int cw = warp - kWarpConv;
    constexpr int kItems = kDim / 32, kRows = 32 / kItems;
    const int seg = kDim == 128 ? (lane & 1) + 2 * (lane >> 4) : lane & 1;
    const int of = 32 * cw + (kDim == 128 ? (lane >> 1) & 7 : lane >> 1);
    int live = 0;
    for (int n = 0; n < items && ok; ++n) {
      ItemInfo it;
      if (!item_of(n, it)) break;
      if (it.b0 > it.b1) continue;
      uint4 c[kItems];
      uint32_t sc[kItems];
#pragma unroll
      for (int e = 0; e < kItems; ++e) {
        const int row = of + kRows * e, slot = it.base + row;
        c[e] = make_uint4(0, 0, 0, 0);
        sc[e] = 0;
        if (slot <= it.last) {
          const int id = load_page(pv, it.seq, slot >> pv.logP, nullptr, false);
          if (id >= 0) {
            const int64_t at = (static_cast<int64_t>(id * pv.H_kv + it.hk) << pv.logP) + (slot & (pv.P - 1));
            c[e] = reinterpret_cast<const uint4 *>(p.c.K + at * (kDim / 2))[seg];
            sc[e] = reinterpret_cast<const uint16_t *>(p.c.Ks + at * (kDim / 16))[seg];
          }
        }
      }
      const int ks = live % 2;
      ok = wait_warp(&kempty[ks], ((live / 2) & 1) ^ 1) && !*abort_s;
      if (!ok) break;
      uint8_t *dst = smem + L::keys + ks * L::kKeys + (seg >> 1) * Q::kBlock;
#pragma unroll
      for (int e = 0; e < kItems; ++e) {
        const __half2 two = e4m3x2_to_half2(sc[e]);
        const uint32_t words[4] = {c[e].x, c[e].y, c[e].z, c[e].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const __half2 s2 = j < 2 ? __low2half2(two) : __high2half2(two);
          __half2 d[4];
          e2m1x8_to_half2(words[j], d);
          *reinterpret_cast<uint4 *>(dst + sw128_offset(of + kRows * e, 64 * (seg & 1) + 16 * j)) =
              make_uint4(as_u32(__hmul2(d[0], s2)), as_u32(__hmul2(d[1], s2)), as_u32(__hmul2(d[2], s2)),
                         as_u32(__hmul2(d[3], s2)));
        }
      }
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(&kfull[ks]);
      ++live;
    }
    if (!ok && lane == 0) fail();
  } else if (warp < kWarpConv) {
    // ------------------------------- sums: a warpgroup takes every kGroups-th tile
    const int w = warp >> 2, row = tid & 127;
    const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    int m = 0, met = 0;
    for (int n = 0; n < items && ok; ++n) {
      ItemInfo it;
      if (!item_of(n, it)) break;
      if (it.b0 > it.b1) continue;
      const int slot = it.base + row;
      const bool held = slot <= it.last && ((it.have >> (row >> 4)) & 1u);
      float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
      for (int b = it.b0; b <= it.b1; ++b, ++m) {
        if (m % kGroups != w) continue;
        const int cslot = m % kConsts, buf = m % kBufs;
        ok = wait_warp(&sfull[buf], (m / kBufs) & 1) && wait_warp(&cfull[cslot], (m / kConsts) & 1) && !*abort_s;
        if (!ok) break;
        tc_fence_after();
        const uint8_t *tile = smem + L::consts + cslot * Q::consts - Q::factor;
        // columns of this run, and whether all of them see all of the keys
        const int tb = b * p.nt, te = min(tb + p.nt, pv.T);
        const bool all = tb >= it.t0 && te <= it.t1 &&
                         reinterpret_cast<const int *>(tile + Q::low)[0] >= it.base + kTile - 1;
        const int c0 = (it.t0 - tb) * p.group, c1 = (min(it.t1, te) - tb) * p.group;
        const float4 *fc = reinterpret_cast<const float4 *>(tile + Q::factor);
        const int *limit = reinterpret_cast<const int *>(tile + Q::limit);
        // 32 columns at a time, the next ones on their way
        float v[2][32];
        const uint32_t at = tmem + lanes + 128 * buf;
        tmem_load(at, reinterpret_cast<uint32_t(&)[32]>(v[0][0]));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          tmem_ld_wait();
          if (i < 3) tmem_load(at + 32 * (i + 1), reinterpret_cast<uint32_t(&)[32]>(v[(i + 1) & 1][0]));
          float2 *v2 = reinterpret_cast<float2 *>(v[i & 1]);
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float4 f = fc[16 * i + e];
            v2[e] = fma2(v2[e], make_float2(f.x, f.y), make_float2(f.z, f.w));
          }
          if (all) {
#pragma unroll
            for (int e = 0; e < 16; ++e) sum[e & 1] = add2(sum[e & 1], make_float2(exp2_hw(v2[e].x), exp2_hw(v2[e].y)));
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const int c = 32 * i + e;
              if (c >= c0 && c < c1 && slot <= limit[c]) sum[0].x += exp2_hw(v[i & 1][e]);
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&sempty[buf]);
          mbar_arrive(&cempty[cslot]);
        }
      }
      if (!ok) break;
      // the warpgroups' sums, the first's first
      sum[0] = add2(sum[0], sum[1]);
      const float own = sum[0].x + sum[0].y;
      if (w > 0) {
        ok = wait_warp(&meet[1], (met & 1) ^ 1);  // (those of the item before have been read)
        if (!ok) break;
        sums[128 * (w - 1) + row] = own;
        __syncwarp();
        if (lane == 0) mbar_arrive(&meet[0]);
        ++met;
      } else {
        ok = wait_warp(&meet[0], met & 1);
        if (!ok) break;
        float both = own;
#pragma unroll
        for (int i = 0; i < kGroups - 1; ++i) both += sums[128 * i + row];
        __syncwarp();
        if (lane == 0) mbar_arrive(&meet[1]);
        ++met;
        // one addition a slot and run (a sequence in several runs adds in any order)
        if (held) atomicAdd(p.weight + (static_cast<int64_t>(it.seq) * pv.H_kv + it.hk) * p.ld + slot, both);
      }
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

struct Shape {
  int nt, blocks;
  size_t off, t0, last, n, tiles, total;
};
Shape shape_of(const sa_paged4_args &pa) {
  Shape s{};
  s.nt = std::max(1, kTile / (pa.p.H / pa.p.H_kv));
  s.blocks = (pa.p.T + s.nt - 1) / s.nt;
  const size_t tile = pa.p.D == 128 ? ColumnTile<128>::total : ColumnTile<64>::total;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t was = at;
    at += round_up(bytes);
    return was;
  };
  s.off = take((static_cast<size_t>(pa.p.T) + 2) * 8);
  s.t0 = take((static_cast<size_t>(pa.p.T) + 2) * 4);
  s.last = take((static_cast<size_t>(pa.p.T) + 2) * 4);
  s.n = take(4);
  s.tiles = take(static_cast<size_t>(s.blocks) * pa.p.H_kv * tile);
  s.total = at;
  return s;
}

template <int kDim>
cudaError_t launch(const WParams &p, cudaStream_t stream) {
  cudaError_t e = launch_ex(false, columns_kernel<kDim>, dim3(static_cast<unsigned>(p.blocks) * p.c.v.H_kv + 1), dim3(1024), 0,
                            stream, 1, p);
  if (e != cudaSuccess) return e;
  auto kern = weights_umma_kernel<kDim>;
  static bool done[64] = {};
  e = set_smem_once(reinterpret_cast<const void *>(kern), WSmem<kDim>::total + 1024, done);
  if (e != cudaSuccess) return e;
  return launch_ex(true, kern, dim3(sm_count()), dim3(kThreads), WSmem<kDim>::total + 1024, stream, 1, p);
}

}  // namespace

size_t weights4_umma_scratch(const sa_paged4_args &pa) { return shape_of(pa).total; }

cudaError_t launch_weights4_umma(const sa_paged4_args &pa, const void *q, const float *lse, float *weight, int64_t ld,
                                 void *scratch, uint32_t *status, cudaStream_t stream) {
  const Shape s = shape_of(pa);
  char *w = static_cast<char *>(scratch);
  WParams p;
  p.c = paged4_view(pa);
  p.q = static_cast<const uint16_t *>(q);
  p.lse = lse;
  p.weight = weight;
  p.ld = ld;
  p.runs = Runs{reinterpret_cast<int *>(w + s.t0), reinterpret_cast<int *>(w + s.last), reinterpret_cast<long long *>(w + s.off)};
  p.n_runs = reinterpret_cast<int *>(w + s.n);
  p.tiles = reinterpret_cast<uint8_t *>(w + s.tiles);
  p.group = pa.p.H / pa.p.H_kv;
  p.nt = s.nt;
  p.blocks = s.blocks;
  p.qk_scale = pa.p.scale * pa.k_gain * kLog2e;
  p.status = status;
  return pa.p.D == 128 ? launch<128>(p, stream) : launch<64>(p, stream);
}

}  // namespace sa
