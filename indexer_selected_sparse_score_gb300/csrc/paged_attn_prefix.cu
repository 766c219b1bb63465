// Attention of a batch whose sequences share their first pages, on the 5th-
// generation tensor cores.
//
// The shared keys are met by every query row of the batch (T tokens x G heads
// per KV head), so that part is two dense products with a softmax between them
// and bound by the tensor pipe once there are a few hundred rows (4 D flops a
// row and key against 4 D / rows bytes); with few rows it streams the shared
// pages once and HBM is the bound.  The rows sit in the accumulator's lanes:
//   S = Q K^T   M = 128 rows, N = 128 keys, K = D; a thread owns a row, so the
//               running maximum and sum need no exchange between threads
//   P           bf16, written over S in tensor memory (the A operand of P V)
//   O += P V    M = 128 rows, N = D, K = 128 keys, V read MN-major as it landed
// A CTA holds two row tiles (A, B: 256 rows) against the same K and V tiles,
// each with its own softmax warpgroup and its own issuing warp; the issuers take
// turns, so one tile's products run while the other's weights are computed.  A
// row's logits are taken relative to a reference set by the piece's first tile;
// only when a vote of the warp finds one that passes it by 2^8 is it raised and O
// rescaled.  Weights are rounded to bf16 for the product (2^-8 of each at most);
// logits, statistics and O are fp32.
//
// Work: (KV head, 256 rows) items x key tiles form one list cut evenly over one
// CTA per SM.  Every piece leaves (reference, sum) and O per row in scratch.
// The positions past the shared pages, each sequence's own, are a page-list
// call (paged_attn_list.cu) that starts as SMs fall free, and a last kernel
// merges a row's pieces of both.
//
// Measured, heads of 128: 128 tokens of 64 heads over one KV head behind 32 K
// shared keys 116 us, 1.20 PFLOP/s over the whole call (the shared product runs
// at about 1.5 on the 128 SMs it gets; the own pages' list and the merge, 5 us,
// are the rest).  64 tokens of 64 over 8 heads, 32 K shared and up to 1500 own
// keys: 86 us, 4.2 TB/s of the 360 MB it must read beside 0.8 PFLOP/s.  4 tokens
// of 16 over 2 heads, 4160 shared keys: 14 us, three launches.
#include <cudaTypedefs.h>

#include <algorithm>

#include "internal.h"
#include "paged.cuh"
#include "paged_bounds.h"
#include "paged_list.h"
#include "paged_umma.cuh"

namespace sa {
namespace {

using namespace umma;

constexpr int kTile = 128;      // keys per tile, rows per row tile
constexpr int kRows = 256;      // rows per item
constexpr int kThreads = 384;
constexpr int kMaxCtas = 256;   // one CTA per SM
constexpr int kWarpMma = 8;     // and 9: the issuers of row tiles A and B
constexpr int kWarpLoad = 10;   // (warp 11 only joins the block barriers)
constexpr int kSlots = 5;       // ring of K and V tiles: K(0), V(0), K(1), ...
constexpr int kMasks = 8;
// Registers per thread: built for 168 (384 threads); the two softmax warpgroups
// raise their limit and the third lowers its own, 2 * 208 + 88 <= 3 * 168.
constexpr int kLaunchRegs = 168, kSoftmaxRegs = 208, kOtherRegs = 88;
static_assert(2 * kSoftmaxRegs + kOtherRegs <= 3 * kLaunchRegs, "register split exceeds the launch allocation");
constexpr float kLazy = 8.f, kHead = 20.f;  // as in paged_attn_list.cu

struct PrefixParams {
  PagedView pv;
  int pages;                  // shared pages
  int group;
  int64_t rows;               // T * group
  int npairs, nkt;            // items per KV head, key tiles per item
  const uint16_t *q;
  float *part;                // [piece][kRows][D]
  float2 *ml;                 // [piece][kRows]
  float qk_scale;
  uint32_t *status;
};

template <int kDim>
struct PrefixSmem {
  static constexpr uint32_t kBlock = kTile * 128;
  static constexpr uint32_t kKv = kBlock * (kDim / 64);
  static constexpr size_t q = 0;                           // [row tile][D / 64][128 rows][128 B]
  static constexpr size_t kv = q + 2 * kKv;
  static constexpr size_t masks = kv + kSlots * kKv;       // [kMasks] u32: bit g = keys 16 g .. + 15 exist
  static constexpr size_t bars = masks + kMasks * 4;
  static constexpr int kBars = 2 * kSlots + 10 + kMasks + 4;
  static constexpr size_t misc = bars + kBars * 8;
  static constexpr size_t total = misc + 16;
  static_assert(total + 1024 <= 232448, "shared memory budget");
};

// Walk over a CTA's tiles: item, key tile within it, and whether the tile is the
// first or last of this CTA's piece of the item.
struct Walk {
  int64_t left;  // tiles after this one
  int item, kt, nkt;
  bool first;
  __device__ Walk(int64_t x0, int64_t x1, int nkt_) : left(x1 - x0 - 1), nkt(nkt_), first(true) {
    item = static_cast<int>(x0 / nkt);
    kt = static_cast<int>(x0 - static_cast<int64_t>(item) * nkt);
  }
  __device__ bool on() const { return left >= 0; }
  __device__ bool last() const { return left == 0 || kt + 1 == nkt; }
  __device__ void next() {
    --left;
    first = ++kt == nkt;
    if (first) {
      kt = 0;
      ++item;
    }
  }
};

// The CTA whose range of the tile list [tot c / G, tot (c + 1) / G) holds tile y.
__host__ __device__ inline int cta_of(int64_t y, int64_t tot, int G) { return static_cast<int>(((y + 1) * G - 1) / tot); }

template <int kDim>
__global__ void __launch_bounds__(kThreads, 1)
prefix_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
              const PrefixParams p) {
  using L = PrefixSmem<kDim>;
  constexpr int kB = kDim / 64;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t *qs = smem + L::q, *kvs = smem + L::kv;
  uint32_t *masks = reinterpret_cast<uint32_t *>(smem + L::masks);
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::bars);
  uint64_t *full = bars, *empty = full + kSlots;
  uint64_t *qfull = empty + kSlots, *sfull = qfull + 2, *pfull = sfull + 2, *ofull = pfull + 4;  // pfull: [tile][half]
  uint64_t *mfull = ofull + 2, *turn = mfull + kMasks, *done = turn + 2;
  uint32_t *tmem_base_s = reinterpret_cast<uint32_t *>(smem + L::misc);
  volatile int *abort_s = reinterpret_cast<volatile int *>(smem + L::misc + 8);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = gridDim.x, c = blockIdx.x;
  pdl_trigger();
  if (tid == 0) {
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 2);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&qfull[i], 4);
      mbar_init(&sfull[i], 1);
      mbar_init(&pfull[2 * i], 4);
      mbar_init(&pfull[2 * i + 1], 4);
      mbar_init(&ofull[i], 1);
      mbar_init(&turn[i], 1);
      mbar_init(&done[i], 1);
    }
    for (int i = 0; i < kMasks; ++i) mbar_init(&mfull[i], 1);
    *abort_s = 0;
    fence_barrier_init();
  }
  if (warp == kWarpMma) {
    tmem_alloc(tmem_base_s, 512);
    tmem_relinquish();
  }
  const int64_t tot = static_cast<int64_t>(p.pv.H_kv) * p.npairs * p.nkt;
  const int64_t x0 = tot * c / G, x1 = tot * (c + 1) / G;
  // A softmax warp's 32 query rows of an item, into the K-major swizzled layout;
  // a load covers whole rows.
  constexpr int kLanes = kDim / 8, kPer = 32 / kLanes;  // lanes of a row, rows of a load
  auto load_queries = [&](int item) {
    uint4 v[32 / kPer];
    const int hk = item / p.npairs, ch = lane % kLanes;
    // row r is head r % group of token r / group
    int r = (item - hk * p.npairs) * kRows + 128 * (warp >> 2) + 32 * (warp & 3) + lane / kLanes;
    int t = r / p.group, g = r - t * p.group;
#pragma unroll
    for (int i = 0; i < 32 / kPer; ++i, r += kPer, g += kPer) {
      while (g >= p.group) {
        g -= p.group;
        ++t;
      }
      const int64_t src = static_cast<int64_t>(t) * p.pv.H + hk * p.group + g;
      v[i] = make_uint4(0, 0, 0, 0);
      if (r < p.rows) v[i] = reinterpret_cast<const uint4 *>(p.q + src * kDim)[ch];
    }
    uint8_t *dst = qs + (warp >> 2) * L::kKv + (ch >> 3) * L::kBlock;
#pragma unroll
    for (int i = 0; i < 32 / kPer; ++i)
      *reinterpret_cast<uint4 *>(dst + sw128_offset(32 * (warp & 3) + kPer * i + lane / kLanes, 16u * (ch & 7))) = v[i];
  };
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_base_s;
  auto fail = [&]() {
    raise_flag(p.status, kFlagTimeout);
    *abort_s = 1;
  };

  if (warp >= 8) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
  if (warp == kWarpLoad) {
    // ------------------------------------------------------------------ loader
    if (lane == 0) {
      prefetch_tmap(&kmap);
      prefetch_tmap(&vmap);
    }
    const int spt = kTile >> p.pv.logP;
    const uint32_t rows_total = static_cast<uint32_t>(p.pv.n_pages) * p.pv.H_kv * p.pv.P;
    const int q = lane / kB, kb = lane % kB;  // this lane's copy: page slot q of the tile, 64-dim block kb
    auto page_of = [&](int kt) -> int {
      const int j = kt * spt + q;
      return q < spt && j < p.pages ? load_page(p.pv, 0, j, p.status, true) : -1;
    };
    bool ok = true;
    int n = 0, issued = 0;
    Walk at(x0, x1, p.nkt);
    int next = at.on() ? page_of(at.kt) : -1;
    for (; at.on() && ok; at.next(), ++n) {
      const int page = next;
      if (at.left > 0) next = page_of(at.kt + 1 == p.nkt ? 0 : at.kt + 1);
      const int hk = at.item / p.npairs;
      // a slot without a page reads past the tensor's end: the copy fills zeros
      const uint32_t y = page >= 0 ? (static_cast<uint32_t>(page) * p.pv.H_kv + hk) * p.pv.P : rows_total;
      // mask: P / 16 bits per page slot
      const uint32_t have = __ballot_sync(0xffffffffu, page >= 0 && kb == 0);
      uint32_t mask = 0;
      for (int g = 0; g < 8; ++g) mask |= ((have >> (((16 * g) >> p.pv.logP) * kB)) & 1u) << g;
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        const int m = 2 * n + kv, s = m % kSlots;
        if (!mbar_wait_warp(&empty[s], ((m / kSlots) & 1) ^ 1) || *abort_s) {
          ok = false;
          break;
        }
        if (lane == 0) {
          if (kv == 0) {
            masks[n % kMasks] = mask;
            mbar_arrive(&mfull[n % kMasks]);
          }
          mbar_expect_tx(&full[s], L::kKv);
        }
        __syncwarp();
        ++issued;
        if (q < spt)
          tma_load_2d(kvs + s * L::kKv + kb * L::kBlock + q * p.pv.P * 128, kv ? &vmap : &kmap, &full[s], 64 * kb,
                      static_cast<int>(y));
      }
      if (!ok) break;
    }
    if (lane == 0) {
      if (!ok) fail();
      // every copy lands before the CTA exits
      for (int m = max(0, issued - kSlots); m < issued; ++m) mbar_wait(&full[m % kSlots], (m / kSlots) & 1);
    }
    __syncwarp();
  } else if (warp == kWarpMma || warp == kWarpMma + 1) {
    // ------------------------------------------------- issuer of one row tile
    // The two issuers take turns: O_A(n), S_A(n + 1), then O_B(n), S_B(n + 1),
    // so that the softmax of one row tile runs while the products of the other
    // do.  (Without turns the tensor core took both tiles' products together and
    // idled while both softmaxes ran; with one issuer for both, its waits lay
    // between the products.)  A turn is waited for last, when the inputs are in.
    const int w = warp - kWarpMma;
    const bool leader = elect_one();
    constexpr uint32_t idesc_s = idesc_bf16(128, kTile);
    constexpr uint32_t idesc_o = idesc_bf16(128, kDim) | (1u << 16);  // V is MN-major
    const uint32_t ts = tmem + 128 * w, to = tmem + 256 + 128 * w;
    const uint64_t dq = desc_sw128_kmajor(smem_u32(qs + w * L::kKv));
    bool ok = true, two = false, live = false;  // row tile B, this row tile has rows
    int n = 0, qn = 0, ln = 0, turns = 0;
    auto take_turn = [&]() -> bool {
      if (!two) return true;
      const int k = turns++;
      return w == 0 ? k == 0 || mbar_wait_warp(&turn[1], (k - 1) & 1) : mbar_wait_warp(&turn[0], k & 1);
    };
    auto issue_s = [&](int slot) {
      if (leader) {
        const uint64_t db = desc_sw128_kmajor(smem_u32(kvs + slot * L::kKv));
#pragma unroll
        for (int kk = 0; kk < kDim / 16; ++kk) {
          const uint64_t o = ((kk >> 2) * L::kBlock + (kk & 3) * 32) >> 4;
          mma_f16(ts, dq + o, db + o, idesc_s, kk > 0);
        }
        mma_commit(&sfull[w]);
        mma_commit(&empty[slot]);
      }
    };
    for (Walk at(x0, x1, p.nkt); at.on(); at.next(), ++n) {
      const bool first = at.first, last = at.last();
      const int m = 2 * n, v = m + 1, k = m + 2;
      if (first) {
        two = static_cast<int64_t>(at.item % p.npairs) * kRows + 128 < p.rows;
        live = w == 0 || two;
      }
      if (!live) {  // only frees the ring
        ok = mbar_wait_warp(&full[m % kSlots], (m / kSlots) & 1);
        if (ok && leader) mbar_arrive(&empty[m % kSlots]);
        ok = ok && mbar_wait_warp(&full[v % kSlots], (v / kSlots) & 1);
        if (!ok) break;
        if (leader) mbar_arrive(&empty[v % kSlots]);
        __syncwarp();
        continue;
      }
      if (first) {
        ok = mbar_wait_warp(&full[m % kSlots], (m / kSlots) & 1) && mbar_wait_warp(&qfull[w], (qn++) & 1) && take_turn();
        if (!ok) break;
        tc_fence_after();
        issue_s(m % kSlots);
        if (leader && two) mbar_arrive(&turn[w]);
        __syncwarp();
      }
      ok = mbar_wait_warp(&full[v % kSlots], (v / kSlots) & 1) &&
           (last || mbar_wait_warp(&full[k % kSlots], (k / kSlots) & 1)) && mbar_wait_warp(&pfull[2 * w], ln & 1) &&
           take_turn();
      if (!ok || *abort_s) break;
      tc_fence_after();
      const uint64_t dv = desc_mn(smem_u32(kvs + (v % kSlots) * L::kKv), L::kBlock);
      if (leader) {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)  // keys 0-63
          mma_f16_tmem_a(to, ts + 8 * kk, dv + ((kk * 2048) >> 4), idesc_o, !(first && kk == 0));
      }
      ok = mbar_wait_warp(&pfull[2 * w + 1], ln & 1);
      if (!ok) break;
      tc_fence_after();
      if (leader) {
#pragma unroll
        for (int kk = 4; kk < 8; ++kk) mma_f16_tmem_a(to, ts + 8 * kk, dv + ((kk * 2048) >> 4), idesc_o, 1);
        mma_commit(last ? &ofull[w] : &empty[v % kSlots]);
        if (last) mma_commit(&empty[v % kSlots]);
      }
      if (!last) issue_s(k % kSlots);
      if (leader && two) mbar_arrive(&turn[w]);
      __syncwarp();
      ++ln;
    }
    if (!ok && lane == 0) fail();
    if (leader) {
      mma_commit(&done[w]);
      if (!mbar_wait(&done[w], 0)) raise_flag(p.status, kFlagTimeout);
    }
    __syncwarp();
  } else if (warp < 8) {
    // ------------------------------------------------ softmax of one row tile
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    const int w = warp >> 2, row = tid & 127;
    const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const uint32_t ts = tmem + lanes + 128 * w, to = tmem + lanes + 256 + 128 * w;
    const float cs = p.qk_scale;
    const float2 cs2 = make_float2(cs, cs);
    uint8_t *qt = qs + w * L::kKv;
    float ref = 0.f, l = 0.f;
    int n = 0, ln = 0, pieces = 0;
    bool ok = true;
    int64_t r = 0;
    for (Walk at(x0, x1, p.nkt); at.on(); at.next(), ++n) {
      const bool first = at.first, last = at.last();
      if (first) r = static_cast<int64_t>(at.item % p.npairs) * kRows + 128 * w + row;
      if (r - row >= p.rows) continue;
      if (first) {
        // (every product of the piece before has been read out)
        load_queries(at.item);
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&qfull[w]);
        l = 0.f;
      }
      ok = mbar_wait_warp(&mfull[n % kMasks], (n / kMasks) & 1) && mbar_wait_warp(&sfull[w], ln & 1);
      if (!ok || *abort_s) break;
      const uint32_t mask = masks[n % kMasks];
      tc_fence_after();
      // the row's logits, relative to its reference
      float v[128];
#pragma unroll
      for (int i = 0; i < 4; ++i) tmem_load(ts + 32 * i, reinterpret_cast<uint32_t(&)[32]>(v[32 * i]));
      tmem_ld_wait();
      if (mask != 0xFFu) {
#pragma unroll
        for (int e = 0; e < 128; ++e)
          if (!((mask >> (e >> 4)) & 1u)) v[e] = cs > 0.f ? -INFINITY : INFINITY;  // cs v = -inf
      }
      // A sum of 0: the piece has met no key of the row yet.  Its logits are then
      // taken against 0, so that none is lost to a placeholder.
      if (first) ref = 0.f;
      const bool fresh = l == 0.f;
      float2 *v2 = reinterpret_cast<float2 *>(v);
      float top = -INFINITY;
      {
        const float2 nref2 = make_float2(-ref, -ref);
        float t4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int e = 0; e < 64; ++e) {
          v2[e] = fma2(v2[e], cs2, nref2);
          t4[e & 3] = max3(t4[e & 3], v2[e].x, v2[e].y);
        }
        top = fmaxf(max3(t4[0], t4[1], t4[2]), t4[3]);
      }
      if (__any_sync(0xffffffffu, fresh || top > kLazy - kHead)) {
        // the row's first keys, or a logit passes its reference by the lazy
        // margin: set or raise it; the sum and O (which holds the products up to
        // the tile before) shrink in step.  A tile without a key leaves it at 0.
        const float up = top == -INFINITY ? 0.f : fresh ? top + kHead : fmaxf(top + kHead, 0.f);
        const float2 nup2 = make_float2(-up, -up);
        ref += up;
#pragma unroll
        for (int e = 0; e < 64; ++e) v2[e] = add2(v2[e], nup2);
        if (!first) {
          const float fac = exp2f(fminf(-up, 0.f));  // (above 1 for a sum of 0 only)
          l *= fac;
#pragma unroll 1
          for (int i = 0; i < kDim / 16; ++i) {
            uint32_t o[16];
            tmem_load(to + 16 * i, o);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * fac);
            tmem_store(to + 16 * i, o);
          }
          tmem_wait_st();
        }
      }
      // weights, half a tile at a time: the product over the first 64 keys
      // starts while the second half's are computed
      float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t pk[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const float2 x = v2[32 * half + e];
          const float2 w2 = make_float2(exp2_hw(x.x), exp2_hw(x.y));
          sum[e & 1] = add2(sum[e & 1], w2);
          pk[e] = pack_bf16x2(w2.x, w2.y);
        }
        tmem_store(ts + 32 * half, pk);
        tmem_store(ts + 32 * half + 16, pk + 16);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&pfull[2 * w + half]);
      }
      const float2 sum2 = add2(sum[0], sum[1]);
      l += sum2.x + sum2.y;
      ++ln;
      if (last) {
        ok = mbar_wait_warp(&ofull[w], pieces & 1);
        if (!ok) break;
        ++pieces;
        tc_fence_after();
        const int64_t to_row = static_cast<int64_t>(at.item + c) * kRows + 128 * w + row;
        if (r < p.rows) p.ml[to_row] = make_float2(l == 0.f ? -INFINITY : ref, l);
        // O of the warp's rows, 32 columns at a time through this warp's part of
        // the query tile (its products are done), so that a store covers 128
        // contiguous bytes of each of four rows
        float4 *stage = reinterpret_cast<float4 *>(qt + (warp & 3) * 4096);
        const int64_t row0 = to_row - lane;
        const int64_t valid = p.rows - (r - lane);  // rows of this warp
#pragma unroll 1
        for (int i = 0; i < kDim / 32; ++i) {
          uint32_t o[32];
          tmem_load(to + 32 * i, o);
          tmem_ld_wait();
          __syncwarp();
#pragma unroll
          for (int e = 0; e < 8; ++e)
            stage[8 * lane + (e ^ (lane & 7))] =
                make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]), __uint_as_float(o[4 * e + 2]),
                            __uint_as_float(o[4 * e + 3]));
          __syncwarp();
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int rr = 4 * e + (lane >> 3), ch = lane & 7;
            if (rr < valid)
              *reinterpret_cast<float4 *>(p.part + (row0 + rr) * kDim + 32 * i + 4 * ch) = stage[8 * rr + (ch ^ (rr & 7))];
          }
        }
        __syncwarp();
        tc_fence_before();
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

// Output rows: the pieces of the shared part (of the row's item) and of the
// token's own pages.  kSplit warps per row.
template <int kDim, int kSplit>
__global__ void __launch_bounds__(256)
merge_rows_kernel(const PrefixParams p, const ListParams own, int cols, int grid_shared) {
  __shared__ float acc_s[8][kDim + 2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t id = static_cast<int64_t>(blockIdx.x) * (8 / kSplit) + warp / kSplit;
  bool ok = id < static_cast<int64_t>(p.pv.T) * p.pv.H;
  const int t = ok ? static_cast<int>(id / p.pv.H) : 0, h = ok ? static_cast<int>(id - static_cast<int64_t>(t) * p.pv.H) : 0;
  int b, pos;
  ok = ok && load_paged_token(p.pv, t, nullptr, false, b, pos) && pos >= p.pages * p.pv.P;
  const int hk = h / p.group, g = h - hk * p.group;
  const int64_t r = static_cast<int64_t>(t) * p.group + g;
  const int64_t tot = static_cast<int64_t>(p.pv.H_kv) * p.npairs * p.nkt;
  const int64_t item = static_cast<int64_t>(hk) * p.npairs + r / kRows;
  const int a0 = cta_of(item * p.nkt, tot, grid_shared), a1 = cta_of((item + 1) * p.nkt - 1, tot, grid_shared);
  const int64_t u = (static_cast<int64_t>(t) * p.pv.H_kv + hk) * own.gb + g / 64;
  pdl_wait();
  if (blockIdx.x == 0 && threadIdx.x == 0) *own.counter = 0;  // for the next call
  Merge<kDim> m;
  if (ok) {
    const int2 rng = own.info[u];
    m.add(warp % kSplit, kSplit, a1 - a0 + 1, lane, p.ml, p.part,
          [&](int k) { return (item + a0 + k) * kRows + r % kRows; });
    if (part_range_ok(rng.x, rng.y, own.parts))  // (else a wait gave up, and was flagged)
      m.add(warp % kSplit, kSplit, rng.y - rng.x + 1, lane, own.ml, own.part,
            [&](int k) { return (u + rng.x + k) * cols + g % 64; });
  }
  if (m.template join<kSplit>(acc_s, lane) && ok) m.store(own.out + id * kDim, lane);
}

size_t round_up(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

struct Shape {
  int64_t rows, items;
  int npairs, nkt, spt;
  size_t slots;
};
Shape shape_of(const sa_paged_args &pa, int pages) {
  Shape s{};
  s.spt = kTile / pa.P;
  s.rows = static_cast<int64_t>(pa.T) * (pa.H / pa.H_kv);
  s.npairs = static_cast<int>((s.rows + kRows - 1) / kRows);
  s.nkt = (pages + s.spt - 1) / s.spt;
  s.items = static_cast<int64_t>(pa.H_kv) * s.npairs;
  s.slots = static_cast<size_t>(s.items) + kMaxCtas;
  return s;
}

template <int kDim>
cudaError_t launch_shared(const sa_paged_args &pa, const PrefixParams &p, int grid, cudaStream_t stream) {
  CUtensorMap kmap, vmap;
  const uint64_t rows = static_cast<uint64_t>(pa.n_pages) * pa.H_kv * pa.P;
  if (!encode_rows(&kmap, pa.K, rows, kDim, pa.P) || !encode_rows(&vmap, pa.V, rows, kDim, pa.P))
    return cudaErrorInvalidValue;
  auto kern = prefix_kernel<kDim>;
  // the register split assumes kLaunchRegs registers per thread at launch;
  // anything else could leave a raise waiting forever
  static int regs = -1;
  if (regs < 0) {
    cudaFuncAttributes fa;
    const cudaError_t e = cudaFuncGetAttributes(&fa, reinterpret_cast<const void *>(kern));
    if (e != cudaSuccess) return e;
    regs = fa.numRegs;
  }
  if (regs != kLaunchRegs) return cudaErrorInvalidConfiguration;
  const size_t smem = PrefixSmem<kDim>::total + 1024;
  static bool attr_done[64] = {};
  cudaError_t e = set_smem_once(reinterpret_cast<const void *>(kern), smem, attr_done);
  if (e != cudaSuccess) return e;
  return launch_ex(false, kern, dim3(grid), dim3(kThreads), smem, stream, 1, kmap, vmap, p);
}

}  // namespace

size_t prefix_attn_scratch(const sa_paged_args &pa, int shared_pages) {
  if (shared_pages == 0) return list_scratch(pa, false);
  const Shape s = shape_of(pa, shared_pages);
  return list_scratch(pa, true) + round_up(s.slots * kRows * pa.D * sizeof(float)) +
         round_up(s.slots * kRows * sizeof(float2));
}

cudaError_t launch_prefix_attn(const sa_paged_args &pa, const void *q, int shared_pages, void *out, void *scratch,
                               uint32_t *status, cudaStream_t stream) {
  if (pa.T == 0) return cudaSuccess;
  ListParams own{};
  own.whole = 1;
  own.first_page = shared_pages;
  if (shared_pages == 0) return launch_page_list(pa, q, own, out, scratch, status, false, stream);
  own.keep = 1;
  const Shape s = shape_of(pa, shared_pages);
  PrefixParams p{};
  p.pv = paged_view(pa);
  p.pages = shared_pages;
  p.group = pa.H / pa.H_kv;
  p.rows = s.rows;
  p.npairs = s.npairs;
  p.nkt = s.nkt;
  p.q = static_cast<const uint16_t *>(q);
  char *w = static_cast<char *>(scratch) + list_scratch(pa, true);
  p.part = reinterpret_cast<float *>(w);
  p.ml = reinterpret_cast<float2 *>(w + round_up(s.slots * kRows * pa.D * sizeof(float)));
  // masked keys become infinite logits of the sign that the scale turns to
  // -inf, so a scale of 0 is taken as one too small to tell
  p.qk_scale = pa.scale == 0.f ? 1e-37f : pa.scale * kLog2e;
  p.status = status;
  // The page list of the sequences' own pages streams from HBM while the shared
  // part keeps the tensor cores busy: it gets SMs of its own, by the two parts'
  // costs: about 1.4 us a tile of 256 rows, and 1 us a unit and 0.75 a list tile
  // (with many heads 1.5 and 1.5), the own pages taken as half the table's.  What
  // it has left is shared out as the shared part's CTAs leave.  (The host does not
  // know the sequences' lengths, so a table much wider than they are takes SMs from
  // the shared product: 128 tokens of 64 heads behind 256 pages of 128 with 4 own
  // pages 120 us, in a table of twice the width 210; 64 of 64 over 8 behind 512
  // pages of 64 with 11 own pages 89 and 108.)
  const int sms = std::min(sm_count(), kMaxCtas);
  const bool few = list_cols(pa) == 16;
  const double shared_us = 1.4 * static_cast<double>(s.items) * s.nkt;
  const double unit_us = (few ? 1.0 : 1.5) + (few ? 0.75 : 1.5) * 0.5 * ((pa.max_pages - shared_pages + s.spt - 1) / s.spt);
  const double own_us = unit_us * static_cast<double>(pa.T) * pa.H_kv * ((pa.H / pa.H_kv + 63) / 64);
  int most = std::max(sms / 2, static_cast<int>(sms * shared_us / (shared_us + own_us) + 0.5));
  // a CTA whose range crosses into another item pays about four tiles for the
  // change (O out, queries in): with at least one CTA per item, whole CTAs per
  // item (128 x 64 heads: 134 us with 142 CTAs for 32 items, 129 with 128)
  if (s.items <= most)
    most = static_cast<int>(std::min<int64_t>(sms / s.items, (most + s.items / 2) / s.items) * s.items);
  const int grid = static_cast<int>(std::min<int64_t>(most, s.items * s.nkt));
  cudaError_t e = pa.D == 128 ? launch_shared<128>(pa, p, grid, stream) : launch_shared<64>(pa, p, grid, stream);
  if (e != cudaSuccess) return e;
  e = launch_page_list(pa, q, own, out, scratch, status, true, stream);
  if (e != cudaSuccess) return e;
  const int64_t rows = static_cast<int64_t>(pa.T) * pa.H;
  // eight or four warps to a row when it has pieces of the shared part for each
  // of them and the rows are one wave of blocks (85 tokens of 16 heads in 17
  // pieces: 43.7 us with one, 42.2 with four; 4 of 16 in 33: 20.2 with one, 16.7
  // with eight; 61 of 48 in 9: 26.1 with one, 38 with eight)
  const int64_t pieces = (grid + s.items - 1) / s.items;
  auto pays = [&](int split) { return pieces >= 2 * split && rows * split <= 40ll * sm_count(); };
  const int split = pays(8) ? 8 : pays(4) ? 4 : 1;
  const int cols = list_cols(pa);
  auto merge = [&](auto kernel) {
    const dim3 blocks(static_cast<unsigned>((rows * split + 7) / 8));
    return launch_ex(true, kernel, blocks, dim3(256), 0, stream, 1, p, own, cols, grid);
  };
  if (pa.D == 128)
    return split == 8   ? merge(merge_rows_kernel<128, 8>)
           : split == 4 ? merge(merge_rows_kernel<128, 4>)
                        : merge(merge_rows_kernel<128, 1>);
  return split == 8   ? merge(merge_rows_kernel<64, 8>)
         : split == 4 ? merge(merge_rows_kernel<64, 4>)
                      : merge(merge_rows_kernel<64, 1>);
}

}  // namespace sa
