// Slots freed by the attention weight they have gathered: selection per (sequence,
// KV head) row, and the rows that move into the freed slots.
//
// Selection: a slot's key is its weight's bits in order (recent slots count above
// all); the budget-th largest key is found by a radix select, digits of 11, 11
// and 10 bits, a histogram in shared memory each.  Of the slots of exactly that
// key the lowest stay.  What stays becomes a bit a slot; a thread counts the freed
// and the moving slots of a word of them, and the counts before it number them.
//
// Moves: freed slots before the new end are filled from behind it, so a row moves
// at most once and no more rows move than slots are freed (keeping the rows in
// order would move nearly all of them: 150 MB instead of 5 for 64 sequences of 8
// heads and 2112 slots cut to 2048).  Sources lie at or past the new end and
// destinations before it, so the moves of a call need no order.
//
// A row is one CTA's, or where rows are few, a cluster's: each of its CTAs holds the
// keys of a stretch of slots and the histograms and counts are added up over
// distributed shared memory (2 prompts of 4 heads and 16 .. 33 K slots: 26.6 us; 16 CTAs
// that each hold all of a row's keys 40.9).  64 sequences of 8 heads and 2112 slots: 22.4 us.
#include <algorithm>

#include "internal.h"
#include "paged4.cuh"
#include "umma.cuh"

namespace sa {
namespace {

using umma::cluster_ctarank;
using umma::cluster_sync;

constexpr int kBins = 2048;
constexpr int kKeysInSmem = 49152;  // of a CTA

struct EvictParams {
  Paged4View c;
  const int32_t *length, *newest;
  const float *weight;
  const int32_t *born;
  float *weight_out;
  int32_t *born_out;
  int32_t *length_out;
  int64_t ld;
  int budget, recent, D, share;
  int list;         // entries of a row's lists
  int *lists;       // [row][2][list]: freed slots, staying slots that move (clusters)
  int words;        // of a row's bits
  uint32_t *bits;   // [row][words]: slots that stay (where a CTA does not hold its keys)
  uint32_t *status;
};

// The value at the same place of shared memory in the cluster's CTA `rank`.
__device__ __forceinline__ uint32_t remote_smem(const void *p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(umma::smem_u32(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ int2 remote_int2(const int2 *p, uint32_t rank) {
  int2 v;
  asm volatile("ld.shared::cluster.v2.s32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(remote_smem(p, rank)) : "memory");
  return v;
}

// kThreads: 256 where rows are many, four CTAs to an SM; kCluster: share CTAs a row;
// kCached: a CTA's keys are held in shared memory.
template <bool kCached, int kThreads, bool kCluster>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads)
evict4_kernel(const EvictParams p) {
  constexpr int kWarps = kThreads / 32, kHists = kCluster ? 3 : 1;
  extern __shared__ __align__(16) uint32_t keys_s[];
  __shared__ __align__(16) int hist[kHists][kBins];
  __shared__ long long scan[32];
  __shared__ int2 exchange[2];
  __shared__ int2 pick;  // digit, keys above it
  __shared__ int found;  // keys of it
  const PagedView &pv = p.c.v;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int share = kCluster ? p.share : 1, rank = kCluster ? static_cast<int>(cluster_ctarank()) : 0;
  const int64_t row = blockIdx.x / share;
  const int b = static_cast<int>(row / pv.H_kv), h = static_cast<int>(row - static_cast<int64_t>(b) * pv.H_kv);
  for (int i = tid; i < kHists * kBins / 4; i += kThreads) reinterpret_cast<int4 *>(hist)[i] = make_int4(0, 0, 0, 0);
  int n = p.length[b];
  if (n < 0 || n > pv.max_pages * pv.P) {
    if (tid == 0) raise_flag(p.status, kFlagBadPos);
    n = 0;
  }
  const int keep = min(n, p.budget);
  if (h == 0 && rank == 0 && tid == 0) p.length_out[b] = keep;
  const float *weight = p.weight + row * p.ld;
  const int32_t *born = p.born + row * p.ld;
  float *weight_out = p.weight_out + row * p.ld;
  int32_t *born_out = p.born_out + row * p.ld;
  if (n <= p.budget) {  // (the CTAs of a row alike)
    for (int j = rank * kThreads + tid; j < n; j += share * kThreads) {
      weight_out[j] = weight[j];
      born_out[j] = born[j];
    }
    return;
  }
  // this CTA's slots
  const int each = (n + 32 * share - 1) / (32 * share) * 32;
  const int s0 = min(rank * each, n), s1 = min(s0 + each, n), words = (s1 - s0 + 31) >> 5;
  const int64_t oldest = static_cast<int64_t>(p.newest[b]) - p.recent;  // recent: born after it
  auto make_key = [&](int b_, float w) -> uint32_t {
    return b_ > oldest ? 0xFFFFFFFFu : w != w ? 0xFFFFFFFEu : ordered_key(w);
  };
  auto key = [&](int j) -> uint32_t { return kCached ? keys_s[j - s0] : make_key(born[j], weight[j]); };
  // Counts digit d, one addition for those of the first lane's: many may be alike, the
  // recent slots are.
  auto count = [&](int *at, uint32_t d) {
    const uint32_t active = __activemask();
    const int lead = __ffs(active) - 1;
    const uint32_t same = __ballot_sync(active, d == __shfl_sync(active, d, lead));
    if (lane == lead)
      atomicAdd(at + d, __popc(same));
    else if (!((same >> lane) & 1u))
      atomicAdd(at + d, 1);
  };
  __syncthreads();
  if (kCached) {
    constexpr int kBatch = 8;  // loads that go out together
    for (int j0 = s0 + tid; j0 < s1; j0 += kBatch * kThreads) {
      int bb[kBatch];
      float ww[kBatch];
#pragma unroll
      for (int e = 0; e < kBatch; ++e) {
        const int j = min(j0 + e * kThreads, s1 - 1);
        bb[e] = born[j];
        ww[e] = weight[j];
      }
#pragma unroll
      for (int e = 0; e < kBatch; ++e) {
        const int j = j0 + e * kThreads;
        if (j < s1) {
          const uint32_t x = make_key(bb[e], ww[e]);
          keys_s[j - s0] = x;
          count(hist[0], x >> 21);
        }
      }
    }
  }
  // ------------------------------------------------------------ selection
  uint32_t prefix = 0, mask = 0;
  int need = keep;  // of the keys that match the digits so far
  int equal = 0;    // keys that are the budget-th largest's
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
    int *now = hist[kCluster ? pass : 0];
    if (!kCached || pass > 0) {
      for (int j = s0 + tid; j < s1; j += kThreads) {
        const uint32_t x = key(j);
        if ((x & mask) == prefix) count(now, (x >> shift) & ((1u << bits) - 1));
      }
    }
    kCluster ? cluster_sync() : __syncthreads();
    // the digit that holds the need-th largest: sums from the top, kPer bins a thread
    constexpr int kPer = kBins / kThreads;
    int own[kPer] = {}, sum = 0;  // (ascending bins)
    const int2 *mine = reinterpret_cast<const int2 *>(now + kBins - (tid + 1) * kPer);
    for (int r = 0; r < share; ++r)
#pragma unroll
      for (int e = 0; e < kPer / 2; ++e) {
        const int2 v = kCluster ? remote_int2(mine + e, r) : mine[e];
        own[2 * e] += v.x;
        own[2 * e + 1] += v.y;
      }
#pragma unroll
    for (int e = 0; e < kPer; ++e) sum += own[e];
    long long total;
    int above = static_cast<int>(block_prefix(sum, scan, total));
#pragma unroll
    for (int e = kPer - 1; e >= 0; --e) {
      if (above < need && above + own[e] >= need) {
        pick = make_int2(kBins - (tid + 1) * kPer + e, above);
        found = own[e];
      }
      above += own[e];
    }
    __syncthreads();
    prefix |= static_cast<uint32_t>(pick.x) << shift;
    mask |= ((1u << bits) - 1) << shift;
    need -= pick.y;
    equal = found;
    if (!kCluster && pass < 2) {
      for (int i = tid; i < kBins / 4; i += kThreads) reinterpret_cast<int4 *>(now)[i] = make_int4(0, 0, 0, 0);
      __syncthreads();
    }
  }
  // The sums of v over the cluster's CTAs before this one, and over all.
  auto over_ranks = [&](int which, int2 v, int2 &all) {
    all = v;
    int2 before = make_int2(0, 0);
    if (kCluster) {
      if (tid == 0) exchange[which] = v;
      cluster_sync();
      all = make_int2(0, 0);
      for (int r = 0; r < share; ++r) {
        const int2 x = remote_int2(exchange + which, r);
        if (r < rank) before = make_int2(before.x + x.x, before.y + x.y);
        all = make_int2(all.x + x.x, all.y + x.y);
      }
    }
    return before;
  };
  // Kept: keys above `prefix`, and the lowest `need` slots of that key.  Each warp
  // takes a stretch of words.
  uint32_t *bits = kCached ? keys_s + each : p.bits + row * p.words + (s0 >> 5);
  const int stretch = (words + kWarps - 1) / kWarps, w0 = min(warp * stretch, words), w1 = min(w0 + stretch, words);
  if (equal == need) {  // (no ties to break)
    for (int w = w0; w < w1; ++w) {
      const int j = s0 + 32 * w + lane;
      const uint32_t kept = __ballot_sync(0xffffffffu, j < s1 && key(j) >= prefix);
      if (lane == 0) bits[w] = kept;
    }
  } else {
    int ties = 0;
    for (int w = w0; w < w1; ++w) {
      const int j = s0 + 32 * w + lane;
      ties += __popc(__ballot_sync(0xffffffffu, j < s1 && key(j) == prefix));
    }
    long long total;
    int seen = static_cast<int>(block_prefix(lane == 0 ? ties : 0, scan, total));
    int2 all;
    seen = __shfl_sync(0xffffffffu, seen, 0) + over_ranks(0, make_int2(static_cast<int>(total), 0), all).x;
    for (int w = w0; w < w1; ++w) {
      const int j = s0 + 32 * w + lane;
      const uint32_t x = j < s1 ? key(j) : 0u;
      const bool tie = j < s1 && x == prefix;
      const uint32_t tied = __ballot_sync(0xffffffffu, tie);
      const uint32_t kept = __ballot_sync(
          0xffffffffu, j < s1 && (x > prefix || (tie && seen + __popc(tied & ((1u << lane) - 1)) < need)));
      seen += __popc(tied);
      if (lane == 0) bits[w] = kept;
    }
  }
  __syncthreads();
  // Freed slots before the new end, and slots that move from behind it, of the words a
  // .. z - 1; numbered in order.
  const int per = (words + kThreads - 1) / kThreads, a = min(tid * per, words), z = min(a + per, words);
  auto freed = [&](int w) {  // (of the slots before the new end)
    const int left = min(keep, s1) - s0 - 32 * w;
    return left <= 0 ? 0u : ~bits[w] & (left >= 32 ? 0xffffffffu : (1u << left) - 1);
  };
  auto moving = [&](int w) {
    const int left = keep - s0 - 32 * w;
    return left >= 32 ? 0u : left <= 0 ? bits[w] : bits[w] & ~((1u << left) - 1);
  };
  long long own = 0;
  for (int w = a; w < z; ++w) own += __popc(freed(w)) | static_cast<long long>(__popc(moving(w))) << 32;
  __syncthreads();
  long long total;
  own = block_prefix(own, scan, total);
  int2 all;
  const int2 before =
      over_ranks(1, make_int2(static_cast<int>(total & 0xffffffff), static_cast<int>(total >> 32)), all);
  int hole = before.x + static_cast<int>(own & 0xffffffff), mover = before.y + static_cast<int>(own >> 32);
  const int moves = all.y;
  // (one CTA's lists lie over its keys, at most half of its slots each)
  int *holes_at = kCached && !kCluster ? reinterpret_cast<int *>(keys_s) : p.lists + 2 * row * p.list;
  int *movers_at = holes_at + (kCached && !kCluster ? each / 2 : p.list);
  for (int w = a; w < z; ++w) {
    for (uint32_t m = freed(w); m; m &= m - 1) holes_at[hole++] = s0 + 32 * w + __ffs(m) - 1;
    for (uint32_t m = moving(w); m; m &= m - 1) movers_at[mover++] = s0 + 32 * w + __ffs(m) - 1;
  }
  // the records of slots that stay in place
  {
    constexpr int kBatch = 4;
    const int end = min(keep, s1);
    for (int a0 = s0 + tid; a0 < end; a0 += kBatch * kThreads) {
      float ww[kBatch];
      int bb[kBatch];
#pragma unroll
      for (int e = 0; e < kBatch; ++e) {
        const int j = min(a0 + e * kThreads, end - 1);
        ww[e] = weight[j];
        bb[e] = born[j];
      }
#pragma unroll
      for (int e = 0; e < kBatch; ++e) {
        const int j = a0 + e * kThreads;
        if (j < end && ((bits[(j - s0) >> 5] >> (j & 31)) & 1u)) {
          weight_out[j] = ww[e];
          born_out[j] = bb[e];
        }
      }
    }
  }
  kCluster ? cluster_sync() : __syncthreads();
  // ---------------------------------------------------------------- moves
  // 16 lanes a row: codes of K and V (D / 2 bytes each) and scales
  const int sub = lane & 15, mine = (moves - rank + share - 1) / share;
  const int chunks = p.D / 32;  // 16-byte chunks of a row's codes
  constexpr int kRows = 2;      // rows a group of lanes has in flight
  const int groups = 2 * kWarps;
  for (int i0 = 2 * warp + (lane >> 4); i0 < mine; i0 += kRows * groups) {
    uint4 x[kRows];
    int to[kRows];
    int64_t dst[kRows];
    int2 mv[kRows];  // freed slot, staying slot
    int64_t src[kRows];
#pragma unroll
    for (int e = 0; e < kRows; ++e) {
      const int i = i0 + e * groups;
      mv[e] = i < mine ? make_int2(holes_at[rank + i * share], movers_at[rank + i * share]) : make_int2(-1, -1);
    }
#pragma unroll
    for (int e = 0; e < kRows; ++e) {
      to[e] = -1;
      if (mv[e].x < 0) continue;
      const int pd = load_page(pv, b, mv[e].x >> pv.logP, p.status, sub == 0);
      const int ps = load_page(pv, b, mv[e].y >> pv.logP, p.status, sub == 0);
      if (pd < 0 || ps < 0) continue;
      to[e] = 1;
      dst[e] = (static_cast<int64_t>(pd) * pv.H_kv + h) * pv.P + (mv[e].x & (pv.P - 1));
      src[e] = (static_cast<int64_t>(ps) * pv.H_kv + h) * pv.P + (mv[e].y & (pv.P - 1));
    }
    // lane sub: chunk sub of K's codes, of V's, then the scales and the records
    const int what = sub < chunks ? 0 : sub < 2 * chunks ? 1 : sub - 2 * chunks + 2;
    const int ch = sub % chunks;
#pragma unroll
    for (int e = 0; e < kRows; ++e) {
      if (mv[e].x < 0) continue;
      if (what < 2) {
        if (to[e] > 0) x[e] = *reinterpret_cast<const uint4 *>((what ? p.c.V : p.c.K) + src[e] * (p.D / 2) + 16 * ch);
      } else if (what < 4) {
        const uint8_t *s = (what == 3 ? p.c.Vs : p.c.Ks) + (to[e] > 0 ? src[e] : 0) * (p.D / 16);
        if (to[e] > 0) {
          x[e].x = *reinterpret_cast<const uint32_t *>(s);
          if (p.D == 128) x[e].y = *reinterpret_cast<const uint32_t *>(s + 4);
        }
      } else if (what == 4) {
        x[e].x = __float_as_uint(weight[mv[e].y]);
        x[e].y = static_cast<uint32_t>(born[mv[e].y]);
      }
    }
#pragma unroll
    for (int e = 0; e < kRows; ++e) {
      if (mv[e].x < 0) continue;
      if (what < 2) {
        if (to[e] > 0) *reinterpret_cast<uint4 *>((what ? p.c.V : p.c.K) + dst[e] * (p.D / 2) + 16 * ch) = x[e];
      } else if (what < 4) {
        uint8_t *s = (what == 3 ? p.c.Vs : p.c.Ks) + (to[e] > 0 ? dst[e] : 0) * (p.D / 16);
        if (to[e] > 0) {
          *reinterpret_cast<uint32_t *>(s) = x[e].x;
          if (p.D == 128) *reinterpret_cast<uint32_t *>(s + 4) = x[e].y;
        }
      } else if (what == 4) {
        weight_out[mv[e].x] = __uint_as_float(x[e].x);
        born_out[mv[e].x] = static_cast<int32_t>(x[e].y);
      }
    }
  }
}

// CTAs of a row: enough that the rows fill the SMs, each with 1024 slots or more, and that
// their shared memory holds the keys, but not more than a cluster has.
int share_of(const sa_paged4_args &pa) {
  const int64_t rows = static_cast<int64_t>(pa.p.B) * pa.p.H_kv, most = static_cast<int64_t>(pa.p.max_pages) * pa.p.P;
  int share = 1;
  while (share < 8 && ((rows * share * 2 <= sm_count() && most > 1024 * share) || most > static_cast<int64_t>(kKeysInSmem) * share))
    share *= 2;
  return share;
}
int list_of(const sa_paged4_args &pa) { return pa.p.max_pages * pa.p.P / 2 + 1; }
int slice_of(const sa_paged4_args &pa) {
  const int unit = 32 * share_of(pa);
  return (pa.p.max_pages * pa.p.P + unit - 1) / unit * 32;
}
int words_of(const sa_paged4_args &pa) { return slice_of(pa) > kKeysInSmem ? share_of(pa) * slice_of(pa) / 32 : 0; }

template <bool kCached, int kThreads, bool kCluster>
cudaError_t launch(const EvictParams &p, int64_t rows, int slice, cudaStream_t stream) {
  auto kern = evict4_kernel<kCached, kThreads, kCluster>;
  static bool done[64] = {};
  const cudaError_t e = set_smem_once(reinterpret_cast<const void *>(kern), (kKeysInSmem + kKeysInSmem / 32) * 4, done);
  if (e != cudaSuccess) return e;
  return launch_ex(false, kern, dim3(static_cast<unsigned>(rows * p.share)), dim3(kThreads),
                   kCached ? (static_cast<size_t>(slice) + slice / 32) * 4 : 0, stream, p.share, p);
}

}  // namespace

size_t evict4_scratch(const sa_paged4_args &pa) {
  const size_t rows = static_cast<size_t>(pa.p.B) * pa.p.H_kv;
  return rows * (share_of(pa) > 1 ? 2 * list_of(pa) * sizeof(int) + words_of(pa) * sizeof(uint32_t) : 0);
}

cudaError_t launch_evict4(const sa_paged4_args &pa, const int32_t *length, const int32_t *newest, int budget, int recent,
                          const float *weight, const int32_t *born, float *weight_out, int32_t *born_out, int64_t ld,
                          int32_t *length_out, void *scratch, uint32_t *status, cudaStream_t stream) {
  const int64_t rows = static_cast<int64_t>(pa.p.B) * pa.p.H_kv;
  EvictParams p;
  p.c = paged4_view(pa);
  p.length = length;
  p.newest = newest;
  p.weight = weight;
  p.born = born;
  p.weight_out = weight_out;
  p.born_out = born_out;
  p.length_out = length_out;
  p.ld = ld;
  p.budget = budget;
  p.recent = recent;
  p.D = pa.p.D;
  p.share = share_of(pa);
  p.list = list_of(pa);
  p.lists = static_cast<int *>(scratch);
  p.words = words_of(pa);
  p.bits = reinterpret_cast<uint32_t *>(p.lists + 2 * rows * p.list);
  p.status = status;
  const int slice = slice_of(pa);
  if (slice > kKeysInSmem) return launch<false, 1024, true>(p, rows, slice, stream);
  if (p.share > 1) return launch<true, 1024, true>(p, rows, slice, stream);
  return rows > sm_count() && slice <= 8192 ? launch<true, 256, false>(p, rows, slice, stream)
                                            : launch<true, 1024, false>(p, rows, slice, stream);
}

}  // namespace sa
