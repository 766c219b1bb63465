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
// distributed shared memory (2 prompts of 4 heads and 16 .. 33 K slots: 20.5 us; 16 CTAs
// that each hold all of a row's keys 40.9; a barrier of a cluster costs 2500 clocks, and one
// fewer by lists that stay apart, with one before the end, is no gain: 22.5).  64 sequences
// of 8 heads and 2112 slots: 20.5 us, a row's chain of loads, three digits, counts and moves.
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

constexpr int kMostShare = 8;

// The values at p's place in the shared memory of the cluster's `share` CTAs, zeros past
// them; the loads go out together.
template <bool kCluster>
__device__ __forceinline__ void load_ranks(const int2 *p, int share, int2 (&v)[kMostShare]) {
  v[0] = kCluster ? make_int2(0, 0) : *p;
#pragma unroll
  for (int r = kCluster ? 0 : 1; r < kMostShare; ++r) {
    v[r] = make_int2(0, 0);
    if (kCluster && r < share) {
      uint32_t a;
      asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(umma::smem_u32(p)), "r"(r));
      asm volatile("ld.shared::cluster.v2.s32 {%0, %1}, [%2];" : "=r"(v[r].x), "=r"(v[r].y) : "r"(a) : "memory");
    }
  }
}

// Sum of x over the lanes up to this one.
__device__ __forceinline__ int scan_warp(int x, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int up = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += up;
  }
  return x;
}

// kThreads: 256 where rows are many, four CTAs to an SM; kCluster: share CTAs a row;
// kCached: a CTA's keys are held in shared memory.
template <bool kCached, int kThreads, bool kCluster>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads)
evict4_kernel(const EvictParams p) {
  constexpr int kWarps = kThreads / 32, kHists = kCluster ? 3 : 1;
  extern __shared__ __align__(16) uint32_t keys_s[];
  __shared__ __align__(16) int hist[kHists][kBins];
  __shared__ __align__(16) int sums[kHists][kBins / 32];
  __shared__ long long scan[32];
  __shared__ int2 ties_s, count_s, ranks_s[2];  // (of a cluster)
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
    __syncthreads();
    // the digit that holds the need-th largest: sums of 32 bins each, then one warp looks
    // for the 32 bins that hold it, and for the bin
    constexpr int kPer = kBins / kThreads;
    int sum = 0;
#pragma unroll
    for (int e = 0; e < kPer / 2; ++e) {
      const int2 v = reinterpret_cast<const int2 *>(now + tid * kPer)[e];
      sum += v.x + v.y;
    }
#pragma unroll
    for (int o = 16 / kPer; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    int *coarse = sums[kCluster ? pass : 0];
    if (tid % (32 / kPer) == 0) coarse[tid * kPer / 32] = sum;
    kCluster ? cluster_sync() : __syncthreads();
    if (warp == 0) {
      // lane l: sums 62 - 2 l, + 1, so that a scan over lanes goes down from the top
      int2 v[kMostShare];
      load_ranks<kCluster>(reinterpret_cast<const int2 *>(coarse) + 31 - lane, share, v);
      int2 x = v[0];
#pragma unroll
      for (int i = 1; i < kMostShare; ++i) x = make_int2(x.x + v[i].x, x.y + v[i].y);
      int upto = scan_warp(x.x + x.y, lane);
      int above = upto - x.x - x.y;  // keys of larger digits
      const uint32_t at = __ballot_sync(0xffffffffu, above < need && upto >= need);
      const int l = __ffs(at) - 1;  // (there is one: need is at least 1 and at most the keys)
      const bool low = above + x.y < need;
      const int group = __shfl_sync(0xffffffffu, 2 * (31 - lane) + (low ? 0 : 1), l);
      above = __shfl_sync(0xffffffffu, low ? above + x.y : above, l);
      // lane l: bin 31 - l of the 32
      load_ranks<kCluster>(reinterpret_cast<const int2 *>(now + 32 * group) + (31 - lane) / 2, share, v);
      int own = 0;
#pragma unroll
      for (int i = 0; i < kMostShare; ++i) own += lane & 1 ? v[i].x : v[i].y;
      upto = above + scan_warp(own, lane);
      if (upto - own < need && upto >= need) {
        pick = make_int2(32 * group + 31 - lane, upto - own);
        found = own;
      }
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
  auto over_ranks = [&](int2 &v_s, int2 v, int2 &all) {
    all = v;
    if (!kCluster) return make_int2(0, 0);
    if (tid == 0) v_s = v;
    cluster_sync();
    if (warp == 0) {
      int2 x[kMostShare], before = make_int2(0, 0), sum = before;
      load_ranks<true>(&v_s, share, x);
#pragma unroll
      for (int r = 0; r < kMostShare; ++r) {
        if (r < rank) before = make_int2(before.x + x[r].x, before.y + x[r].y);
        sum = make_int2(sum.x + x[r].x, sum.y + x[r].y);
      }
      if (lane == 0) {
        ranks_s[0] = before;
        ranks_s[1] = sum;
      }
    }
    __syncthreads();
    all = ranks_s[1];
    return ranks_s[0];
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
    seen = __shfl_sync(0xffffffffu, seen, 0) + over_ranks(ties_s, make_int2(static_cast<int>(total), 0), all).x;
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
      over_ranks(count_s, make_int2(static_cast<int>(total & 0xffffffff), static_cast<int>(total >> 32)), all);
  int hole = before.x + static_cast<int>(own & 0xffffffff), mover = before.y + static_cast<int>(own >> 32);
  const int moves = all.y;  // (as many slots are freed)
  // (one CTA's lists lie over its keys, at most half of its slots each)
  int *holes_at = kCluster ? p.lists + 2 * row * p.list : reinterpret_cast<int *>(keys_s);
  int *movers_at = holes_at + (kCluster ? p.list : each / 2);
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
  // 16 lanes a row, each a piece: 16 bytes of K's or V's codes, the scales of K or V, the
  // weight, the birth; rows whose page is out of range move their record alone
  const int sub = lane & 15, mine = (moves - rank + share - 1) / share;
  const int chunks = p.D / 32, what = sub - 2 * chunks;  // (of a row's codes)
  const uint8_t *from = nullptr;
  uint8_t *to = nullptr;
  int unit = 0, bytes = 0;  // between slots, of the piece
  const bool record = what >= 2 && what < 4;
  if (what < 0) {
    from = to = (sub < chunks ? p.c.K : p.c.V) + 16 * (sub % chunks);
    unit = p.D / 2;
    bytes = 16;
  } else if (what < 2) {
    from = to = what ? p.c.Vs : p.c.Ks;
    unit = bytes = p.D / 16;
  } else if (record) {
    from = what == 2 ? reinterpret_cast<const uint8_t *>(weight) : reinterpret_cast<const uint8_t *>(born);
    to = what == 2 ? reinterpret_cast<uint8_t *>(weight_out) : reinterpret_cast<uint8_t *>(born_out);
    unit = bytes = 4;
  }
  constexpr int kRows = 4;      // rows a group of lanes has in flight
  const int groups = 2 * kWarps;
  for (int i0 = 2 * warp + (lane >> 4); i0 < mine; i0 += kRows * groups) {
    int2 mv[kRows];  // freed slot, staying slot
    int64_t src[kRows], dst[kRows];
    uint4 x[kRows];
#pragma unroll
    for (int e = 0; e < kRows; ++e) {
      const int i = rank + min(i0 + e * groups, mine - 1) * share;
      mv[e] = make_int2(holes_at[i], movers_at[i]);
    }
#pragma unroll
    for (int e = 0; e < kRows; ++e) {
      const int pd = load_page(pv, b, mv[e].x >> pv.logP, p.status, sub == 0);
      const int ps = load_page(pv, b, mv[e].y >> pv.logP, p.status, sub == 0);
      const bool held = pd >= 0 && ps >= 0;
      dst[e] = record ? mv[e].x : held ? (static_cast<int64_t>(pd) * pv.H_kv + h) * pv.P + (mv[e].x & (pv.P - 1)) : -1;
      src[e] = record ? mv[e].y : held ? (static_cast<int64_t>(ps) * pv.H_kv + h) * pv.P + (mv[e].y & (pv.P - 1)) : -1;
      if (bytes == 0 || i0 + e * groups >= mine) dst[e] = -1;
    }
#pragma unroll
    for (int e = 0; e < kRows; ++e) {
      const uint8_t *at = from + src[e] * unit;
      if (dst[e] >= 0) {
        if (bytes == 16) x[e] = *reinterpret_cast<const uint4 *>(at);
        if (bytes == 8) *reinterpret_cast<uint2 *>(&x[e]) = *reinterpret_cast<const uint2 *>(at);
        if (bytes == 4) x[e].x = *reinterpret_cast<const uint32_t *>(at);
      }
    }
#pragma unroll
    for (int e = 0; e < kRows; ++e) {
      uint8_t *at = to + dst[e] * unit;
      if (dst[e] >= 0) {
        if (bytes == 16) *reinterpret_cast<uint4 *>(at) = x[e];
        if (bytes == 8) *reinterpret_cast<uint2 *>(at) = make_uint2(x[e].x, x[e].y);
        if (bytes == 4) *reinterpret_cast<uint32_t *>(at) = x[e].x;
      }
    }
  }
}

// CTAs of a row: enough that the rows fill the SMs, each with 1024 slots or more, and that
// their shared memory holds the keys, but not more than a cluster has.
int share_of(const sa_paged4_args &pa) {
  const int64_t rows = static_cast<int64_t>(pa.p.B) * pa.p.H_kv, most = static_cast<int64_t>(pa.p.max_pages) * pa.p.P;
  int share = 1;
  while (share < kMostShare && ((rows * share * 2 <= sm_count() && most > 1024 * share) || most > static_cast<int64_t>(kKeysInSmem) * share))
    share *= 2;
  return share;
}
int slice_of(const sa_paged4_args &pa) {
  const int unit = 32 * share_of(pa);
  return (pa.p.max_pages * pa.p.P + unit - 1) / unit * 32;
}
int list_of(const sa_paged4_args &pa) { return pa.p.max_pages * pa.p.P / 2 + 1; }
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
  return rows * (share_of(pa) > 1 ? 2 * static_cast<size_t>(list_of(pa)) * sizeof(int) + words_of(pa) * sizeof(uint32_t) : 0);
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
