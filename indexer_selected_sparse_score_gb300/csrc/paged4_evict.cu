// Slots freed by the attention weight they have gathered: selection per (sequence,
// KV head) row, and the rows that move into the freed slots.
//
// Selection: a slot's key is its weight's bits in order (recent slots count above
// all); the budget-th largest key is found by a radix select, digits of 11, 11
// and 10 bits, a histogram in shared memory each.  Of the slots of exactly that
// key the lowest stay.
//
// Moves: freed slots before the new end are filled from behind it, so a row moves
// at most once and no more rows move than slots are freed (keeping the rows in
// order would move nearly all of them: 150 MB instead of 5 for 64 sequences of 8
// heads and 2112 slots cut to 2048).  Sources lie at or past the new end and
// destinations before it, so the moves of a call need no order.
//
// A row is selected by `share` CTAs alike (each reads all of its records) and each
// moves its share of the rows: with few sequences the moves would otherwise be
// bound by one SM's loads in flight.  Records are read from L2 twice or more;
// keys of up to kKeysInSmem slots stay in shared memory.
#include <algorithm>

#include "internal.h"
#include "paged4.cuh"

namespace sa {
namespace {

constexpr int kBins = 2048;
constexpr int kKeysInSmem = 49152;

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
  int list;       // entries of a CTA's lists
  int2 *lists;    // [CTA][list]: (freed slot, staying slot)
  uint32_t *status;
};

// Every thread of the CTA calls it: the sum of v over the warps before this one
// (v alike in a warp), and over all.
template <int kWarps>
__device__ __forceinline__ int warp_prefix(int v, int *s, int &total) {
  const int warp = threadIdx.x >> 5;
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s[warp] = v;
  __syncthreads();
  int before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += s[w];
    total += s[w];
  }
  return before;
}

// kThreads: 256 for short rows, four CTAs to an SM; 1024 for long ones.
template <bool kCached, int kThreads>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads)
evict4_kernel(const EvictParams p) {
  constexpr int kWarps = kThreads / 32;
  extern __shared__ uint32_t keys_s[];
  __shared__ int hist[kBins];
  __shared__ int scan[kWarps];
  __shared__ int2 pick;  // digit, keys above it
  __shared__ int found;  // keys of it
  const PagedView &pv = p.c.v;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int part = blockIdx.x % p.share;
  const int64_t row = blockIdx.x / p.share;
  const int b = static_cast<int>(row / pv.H_kv), h = static_cast<int>(row - static_cast<int64_t>(b) * pv.H_kv);
  int n = p.length[b];
  if (n < 0 || n > pv.max_pages * pv.P) {
    if (tid == 0) raise_flag(p.status, kFlagBadPos);
    n = 0;
  }
  const int keep = min(n, p.budget);
  if (h == 0 && part == 0 && tid == 0) p.length_out[b] = keep;
  const float *weight = p.weight + row * p.ld;
  const int32_t *born = p.born + row * p.ld;
  float *weight_out = p.weight_out + row * p.ld;
  int32_t *born_out = p.born_out + row * p.ld;
  if (n <= p.budget) {
    for (int j = part * kThreads + tid; j < n; j += p.share * kThreads) {
      weight_out[j] = weight[j];
      born_out[j] = born[j];
    }
    return;
  }
  const int64_t oldest = static_cast<int64_t>(p.newest[b]) - p.recent;  // recent: born after it
  auto make_key = [&](int b_, float w) -> uint32_t {
    return b_ > oldest ? 0xFFFFFFFFu : w != w ? 0xFFFFFFFEu : ordered_key(w);
  };
  auto key = [&](int j) -> uint32_t { return kCached ? keys_s[j] : make_key(born[j], weight[j]); };
  if (kCached) {
    constexpr int kBatch = 8;  // loads that go out together
    for (int j0 = tid; j0 < n; j0 += kBatch * kThreads) {
      int bb[kBatch];
      float ww[kBatch];
#pragma unroll
      for (int e = 0; e < kBatch; ++e) {
        const int j = min(j0 + e * kThreads, n - 1);
        bb[e] = born[j];
        ww[e] = weight[j];
      }
#pragma unroll
      for (int e = 0; e < kBatch; ++e)
        if (j0 + e * kThreads < n) keys_s[j0 + e * kThreads] = make_key(bb[e], ww[e]);
    }
  }
  // ------------------------------------------------------------ selection
  uint32_t prefix = 0, mask = 0;
  int need = keep;  // of the keys that match the digits so far
  int equal = 0;    // keys that are the budget-th largest's
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
    for (int i = tid; i < kBins; i += kThreads) hist[i] = 0;
    __syncthreads();
    for (int j = tid; j < n; j += kThreads) {
      const uint32_t x = key(j);
      if ((x & mask) == prefix) {
        const uint32_t d = (x >> shift) & ((1u << bits) - 1);
        // (many may be alike, the recent slots are: one addition for those of the first
        // lane's digit)
        const uint32_t active = __activemask();
        const int lead = __ffs(active) - 1;
        const uint32_t same = __ballot_sync(active, d == __shfl_sync(active, d, lead));
        if (lane == lead)
          atomicAdd(&hist[d], __popc(same));
        else if (!((same >> lane) & 1u))
          atomicAdd(&hist[d], 1);
      }
    }
    __syncthreads();
    // the digit that holds the need-th largest: sums from the top, four bins a thread
    constexpr int kPer = kBins / kThreads;
    int own[kPer], sum = 0;
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      own[e] = hist[kBins - 1 - (tid * kPer + e)];
      sum += own[e];
    }
    int up = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, up, o);
      if (lane >= o) up += v;
    }
    int total;
    int above = warp_prefix<kWarps>(__shfl_sync(0xffffffffu, up, 31), scan, total) + up - sum;
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      if (above < need && above + own[e] >= need) {
        pick = make_int2(kBins - 1 - (tid * kPer + e), above);
        found = own[e];
      }
      above += own[e];
    }
    __syncthreads();
    prefix |= static_cast<uint32_t>(pick.x) << shift;
    mask |= ((1u << bits) - 1) << shift;
    need -= pick.y;
    equal = found;
  }
  // Kept: keys above `prefix`, and the lowest `need` slots of that key.  Each warp
  // takes a stretch of slots.
  const int each = ((n + kWarps - 1) / kWarps + 31) & ~31;
  const int j0 = min(warp * each, n), j1 = min(j0 + each, n);
  const bool all_equal = equal == need;  // (no ties to break)
  int ties_before = 0, total;
  if (!all_equal) {
    int ties = 0;
    for (int j = j0 + lane; j - lane < j1; j += 32)
      ties += __popc(__ballot_sync(0xffffffffu, j < j1 && key(j) == prefix));
    ties_before = warp_prefix<kWarps>(ties, scan, total);
  }
  // walk(use): use(j, kept, in) for 32 slots at a time
  auto walk = [&](const auto &use) {
    int seen = ties_before;
    for (int jb = j0; jb < j1; jb += 32) {
      const int j = jb + lane;
      const uint32_t x = j < j1 ? key(j) : 0u;
      bool kept = j < j1 && (all_equal ? x >= prefix : x > prefix);
      if (!all_equal) {
        const bool tie = j < j1 && x == prefix;
        const uint32_t tied = __ballot_sync(0xffffffffu, tie);
        kept |= tie && seen + __popc(tied & ((1u << lane) - 1)) < need;
        seen += __popc(tied);
      }
      use(j, kept, j < j1);
    }
  };
  int holes = 0, movers = 0;
  walk([&](int j, bool kept, bool in) {
    holes += in && !kept && j < keep;
    movers += kept && j >= keep;
    if (kCached && in) keys_s[j] = kept;  // from here on (a slot is read by its lane alone)
  });
  holes = __reduce_add_sync(0xffffffffu, holes);
  movers = __reduce_add_sync(0xffffffffu, movers);
  int moves;
  int hole = warp_prefix<kWarps>(holes, scan, moves), mover = warp_prefix<kWarps>(movers, scan, total);
  int2 *list = p.lists + static_cast<int64_t>(blockIdx.x) * p.list;
  auto note = [&](int j, bool kept, bool in) {
    const bool is_hole = in && !kept && j < keep, is_mover = kept && j >= keep;
    const uint32_t bh = __ballot_sync(0xffffffffu, is_hole), bm = __ballot_sync(0xffffffffu, is_mover);
    const uint32_t below = (1u << lane) - 1;
    if (is_hole) {
      const int i = hole + __popc(bh & below);
      if (i % p.share == part) list[i / p.share].x = j;
    }
    if (is_mover) {
      const int i = mover + __popc(bm & below);
      if (i % p.share == part) list[i / p.share].y = j;
    }
    hole += __popc(bh);
    mover += __popc(bm);
  };
  if (kCached) {
    for (int jb = j0; jb < j1; jb += 32) {
      const int j = jb + lane;
      note(j, j < j1 && keys_s[j], j < j1);
    }
    __syncthreads();
    // the records of slots that stay in place: this CTA's share
    constexpr int kBatch = 4;
    const int stride = p.share * kThreads;
    for (int a0 = part * kThreads + tid; a0 < keep; a0 += kBatch * stride) {
      float ww[kBatch];
      int bb[kBatch];
#pragma unroll
      for (int e = 0; e < kBatch; ++e) {
        const int j = min(a0 + e * stride, keep - 1);
        ww[e] = weight[j];
        bb[e] = born[j];
      }
#pragma unroll
      for (int e = 0; e < kBatch; ++e) {
        const int j = a0 + e * stride;
        if (j < keep && keys_s[j]) {
          weight_out[j] = ww[e];
          born_out[j] = bb[e];
        }
      }
    }
  } else {
    walk([&](int j, bool kept, bool in) {
      note(j, kept, in);
      if (kept && j < keep && (j >> 5) % p.share == part) {
        weight_out[j] = weight[j];
        born_out[j] = born[j];
      }
    });
  }
  __syncthreads();
  // ---------------------------------------------------------------- moves
  // 16 lanes a row: codes of K and V (D / 2 bytes each) and scales
  const int sub = lane & 15, mine = (moves - part + p.share - 1) / p.share;
  const int chunks = p.D / 32;  // 16-byte chunks of a row's codes
  constexpr int kRows = 2;      // rows a group of lanes has in flight
  const int groups = 2 * kWarps;
  for (int i0 = 2 * warp + (lane >> 4); i0 < mine; i0 += kRows * groups) {
    uint4 x[kRows];
    int to[kRows];
    int64_t dst[kRows];
    int2 mv[kRows];
    int64_t src[kRows];
#pragma unroll
    for (int e = 0; e < kRows; ++e) {
      const int i = i0 + e * groups;
      mv[e] = i < mine ? list[i] : make_int2(-1, -1);
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

// CTAs that share a row: enough that the rows fill the SMs.
int share_of(const sa_paged4_args &pa) {
  const int64_t rows = static_cast<int64_t>(pa.p.B) * pa.p.H_kv;
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(16, sm_count() / rows)));
}
template <int kThreads>
cudaError_t launch_cached(const EvictParams &p, dim3 grid, int most, cudaStream_t stream) {
  auto kern = evict4_kernel<true, kThreads>;
  static bool done[64] = {};
  const cudaError_t e = set_smem_once(reinterpret_cast<const void *>(kern), kKeysInSmem * 4, done);
  if (e != cudaSuccess) return e;
  return launch_ex(false, kern, grid, dim3(kThreads), static_cast<size_t>(most) * 4, stream, 1, p);
}
int list_of(const sa_paged4_args &pa) { return (pa.p.max_pages * pa.p.P / 2) / share_of(pa) + 1; }

}  // namespace

size_t evict4_scratch(const sa_paged4_args &pa) {
  return static_cast<size_t>(pa.p.B) * pa.p.H_kv * share_of(pa) * list_of(pa) * sizeof(int2);
}

cudaError_t launch_evict4(const sa_paged4_args &pa, const int32_t *length, const int32_t *newest, int budget, int recent,
                          const float *weight, const int32_t *born, float *weight_out, int32_t *born_out, int64_t ld,
                          int32_t *length_out, void *scratch, uint32_t *status, cudaStream_t stream) {
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
  p.lists = static_cast<int2 *>(scratch);
  p.status = status;
  const int most = pa.p.max_pages * pa.p.P;
  const dim3 grid(static_cast<unsigned>(static_cast<int64_t>(pa.p.B) * pa.p.H_kv * p.share));
  if (most > kKeysInSmem) return launch_ex(false, evict4_kernel<false, 1024>, grid, dim3(1024), 0, stream, 1, p);
  return most > 8192 ? launch_cached<1024>(p, grid, most, stream) : launch_cached<256>(p, grid, most, stream);
}

}  // namespace sa
