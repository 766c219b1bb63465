// How the tokens of a call on a 4-bit paged cache form units of work.
//
// Tokens are taken in blocks of `nt` consecutive ones; the tokens of a block that
// follow one another in one sequence are a unit: they attend the same slots, up
// to their own.  A unit costs, for every KV head, the tiles of `tile` slots up to its
// last valid token; the tiles of all units, unit by unit, KV head by KV head,
// form one list that the CTAs cut evenly.
#pragma once

#include "paged4.cuh"
#include "paged_bounds.h"

namespace sa {

// a / b of non-negative values, mostly below 2^32.
__device__ __forceinline__ long long divide(long long a, long long b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

// One thread, after a barrier of the threads that have written: counts a part as added.
// What they wrote before is seen by whoever's call returns a larger number (and by
// those that it meets at a barrier afterwards).
__device__ __forceinline__ uint32_t count_part(uint32_t *counter) {
  uint32_t before;
  asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(before) : "l"(counter) : "memory");
  return before;
}

// Where a CTA's range of tiles begins.
struct UnitStart {
  int block, t0, head, tile;
  long long total;  // tiles of the call
  int round;        // units count as multiples of it
  int tiles;        // above 1: the tiles that there are of the CTA's
};

// One warp: calls use(first token, last slot) for the units that begin among tokens
// t0 .. t1 - 1 (t0 begins one), in order, until it returns false; the slot is -1 for
// a unit without a valid token.  Tokens that have to be skipped are flagged (status
// may be NULL).
template <typename Use>
__device__ __forceinline__ void units_of_tokens(const PagedView &v, int nt, int t0, int t1, uint32_t *status,
                                                const Use &use) {
  const int lane = threadIdx.x & 31;
  int open = -1, last = -1, prev = 0;  // the unit under way, its last slot; the token before
  for (int base = t0; base < v.T && (base < t1 || open >= 0); base += 32) {
    const int t = base + lane;
    const bool in = t < v.T;
    const int b = in ? v.q_seq[t] : 0, pos = in ? v.q_pos[t] : -1;
    int slot = -1;
    if (in) {
      const bool bad_seq = b < 0 || b >= v.B, bad_pos = pos < 0 || (pos >> v.logP) >= v.max_pages;
      if (!bad_seq && !bad_pos)
        slot = pos;
      else if (t < t1)
        raise_flag(status, bad_seq ? kFlagBadSeq : kFlagBadPos);
    }
    int before = __shfl_up_sync(0xffffffffu, b, 1);
    if (lane == 0) before = prev;
    prev = __shfl_sync(0xffffffffu, b, 31);
    uint32_t starts = __ballot_sync(0xffffffffu, in && (t == t0 || t % nt == 0 || b != before));
    // tokens before the first start belong to the unit under way
    for (int l = 0; l < 32;) {
      const bool begins = (starts >> l) & 1u;
      if (begins) {
        if (open >= 0 && !use(open, last)) return;
        open = -1;
        if (base + l >= t1) return;
        open = base + l;
        last = -1;
        starts &= ~(1u << l);
      }
      const int end = starts ? __ffs(starts) - 1 : 32;  // (a start at l itself has been taken)
      last = max(last, __reduce_max_sync(0xffffffffu, lane >= l && lane < end ? slot : -1));
      l = end;
    }
  }
  if (open >= 0) use(open, last);
}

// Every thread of the CTA calls it.  CTA c of g takes the tiles total * c / g ..
// total * (c + 1) / g - 1 with g = min(grid, total / least) (at least one); x0 and
// x1 get them, `ctas` g, and out (shared memory) the first one's place.  warp_s:
// 32 long longs of shared memory.
//
// kWhole (unit_s: 128 ints of shared memory): where there are no more units (for all
// heads) than CTAs, at most 64, among no more tokens than threads, no CTA has to have
// parts of two: every unit is cut into pieces of one length (out->round; units then count
// as multiples of it), if one that is at most 7 tiles above the even share gives no more
// pieces than CTAs.  (A second part costs a CTA about 4 us, a tile of 128 rows of 144
// bytes 0.8 us when all stream: 16 tokens of 32 over 8 heads of 64 at 0.1 .. 3 K slots
// 14.4 us, by even shares 19.9.)  Of up to 64 units each warp finds its CTA's place by itself.
template <bool kWhole = false>
__device__ __forceinline__ void find_units(const PagedView &v, int nt, int heads, int tile, int least, long long *warp_s,
                                           UnitStart *out, uint32_t *status, long long &x0, long long &x1, int &ctas,
                                           int *unit_s = nullptr) {
  // warp w takes the units that begin in its stretch of blocks (of whole 32s of tokens,
  // where a block is one)
  const int warps = (blockDim.x + 31) >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int grain = nt == 1 ? 32 : nt;
  const int grains = (v.T + grain - 1) / grain, per = (grains + warps - 1) / warps;
  const int t0 = static_cast<int>(min(static_cast<int64_t>(v.T), static_cast<int64_t>(warp) * per * grain));
  const int t1 = static_cast<int>(min(static_cast<int64_t>(v.T), (static_cast<int64_t>(warp) + 1) * per * grain));
  uint32_t *report = blockIdx.x == 0 ? status : nullptr;
  int units = 65;
  int cost[2] = {0, 0}, first[2] = {0, 0};  // of units lane and 32 + lane: tiles, first token
  if (kWhole && nt == 1 && v.T <= 64) {
    uint32_t *own = warp == 0 ? report : nullptr;
    units = v.T;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int t = 32 * e + lane;
      int b, pos;
      first[e] = t;
      if (t < v.T && load_paged_token(v, t, own, own != nullptr, b, pos)) cost[e] = (pos + tile) / tile;
    }
  } else if (kWhole && v.T <= static_cast<int>(blockDim.x)) {
    // a thread per token; unit_s: first tokens, last slots
    const int t = threadIdx.x;
    int b = -1, pos = -1;
    const bool in = t < v.T, valid = in && load_paged_token(v, t, report, report != nullptr, b, pos);
    const bool begins = in && (t % nt == 0 || b != v.q_seq[t - 1]);
    if (t < 64) unit_s[64 + t] = -1;
    long long all;
    const int u = static_cast<int>(block_prefix(begins ? 1 : 0, warp_s, all)) - (begins ? 0 : 1);
    if (all <= 64) {
      if (begins) unit_s[u] = t;
      if (valid) atomicMax(&unit_s[64 + u], pos);
    }
    __syncthreads();
    if (all <= 64) {
      units = static_cast<int>(all);
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (32 * e + lane < units) {
          first[e] = unit_s[32 * e + lane];
          cost[e] = (unit_s[64 + 32 * e + lane] + tile) / tile;
        }
    }
  }
  if (units <= 64) {
    const int all = __reduce_add_sync(0xffffffffu, cost[0] + cost[1]);
    long long total = static_cast<long long>(all) * heads;
    const int most = static_cast<int>(min(static_cast<long long>(gridDim.x), max(1ll, total / least)));
    const int shortest = max(least, static_cast<int>(divide(total + gridDim.x - 1, gridDim.x)));
    // the shortest of 8 lengths that is long enough (a longer one gives no more pieces)
    auto pieces = [&](int n) {
      return __reduce_add_sync(0xffffffffu, (cost[0] + n - 1) / n + (cost[1] + n - 1) / n) * heads;
    };
    int round = 1;
    ctas = most;
    if (all > 0 && static_cast<int64_t>(units) * heads <= gridDim.x && pieces(shortest + 7) <= static_cast<int>(gridDim.x)) {
      round = shortest;
#pragma unroll
      for (int step = 4; step > 0; step >>= 1)
        if (pieces(round + step - 1) > static_cast<int>(gridDim.x)) round += step;
      ctas = pieces(round);
      total = static_cast<long long>(ctas) * round;
    }
    const int c = blockIdx.x;
    x0 = c < ctas ? divide(total * c, ctas) : total;
    x1 = c < ctas ? divide(total * (c + 1), ctas) : total;
    long long before = 0;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int counted = (cost[e] + round - 1) / round * round;
      long long upto = static_cast<long long>(counted) * heads;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += u;
      }
      upto += before;
      const long long from = upto - static_cast<long long>(counted) * heads;
      if (warp == 0 && x0 < x1 && x0 >= from && x0 < upto) {
        const TilePlace at = tile_place(x0 - from, counted);
        const int t = first[e];
        *out = UnitStart{t / nt, t, at.head, at.tile, total, round, min(round, cost[e] - at.tile)};
      }
      before = __shfl_sync(0xffffffffu, upto, 31);
    }
    return;
  }
  long long sum = 0;
  if (nt == 1) {
    for (int t = t0 + lane; t < t1; t += 32) {
      int b, pos;
      if (load_paged_token(v, t, report, report != nullptr, b, pos)) sum += (pos + tile) / tile;
    }
  } else if (t0 < t1) {
    units_of_tokens(v, nt, t0, t1, report, [&](int, int last) {
      if (lane == 0) sum += (last + tile) / tile;
      return true;
    });
  }
  sum *= heads;
  long long total;
  long long before = block_prefix(sum, warp_s, total);
  const long long most = total / least;
  ctas = static_cast<int>(max(1ll, min(static_cast<long long>(gridDim.x), most)));
  const int c = blockIdx.x;
  x0 = c < ctas ? divide(total * c, ctas) : total;
  x1 = c < ctas ? divide(total * (c + 1), ctas) : total;
  // (the warp's first tile and its number of tiles)
  before = __shfl_sync(0xffffffffu, before, 0);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (x0 < x1 && x0 >= before && x0 < before + sum) {
    long long at = before;
    auto take = [&](int t, int last) {
      const int cost = (last + tile) / tile;
      if (x0 < at + static_cast<long long>(cost) * heads) {
        const TilePlace place = tile_place(x0 - at, cost);
        if (lane == 0) *out = UnitStart{t / nt, t, place.head, place.tile, total, 1, 0};
        return false;
      }
      at += static_cast<long long>(cost) * heads;
      return true;
    };
    if (nt == 1) {
      // 32 tokens at a time: skip those whose tiles end before x0
      for (int base = t0; base < t1; base += 32) {
        const int t = base + lane;
        int b, pos, last = -1;
        if (t < t1 && load_paged_token(v, t, nullptr, false, b, pos)) last = pos;
        long long cost = static_cast<long long>((last + tile) / tile) * heads;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) cost += __shfl_xor_sync(0xffffffffu, cost, o);
        if (x0 >= at + cost) {
          at += cost;
          continue;
        }
        for (int l = 0; l < 32; ++l)
          if (!take(base + l, __shfl_sync(0xffffffffu, last, l))) return;
      }
    } else {
      units_of_tokens(v, nt, t0, t1, nullptr, take);
    }
  }
}

// ------------------------------------------------------------------- runs --
// The tokens of a call that follow one another in one sequence, however many.

struct Runs {
  int *t0;         // [runs + 1] first token; t0[runs] = T
  int *last;       // [runs] highest slot of the valid tokens, -1 if there is none
  long long *off;  // [runs + 1] tiles before the run, all KV heads
};

// Shared memory of plan_runs for `threads` threads: 32 long longs.
// Every thread of one CTA calls it; r has room for T runs.  Returns the number of
// runs.  Tokens that have to be skipped are flagged (status may be NULL).
__device__ __forceinline__ int plan_runs(const PagedView &v, int tile, long long *warp_s, const Runs &r,
                                         uint32_t *status) {
  const int threads = blockDim.x;
  int runs = 0;
  for (int base = 0; base < v.T; base += threads) {
    const int t = base + threadIdx.x;
    const bool first = t < v.T && (t == 0 || v.q_seq[t] != v.q_seq[t - 1]);
    long long total;
    const long long before = block_prefix(first ? 1 : 0, warp_s, total);
    __syncthreads();
    if (first) {
      r.t0[runs + before] = t;
      r.last[runs + before] = -1;
    }
    runs += static_cast<int>(total);
  }
  if (threadIdx.x == 0) r.t0[runs] = v.T;
  __syncthreads();
  // (a second pass over the tokens: their run is the number of starts up to them)
  int done = 0;
  for (int base = 0; base < v.T; base += threads) {
    const int t = base + threadIdx.x;
    const bool first = t < v.T && (t == 0 || v.q_seq[t] != v.q_seq[t - 1]);
    long long total;
    const long long before = block_prefix(first ? 1 : 0, warp_s, total);
    __syncthreads();
    if (t < v.T) {
      int b, pos;
      if (load_paged_token(v, t, status, status != nullptr, b, pos))
        atomicMax(&r.last[done + before - (first ? 0 : 1)], pos);
    }
    done += static_cast<int>(total);
  }
  __syncthreads();
  long long at = 0;
  for (int base = 0; base < runs; base += threads) {
    const int i = base + threadIdx.x;
    const long long cost = i < runs ? static_cast<long long>((r.last[i] + tile) / tile) * v.H_kv : 0;
    long long total;
    const long long before = block_prefix(cost, warp_s, total);
    __syncthreads();
    if (i < runs) r.off[i] = at + before;
    at += total;
  }
  if (threadIdx.x == 0) r.off[runs] = at;
  __syncthreads();
  return runs;
}

// The run that holds tile x (off[run] <= x < off[run + 1]).
__device__ __forceinline__ int run_of_tile(const long long *off, int runs, long long x) {
  int lo = 0, hi = runs;  // off[lo] <= x < off[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (off[mid] <= x)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// The CTA of `ctas` whose range holds tile y of `total`.
__device__ __forceinline__ int cta_of_tile(long long y, long long total, int ctas) {
  return static_cast<int>(divide((y + 1) * ctas - 1, total));
}

}  // namespace sa
