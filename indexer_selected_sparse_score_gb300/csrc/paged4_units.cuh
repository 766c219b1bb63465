// How the tokens of a call on a 4-bit paged cache form units of work.
//
// Tokens are taken in blocks of `nt` consecutive ones; the tokens of a block that
// follow one another in one sequence are a unit: they attend the same slots, up
// to their own.  A unit costs, for every KV head (or part of its query heads), the tiles of `tile` slots up to
// its last valid token; the tiles of all units, unit by unit, KV head by KV head,
// form one list that the CTAs cut evenly.
#pragma once

#include "paged4.cuh"

namespace sa {

// Highest slot of a unit's tokens that are valid, -1 if none is.
struct UnitSpan {
  int t0, n, b, last;
};

// Calls use(span) for the units of token block i; flags its tokens that have to be
// skipped (status may be NULL).
template <typename Use>
__device__ __forceinline__ void units_of_block(const PagedView &v, int nt, int i, uint32_t *status, const Use &use) {
  const int t1 = min(v.T, (i + 1) * nt);
  UnitSpan u{0, 0, -1, -1};
  for (int t = i * nt; t < t1; ++t) {
    const int b = v.q_seq[t], pos = v.q_pos[t];
    if (u.n == 0 || b != u.b) {
      if (u.n > 0) use(u);
      u = UnitSpan{t, 0, b, -1};
    }
    ++u.n;
    if (b < 0 || b >= v.B)
      raise_flag(status, kFlagBadSeq);
    else if (pos < 0 || (pos >> v.logP) >= v.max_pages)
      raise_flag(status, kFlagBadPos);
    else
      u.last = max(u.last, pos);
  }
  if (u.n > 0) use(u);
}

// Where a CTA's range of tiles begins.
struct UnitStart {
  int block, t0, head, tile;
  long long total;  // tiles of the call
};

// Every thread of the CTA calls it.  CTA c of g takes the tiles total * c / g ..
// total * (c + 1) / g - 1 with g = min(grid, total / least) (at least one); x0 and
// x1 get them, `ctas` g, and out (shared memory) the first one's place.  warp_s:
// 32 long longs of shared memory.
__device__ __forceinline__ void find_units(const PagedView &v, int nt, int heads, int tile, int least, long long *warp_s,
                                           UnitStart *out, uint32_t *status, long long &x0, long long &x1, int &ctas) {
  const int blocks = (v.T + nt - 1) / nt, threads = blockDim.x;
  const int per = (blocks + threads - 1) / threads;
  const int i0 = min(static_cast<int>(threadIdx.x) * per, blocks), i1 = min(i0 + per, blocks);
  long long sum = 0;
  for (int i = i0; i < i1; ++i)
    units_of_block(v, nt, i, blockIdx.x == 0 ? status : nullptr, [&](const UnitSpan &u) { sum += (u.last + tile) / tile; });
  sum *= heads;
  long long total;
  const long long before = block_prefix(sum, warp_s, total);
  const long long most = total / least;
  ctas = static_cast<int>(max(1ll, min(static_cast<long long>(gridDim.x), most)));
  const int c = blockIdx.x;
  x0 = c < ctas ? total * c / ctas : total;
  x1 = c < ctas ? total * (c + 1) / ctas : total;
  if (x0 < x1 && x0 >= before && x0 < before + sum) {
    long long at = before;
    bool found = false;
    for (int i = i0; i < i1 && !found; ++i)
      units_of_block(v, nt, i, nullptr, [&](const UnitSpan &u) {
        const int cost = (u.last + tile) / tile;
        if (!found && x0 < at + static_cast<long long>(cost) * heads) {
          const int rest = static_cast<int>(x0 - at);
          *out = UnitStart{i, u.t0, rest / cost, rest % cost, total};
          found = true;
        }
        at += static_cast<long long>(cost) * heads;
      });
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
  return static_cast<int>(((y + 1) * ctas - 1) / total);
}

}  // namespace sa
