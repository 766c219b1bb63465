// Sizes and range checks of the page-list kernel that host code can compile.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define SA_BOUNDS_FN __host__ __device__ inline
#else
#define SA_BOUNDS_FN inline
#endif

namespace sa {

// Tile records that the loader of the page-list kernel keeps, for a ring of
// `slots` K and V tiles.  Record n is written once the slot of K(n) is free: with
// an even ring once S(n - slots / 2) is done, for which the weights of three
// tiles before that were written and so, with at most two P^T buffers, the
// product O of five tiles before has been issued: everyone is past record
// n - slots / 2 - 5.  The end record waits for no slot, so it has only what the
// record before it had: one more.  Rounded up to a power of two, for a mask in
// the place of a division (966 tokens over 13 pages each 206 to 205 us).
constexpr int list_records(int slots) {
  int n = 1;
  while (n < slots / 2 + 6) n *= 2;
  return n;
}

// What a merge reads from scratch is taken only where it can be a range of this
// call: after a wait that gave up (the status word says so) it may be anything.
// The parts first .. last of a unit, of `parts` in all.
SA_BOUNDS_FN bool part_range_ok(int first, int last, int parts) { return first >= 0 && first <= last && last < parts; }
// A unit of `units` that CTA c cut, its last part in CTA `last` of `ctas`.
SA_BOUNDS_FN bool cut_ok(int64_t unit, int last, int64_t units, int c, int ctas) {
  return unit >= 0 && unit < units && part_range_ok(c, last, ctas);
}


// The KV head and the tile of it that the rest-th tile of a unit is, of `cost` tiles a head
// (a unit of 2^30 slots and hundreds of heads has more than 2^31 tiles).
struct TilePlace {
  int head, tile;
};
SA_BOUNDS_FN TilePlace tile_place(int64_t rest, int cost) {
  if ((rest >> 32) == 0) {
    const uint32_t r = static_cast<uint32_t>(rest), c = static_cast<uint32_t>(cost);
    return TilePlace{static_cast<int>(r / c), static_cast<int>(r % c)};
  }
  return TilePlace{static_cast<int>(rest / cost), static_cast<int>(rest % cost)};
}

}  // namespace sa
