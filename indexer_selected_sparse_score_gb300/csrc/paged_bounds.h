// Sizes and range checks of the page-list kernel that host code can compile.
#pragma once

namespace sa {

// Tile records that the loader of the page-list kernel keeps, for a ring of
// `slots` K and V tiles.  Record n is written once the slot of K(n) is free: with
// an even ring once S(n - slots / 2) is done, for which the weights of three
// tiles before that were written and so, with at most two P^T buffers, the
// product O of five tiles before has been issued: everyone is past record
// n - slots / 2 - 5.  The end record waits for no slot, so it has only what the
// record before it had: one more.
constexpr int list_records(int slots) { return slots / 2 + 6; }

}  // namespace sa
