// Rotation frequencies as 64-bit fixed-point turns, in a form that host code can compile.
#pragma once

#include <stdint.h>

#include <cmath>

namespace sa {

// f / (2 pi) modulo one turn, times 2^64, to the nearest or next to it (0 <= f < 2^40).  1 / (2 pi)
// is taken as two doubles, 2^-110 off: a quotient by one rounded 2 pi is off by up to 2^-55 of a
// turn, which 2^31 positions carry to 2^-24 of one.
// (Scaled by products and rounded by floor: a call's frequencies are taken on the host, for each
// call anew; with ldexp, remainder and llround an append took 1.5 us more of it.)
inline uint64_t turns_of(double f) {
  constexpr double kHi = 0x1.45f306dc9c883p-3, kLo = -0x1.6b01ec5417056p-57;
  const double p = f * kHi, low = std::fma(f, kLo, std::fma(f, kHi, -p));  // p + low = f / (2 pi)
  const double whole = (p - std::floor(p)) * 0x1p64, units = std::floor(whole);
  // (a fraction below 1 is at most 1 - 2^-53, so units < 2^64)
  const double rest = (whole - units) + (f < 0x1p40 ? low * 0x1p64 : 0.0);
  return static_cast<uint64_t>(units) + static_cast<uint64_t>(static_cast<int64_t>(std::floor(rest + 0.5)));
}

}  // namespace sa
