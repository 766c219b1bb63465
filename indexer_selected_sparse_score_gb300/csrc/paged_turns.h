// Rotation frequencies as 64-bit fixed-point turns, in a form that host code can compile.
#pragma once

#include <stdint.h>

#include <cmath>

namespace sa {

// f / (2 pi) modulo one turn, times 2^64, to the nearest or next to it (|f| < 2^40).  1 / (2 pi)
// is taken as two doubles, 2^-110 off: a quotient by one rounded 2 pi is off by up to 2^-55 of a
// turn, which 2^31 positions carry to 2^-24 of one.
inline uint64_t turns_of(double f) {
  constexpr double kHi = 0x1.45f306dc9c883p-3, kLo = -0x1.6b01ec5417056p-57;
  const double p = f * kHi, low = std::fma(f, kLo, std::fma(f, kHi, -p));  // p + low = f / (2 pi)
  const double whole = std::ldexp(p - std::floor(p), 64), units = std::floor(whole);
  // (a fraction below 1 is at most 1 - 2^-53, so units < 2^64)
  return static_cast<uint64_t>(units) + static_cast<uint64_t>(std::llround((whole - units) + std::ldexp(std::remainder(low, 1.0), 64)));
}

}  // namespace sa
