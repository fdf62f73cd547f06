// Frequencies of rotary positions as fractions of a turn. Host code without CUDA, so that it can be tested by itself.
#pragma once

#include <cmath>

namespace lla {
namespace rotary {

// freq radians in units of 2^-64 turns, whole turns dropped: |freq| / (2 pi) as a sum of two doubles (1 / (2 pi) = hi +
// lo), rounded once, so off by 2^-65 turns. |freq| <= 2^20.
inline unsigned long long turns_of(double freq) {
  const double f = std::fabs(freq), hi = 0x1.45f306dc9c883p-3, lo = -0x1.6b01ec5417056p-57;
  const double p = f * hi, e = std::fma(f, hi, -p) + f * lo;
  const double units = std::fmod(p, 1.0) * 0x1p64, whole = std::floor(units);  // exact
  const unsigned long long turns =
      (unsigned long long)whole + (unsigned long long)std::llround(units - whole + e * 0x1p64);
  return freq < 0 ? 0ull - turns : turns;
}

}  // namespace rotary
}  // namespace lla
