// Turns per position of a rotated pair as a 64-bit fraction of a turn (host).
#pragma once
#include <cmath>
#include <cstdint>

namespace cpattn {

// radians / (2 pi) modulo 1, times 2^64, for radians in [0, 1e6]: within one
// unit, so that pos times it modulo 2^64 is off by at most |pos| 2^-64 turns,
// 2^-33 at the furthest int32 position. A quotient in double alone is off by
// 2^-54 of radians / (2 pi), which at 1e6 radians per position is 0.018 turn
// there; so 1 / (2 pi) is taken as the sum of two doubles and the product's
// rounding kept.
inline uint64_t turn_fraction(double radians) {
  constexpr double kInv = 0x1.45f306dc9c883p-3, kInvRest = -0x1.6b01ec5417056p-57;
  const double turns = radians * kInv;  // below 2^18
  const double rest = std::fma(radians, kInv, -turns) + radians * kInvRest;
  double whole;
  // modf, not turns - floor(turns), which a compiler may fuse with the product
  const double f = std::modf(turns, &whole) * 4294967296.0;  // exact, as are the next two lines
  const uint64_t hi = uint64_t(f);
  const double g = (f - double(hi)) * 4294967296.0;
  const uint64_t lo = uint64_t(g);
  const double last = (g - double(lo)) + rest * 18446744073709551616.0;  // below 2^29
  return (hi << 32) + lo + uint64_t(int64_t(std::llrint(last)));
}

}  // namespace cpattn
