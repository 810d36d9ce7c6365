// Frequencies of the rotary positions as 64-bit fractions (host, integers but for a first guess of each square root).
#pragma once

#include <math.h>
#include <stdint.h>

namespace dex {

// 1 / 2 pi in units of 2^-64: the turn of pair 0 at position 1.
constexpr uint64_t kTurnPerRadian = 0x28be60db9391054aull;

// power[b] = theta^(-2 2^b / head_dim) in units of 2^-64 (2^64 - 1 for one), for the bits b of a pair's index, each to
// eight units.  power[n - 1] is theta^(-1/2) and each one before it the square root of the next, and a square root
// halves the relative error of what it is taken of, where squaring the first one doubles it: in 53 bits that is off by
// up to 2^-20 of a turn at position 2^31 (theta 1.1, whose frequencies hardly fall).
inline void rope_powers(float theta, int head_dim, uint64_t (&power)[6]) {
  using u128 = unsigned __int128;
  int n = 0;
  while ((4 << n) <= head_dim) ++n;   // bits of an index below head_dim / 2
  // v = q 2^-(63 + k) with q in [2^63, 2^64): 1 / theta, from theta's 24 bits
  int k;
  const uint64_t m = static_cast<uint64_t>(frexp(static_cast<double>(theta), &k) * 16777216.0);
  const u128 inv = (static_cast<u128>(1) << 87) / m;
  uint64_t q = static_cast<uint64_t>(inv);
  if (inv >> 64) q = uint64_t(1) << 63, --k;   // a power of two
  for (int b = n - 1; b >= 0; --b) {
    const int s = (63 + k) % 2 ? 63 : 64;   // an even exponent
    const u128 x = static_cast<u128>(q) << s;
    const double guess = sqrt(static_cast<double>(x));   // 53 bits; one Newton step gives 64
    const uint64_t r = guess < 18446744073709551615.0 ? static_cast<uint64_t>(guess) : ~uint64_t(0);
    const u128 next = (static_cast<u128>(r) + x / r) >> 1;
    q = next >> 64 ? ~uint64_t(0) : static_cast<uint64_t>(next);
    k = (63 + k + s) / 2 - 63;
    power[b] = k > 64 ? 0 : k > 0 ? q >> (k - 1) : ~uint64_t(0);
  }
  for (int b = n; b < 6; ++b) power[b] = 0;   // no index has this bit
}

}  // namespace dex
