// Fractions of a turn in whole numbers: what a frequency (radians per position) adds
// to the angle with each position, modulo one turn.  Plain C++, so that it can be
// tested on the host.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define DUSTIN_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define DUSTIN_HOST_DEVICE inline
#endif

namespace dustin {

// freq / (2 pi) modulo 1, in units of 2^-64, of the fp32 with these bits.  With
// freq = m 2^e, m below 2^24: the upper bits of m round(2^104 / (2 pi)), which
// fits 126 bits, shifted by e.  The constant is off by 2^-105 of a turn, so the
// result by 2^-65 (its own rounding) and |freq| 2^-105: a position of 31 bits keeps
// every angle to 2^-33 of a turn where |freq| < 2^39.  (Larger ones, infinities and
// NaN give some fraction.)  With the product in fp64 each position was off by
// |freq| 2^-56, and 5003 tokens of 14/2/64 took 8.2 instead of 7.3 us.
DUSTIN_HOST_DEVICE uint64_t turn_of(uint32_t bits) {
  const unsigned __int128 inv2pi = (unsigned __int128)0x28BE60DB93ull << 64 | 0x91054A7F09D5F47Dull;
  const int x = int(bits >> 23 & 255u);
  const uint32_t m = (bits & 0x7FFFFFu) | (x ? 0x800000u : 0u);
  int s = 190 - (x ? x : 1);   // the product's bits below 2^-64 of a turn
  if (s < 1) s = 1;
  const uint64_t u = s > 127 ? 0 : uint64_t(((inv2pi * m >> (s - 1)) + 1) >> 1);
  return bits >> 31 ? 0 - u : u;
}

}  // namespace dustin
