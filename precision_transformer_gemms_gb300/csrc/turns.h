// Angles in turns, of which only the fraction matters: position * (frequency / 2 pi)
// modulo 1 in integers.  Shared by the kernel, its launch and a test on the host.
#pragma once
#include <math.h>
#include <stdint.h>

#ifndef LPQ_HOST_DEVICE
#ifdef __CUDACC__
#define LPQ_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define LPQ_HOST_DEVICE inline
#endif
#endif

namespace lpq {

// frequency / 2 pi modulo 1, in units of 2^-96 turns: high * 2^32 + low.  A double's 53
// bits fit for frequencies down to 2^-40; the bits that smaller ones lose are less than
// 2^-33 turns at any position.
struct Turns {
  uint64_t high;
  uint32_t low;
};

// The fraction is taken of the magnitude, where it is exact, and turned round as an
// integer: that of a negative double would be rounded to 2^-53 turns.
inline Turns turns_of(double frequency) {
  double turn = fabs(frequency) * 0.15915494309189535;  // 1 / (2 pi)
  turn = (turn - floor(turn)) * 18446744073709551616.0;
  const uint64_t high = (uint64_t)turn;
  const uint32_t low = (uint32_t)((turn - (double)high) * 4294967296.0);
  if (!(frequency < 0)) return {high, low};
  return {~high + (low == 0), ~low + 1u};
}

// The angle at a position in units of 2^-64 turns is high * position and what the low
// word adds, which is below 2^-33 turns at positions of 32 bits and left out there.
LPQ_HOST_DEVICE bool is_far(int64_t position) { return position != (int64_t)(int32_t)position; }

// A product with the position as an unsigned number has 2^64 times the frequency too much
// where the position is negative: whole turns of the high word, the low one is taken off.
LPQ_HOST_DEVICE uint64_t low_part(uint32_t low, int64_t position) {
  const uint64_t p = (uint64_t)position, part = (p >> 32) * low + (((p & 0xFFFFFFFFu) * low) >> 32);
  return position < 0 ? part - ((uint64_t)low << 32) : part;
}

}  // namespace lpq
