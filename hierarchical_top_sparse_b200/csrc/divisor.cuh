// divisor.cuh -- division by numbers that are fixed for a launch.
#pragma once

#include <stdint.h>

namespace llsa {

// Division of 32-bit numbers by a fixed one, as a product (Granlund and
// Montgomery, Division by Invariant Integers using Multiplication, 1994).
struct Divisor {
  uint32_t d, m, s;
};
inline Divisor divisor(uint32_t d) {
  int l = 0;
  while (l < 32 && (1ull << l) < d) ++l;
  return Divisor{d, (uint32_t)(((1ull << 32) * ((1ull << l) - d)) / d + 1), (uint32_t)l};
}
__host__ __device__ inline uint32_t over(uint32_t n, const Divisor& v) {
  const uint32_t t = (uint32_t)(((uint64_t)v.m * n) >> 32);
  return v.s == 0 ? n : (t + ((n - t) >> 1)) >> (v.s - 1);
}

}  // namespace llsa
