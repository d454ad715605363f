// rollout_divisor.h -- division by numbers that a launch knows beforehand.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fp4q {

// Division of n < 2^31 by a divisor known on the host: a product and a
// shift.  With l = ceil(log2 d) and m = ceil(2^(31+l) / d), m d = 2^(31+l) + r
// with r < d, and n r < 2^(31+l) keeps the quotient exact.
struct Divisor {
  uint32_t d, m, shift;
};

inline Divisor divisor_of(uint32_t d) {
  uint32_t l = 0;
  while (((uint64_t)1 << l) < d) ++l;
  return {d, (uint32_t)((((uint64_t)1 << (31 + l)) + d - 1) / d), 31 + l};
}

__device__ __forceinline__ uint32_t quotient(uint32_t n, const Divisor& v) {
  return (uint32_t)(((uint64_t)n * v.m) >> v.shift);
}

}  // namespace fp4q
