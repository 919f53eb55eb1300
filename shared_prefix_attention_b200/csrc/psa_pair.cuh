// Packed fp32 products, beside the packed sums of psa_device.cuh.
#pragma once

#include <stdint.h>

namespace psa {

__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

}  // namespace psa
