// Division by a number fixed for the call.
#pragma once

#include <stdint.h>

namespace sv {

// The quotient is the high word of a product with 2^32 / d, rounded up (exact while n * d < 2^32; a runtime division
// is about 150 cycles of dependent instructions).
struct Divisor {
    uint32_t d, magic;   // magic 0: d is 1
    __device__ __forceinline__ int of(int n) const { return magic ? (int)__umulhi((uint32_t)n, magic) : n; }
};
inline Divisor divisor(int d) { return {(uint32_t)d, d > 1 ? (uint32_t)(((1ull << 32) + d - 1) / d) : 0u}; }

}  // namespace sv
