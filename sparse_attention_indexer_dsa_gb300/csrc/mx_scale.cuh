// UE8M0 scale arithmetic shared by the quantisers (preprocess.cu) and the
// cache writer (paged_cache.cu).
#pragma once

#include <stdint.h>

namespace dsa {

// UE8M0 exponent of a block from the bit pattern of its max magnitude
// (sign cleared).  With amax = m * 2^E, m in [1, 2), the smallest e with
// amax <= 448 * 2^e = 1.75 * 2^(e+8) is E - 8, plus one when m > 1.75 (mantissa
// field above 0x600000).  Adding 0x1FFFFF to the bit pattern carries into the
// exponent field exactly in that case, so the NOSAT exponent is
// ((bits + 0x1FFFFF) >> 23) - 135 and the FLOOR exponent (bits >> 23) - 135.
// Zero, subnormal and tiny magnitudes land at or below -127 and clamp there;
// the largest pattern (NaN) gives 121, so no upper clamp is needed.
__device__ __forceinline__ int mx_exponent_bits(uint32_t amax_bits, uint32_t carry) {
  return max((int)((amax_bits + carry) >> 23) - 135, -127);
}

// mantissa carry for the rule: 0 = NOSAT, 1 = FLOOR
__device__ __forceinline__ uint32_t mx_carry(int rule) { return rule == 1 ? 0u : 0x1FFFFFu; }

// 2^-e as a float for e in [-127, 121] (always a normal number)
__device__ __forceinline__ float exp2_neg(int e) { return __uint_as_float((uint32_t)(127 - e) << 23); }

}  // namespace dsa
