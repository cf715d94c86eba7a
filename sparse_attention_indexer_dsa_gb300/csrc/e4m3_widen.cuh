// What the kernels that read 8-bit cache rows share: E4M3 codes with a power of
// two widened to BF16, and the exponential of the weights.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

namespace dsa {

namespace attn {

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// E4M3 codes (four to a word) to BF16, times 2^(e8 - 127).  Code bits s.eeee.mmm placed at a BF16's sign, low
// exponent and high mantissa bits read as value * 2^-120 (subnormals included); one exact product with
// 2^(120 + e) restores it.  That is a BF16 up to e8 = 134; FAR: beyond it (values over 2^16) there is a
// second factor.  The NaN code reads as 480 that way.  The quantisers' scale of a block with a NaN is at
// least 247 (the bits of its magnitude are the largest), so every NaN that they stored is FAR, and is put
// back there; so is scale 255, which is NaN.
template <bool FAR, int W>
__device__ __forceinline__ void widen(const uint32_t (&w)[W], uint32_t e8, uint32_t (&o)[2 * W]) {
  const uint32_t first = FAR ? 254u : e8 + 120u;               // 2^(first - 127): BF16 ends at 2^127
  __nv_bfloat162 f;
  *reinterpret_cast<uint32_t*>(&f) = (first << 7) * 0x00010001u;
#pragma unroll
  for (int i = 0; i < W; ++i) {
#pragma unroll
    for (int hlf = 0; hlf < 2; ++hlf) {
      const uint32_t t = __byte_perm(w[i], 0, hlf ? 0x3424 : 0x1404);
      uint32_t b = (t & 0x80008000u) | ((t >> 4) & 0x07F007F0u);
      __nv_bfloat162 v = __hmul2(*reinterpret_cast<__nv_bfloat162*>(&b), f);
      o[2 * i + hlf] = *reinterpret_cast<uint32_t*>(&v);
    }
  }
  if constexpr (FAR) {
    __nv_bfloat162 f2;
    *reinterpret_cast<uint32_t*>(&f2) = ((e8 - 134u + 127u) << 7) * 0x00010001u;
    const __nv_bfloat162 most = __float2bfloat162_rn(e8 == 255u ? -1.f : 57344.f);   // 448 * 2^7: of the numbers
#pragma unroll
    for (int i = 0; i < 2 * W; ++i) {
      const __nv_bfloat162 x = *reinterpret_cast<__nv_bfloat162*>(&o[i]);
      __nv_bfloat162 v = __hmul2(x, f2);
      o[i] = *reinterpret_cast<uint32_t*>(&v) | __hgt2_mask(__habs2(x), most);
    }
  }
}

}  // namespace attn

}  // namespace dsa
