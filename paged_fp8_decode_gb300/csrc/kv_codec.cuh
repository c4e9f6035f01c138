// Encoders of the narrow cache formats, shared by the cache writes: the float32
// quotient x / scale to an e2m3, e3m2 or e2m1 code.
#pragma once

#include <stdint.h>

namespace mj {

// e2m3 code of y: round to nearest, ties to even, saturating at 7.5; the
// sign bit (bit 5) follows the sign of y. Magnitudes below 1 are subnormal
// multiples of 1/8; at or above 1 each binade [2^e, 2^(e+1)) has 8 steps of
// 2^e / 8. The scalings by powers of two are exact, so the only rounding is
// the one __float2uint_rn (to nearest even) does; a mantissa that rounds up
// to 8 carries into the next binade's code, which is the correct result.
__device__ __forceinline__ uint32_t e2m3_code(float y) {
  const float a = fminf(fabsf(y), 7.5f);
  uint32_t c;
  if (a < 1.0f) {
    c = __float2uint_rn(a * 8.0f);  // 0 .. 8 (8 = 1.0, the first normal)
  } else {
    const int e = a >= 4.0f ? 2 : (a >= 2.0f ? 1 : 0);
    const float m = a * __int_as_float((127 - e) << 23);  // a / 2^e, in [1, 2)
    c = (uint32_t(e + 1) << 3) + __float2uint_rn((m - 1.0f) * 8.0f);
  }
  return c | (signbit(y) ? 0x20u : 0u);
}

// e3m2 code of y: round to nearest, ties to even, saturating at 28; sign bit
// 5. Below 0.25 the subnormal grid is k/16; each binade [2^e, 2^(e+1)),
// e = -2 .. 4, has 4 steps of 2^e / 4 (code (e + 3) * 4 + step). As in
// e2m3_code the scalings are exact and __float2uint_rn is the one rounding.
__device__ __forceinline__ uint32_t e3m2_code(float y) {
  const float a = fminf(fabsf(y), 28.0f);
  uint32_t c;
  if (a < 0.25f) {
    c = __float2uint_rn(a * 16.0f);  // 0 .. 4 (4 = 0.25, the first normal)
  } else {
    const int e = (__float_as_int(a) >> 23) - 127;          // floor(log2 a), -2 .. 4
    const float m = a * __int_as_float((127 - e) << 23);    // a / 2^e, in [1, 2)
    c = (uint32_t(e + 3) << 2) + __float2uint_rn((m - 1.0f) * 4.0f);
  }
  return c | (signbit(y) ? 0x20u : 0u);
}

// e2m1 code of y: round to nearest, ties to even, saturating at 6; sign bit 3.
// Below 1 the grid is k/2; binades [1, 2), [2, 4), [4, 8) have 2 steps each.
__device__ __forceinline__ uint32_t e2m1_code(float y) {
  const float a = fminf(fabsf(y), 6.0f);
  uint32_t c;
  if (a < 1.0f) {
    c = __float2uint_rn(a * 2.0f);  // 0 .. 2 (2 = 1.0)
  } else {
    const int e = a >= 4.0f ? 2 : (a >= 2.0f ? 1 : 0);
    const float m = a * __int_as_float((127 - e) << 23);  // a / 2^e, in [1, 2)
    c = (uint32_t(e + 1) << 1) + __float2uint_rn((m - 1.0f) * 2.0f);
  }
  return c | (signbit(y) ? 0x8u : 0u);
}

__device__ __forceinline__ void bf16x8_to_float(uint4 v, float x[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

}  // namespace mj
