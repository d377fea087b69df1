// route_key.cuh -- order-preserving integer keys of router logits, shared by the map's routing
// kernel and the few-token layer's.
#pragma once

#include <stdint.h>

namespace dmoe {

// Selection key of a logit given as its fp32 image u (a bf16 value in the high half): the high
// half is the order-preserving image (negative -> bits inverted, else sign bit set; -0 taken as
// +0), the low half is `low` = 0xFFFF - expert, so among equal logits the lower expert has the
// larger key.  Exact for every value but NaN; route_key_nan also maps NaN to 0 (below -inf).
__device__ __forceinline__ uint32_t route_key(uint32_t u, uint32_t low) {
  const float f = __fadd_rn(__uint_as_float(u), 0.0f);  // -0 + 0 = +0
  const uint32_t z = __float_as_uint(f);
  const uint32_t neg = (uint32_t)((int32_t)z >> 31);
  return (z ^ (neg & 0x7FFF0000u)) ^ (0x80000000u | low);
}
__device__ __forceinline__ uint32_t route_key_nan(uint32_t u, uint32_t low) {
  return ((u & 0x7FFFFFFFu) > 0x7F800000u) ? low : route_key(u, low);
}

// The bf16 value whose order-preserving image (the high half of a route key) is `ord`, for
// any image but that of NaN.
__device__ __forceinline__ float bf16_from_order(uint32_t ord) {
  const uint32_t bits = (ord & 0x8000u) ? (ord & 0x7FFFu) : (~ord & 0xFFFFu);
  return __uint_as_float(bits << 16);
}

}  // namespace dmoe
