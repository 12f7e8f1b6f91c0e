// E4M3 codes with one fp32 scale for a block of values: the rule that the row
// and weight quantisers and the norm share.
//
// With top the largest magnitude of a block (counted as 2^-100 at least),
//   m = 448 / top cut to 16 significant bits,  code = E4M3(x * m),  scale = 1 / m.
// 16 bits of m and 8 of a bf16 x make 24: the product is exact in fp32, so a
// bf16 value gets the code nearest to it at this scale, ties to even. (With all
// 24 bits of m the product would be rounded before it is rounded to a code, and
// values at a tie, a percent of them, would go either way.) m is cut, not
// rounded, so top * m stays at or below 448; m is at most 448 * 2^100, and both
// it and 1 / m are normal numbers.
// A block that holds an infinity or a NaN gets scale NaN and codes 0.
#pragma once

#include "gg_common.h"

namespace gg {

constexpr int kFp8Block = 128;
constexpr float kFp8Max = 448.0f;

// m for a block whose largest magnitude has the fp32 bits `top` (sign cleared);
// 0 where it is not finite, so that every code is 0 (0 * infinity, a NaN, is
// left to the caller's fp8_pair).
__device__ __forceinline__ float fp8_multiplier(uint32_t top) {
  if (top >= 0x7f800000u) return 0.0f;
  const float t = fmaxf(__builtin_bit_cast(float, top), 0x1p-100f);
  return __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, kFp8Max / t) & 0xffffff00u);
}
__device__ __forceinline__ float fp8_scale(float m) {
  return m == 0.0f ? __builtin_bit_cast(float, 0x7fc00000u) : 1.0f / m;
}

// Two values over their scale -> two codes in half HIGH of a dword
// (v_cvt_pk_fp8_f32: nearest, ties to even. Nothing here is above 448, but for the
// norm's values, whose two roundings may pass it by a last bit and which go to 448.)
template <bool HIGH>
__device__ __forceinline__ uint32_t fp8_pair(uint32_t old, float a, float b) {
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(a, b, (int)old, HIGH);
}
__device__ __forceinline__ uint32_t fp8_quad(float a, float b, float c, float d) {
  return fp8_pair<true>(fp8_pair<false>(0, a, b), c, d);
}

__device__ __forceinline__ float bf16_lo(uint32_t two) { return __builtin_bit_cast(float, two << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t two) {
  return __builtin_bit_cast(float, two & 0xffff0000u);
}

// Largest value among the 16 lanes of a row (DPP: quads, then rotations).
__device__ __forceinline__ uint32_t row16_max(uint32_t v) {
  constexpr int kQuad1 = 0xB1, kQuad2 = 0x4E, kRor4 = 0x124, kRor8 = 0x128;
  auto other = [](uint32_t x, auto c) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, decltype(c)::value, 0xf, 0xf, true);
  };
  v = max(v, other(v, std::integral_constant<int, kQuad1>{}));
  v = max(v, other(v, std::integral_constant<int, kQuad2>{}));
  v = max(v, other(v, std::integral_constant<int, kRor4>{}));
  return max(v, other(v, std::integral_constant<int, kRor8>{}));
}

}  // namespace gg
