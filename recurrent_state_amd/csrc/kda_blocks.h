// Scales of e4m3 pages by blocks of tokens: how a scale follows from the values,
// and how rows already in the pages are stored anew (kda_pages_blocks.hip,
// kda_evict.hip).
#pragma once

#include "kda_pages.h"

namespace kda {
namespace {

typedef __attribute__((ext_vector_type(4))) uint32_t codes16;  // 16 e4m3 values

// 2^-64 and 2^120; at 2^120 every fp32 value is below 448 scales.
constexpr uint32_t kLeastScale = (127u - 64) << 23, kMostScale = (127u + 120) << 23;

// |x| as bits, which order as the values do, infinities and then NaN behind
// kLargest; and with 0 for what is not finite.
constexpr uint32_t kLargest = 0x7f7fffffu;
__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7fffffffu; }
__device__ __forceinline__ uint32_t finite_bits(float x) {
  const uint32_t b = magnitude(x);
  return b <= kLargest ? b : 0;
}
// The bits of the least power of two s >= 2^-64 with m <= 448 s, m given by its
// bits: 448 = 1.75 * 2^8, so with m = f * 2^x the exponent is x - 8, one more where
// f > 1.75 (mantissa bits above 0x600000: the sum carries).
__device__ __forceinline__ uint32_t scale_for(uint32_t m) {
  const uint32_t e = (m + 0x1fffffu) >> 23;
  return max(e < 8 ? 0 : (e - 8) << 23, kLeastScale);
}
// s rounded up to a power of two, for scales that no append has set.
__device__ __forceinline__ uint32_t power_of_two(float s) {
  return min(max((__float_as_uint(s) + 0x7fffffu) & 0x7f800000u, kLeastScale), kMostScale);
}
// 1 / s of a power of two within the limits, exactly.
__device__ __forceinline__ float inverse(uint32_t s) { return __uint_as_float((254u << 23) - s); }

__device__ __forceinline__ uint32_t wave_max(uint32_t x) {
#pragma unroll
  for (int i = 1; i < kWave; i *= 2) x = max(x, (uint32_t)__shfl_xor((int)x, i));
  return x;
}

// Codes times f, rounded to nearest even; NaN stays NaN.  CLAMP: products may pass
// 448, since a scale past 2^120 (no call sets one) stands for values that fp32 does
// not hold.
template <bool CLAMP>
__device__ __forceinline__ codes16 times(codes16 x, float f) {
  const auto in = [](float y) { return CLAMP ? to_range(y) : y; };
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)x[i], false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)x[i], true);
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(in(lo[0] * f), in(lo[1] * f), 0, false);
    x[i] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(in(hi[0] * f), in(hi[1] * f), w, true);
    if (CLAMP) asm volatile("" : "+v"(x[i]), "+v"(f));  // four codes at a time: few registers
  }
  return x;
}
// Codes of scale `old` in a block that holds other rows too and has the scale s.  That
// may be 2^184 times less where these are all zeros: the factor ends at fp32's largest,
// since 0 times infinity would be NaN.
__device__ __forceinline__ codes16 rescaled(codes16 x, float old, uint32_t s) {
  const float f = old * inverse(s), most = __uint_as_float(kLargest);
  if (magnitude(old) > kMostScale) return times<true>(x, magnitude(old) <= kLargest ? fminf(fmaxf(f, -most), most) : f);
  return times<false>(x, fminf(fmaxf(f, -most), most));
}

}  // namespace
}  // namespace kda
