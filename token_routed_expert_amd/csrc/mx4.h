// Microscaled block formats shared by the 4-bit kernels and by the 8-bit
// checkpoint epilogues: 32 values along the contraction axis share one
// power-of-two scale 2^s, stored as the E8M0 byte s + 127.
//
//   s = the smallest integer with amax <= M * 2^s, M = 6 (E2M1: 6 = 1.5 * 2^2)
//   or 448 (E4M3: 448 = 1.75 * 2^8), at least -126 (so that 2^s and 2^-s are
//   normal fp32 numbers), 0 for an all-zero block;
//   code(v) = the nearest value of the format to v * 2^-s, ties to even (the
//   product is exact wherever the code is not zero).
//
// The rounded-up scale never saturates a value.  A block that holds a NaN or
// an infinity gets the E8M0 NaN byte 255: all its values read back as NaN, in
// the matrix instructions too (measured), whatever its codes say.
#pragma once

#include "common.h"

namespace tre {
namespace mx {

constexpr uint32_t kNanScale = 255;

// Magnitude bits of v: ordered like |v| for numbers, infinity above them and
// NaNs above infinity, so one integer maximum finds amax and non-finite values.
__device__ __forceinline__ uint32_t mag(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// E8M0 byte of a block from the largest magnitude bits of its values:
// amax = n * 2^e (n in [1, 2)), s = e - log2(M's power) + (n > M's mantissa).
template <bool FP4>
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax) {
  if (amax == 0) return 127u;
  if (amax >= 0x7f800000u) return kNanScale;
  const int e = (int)(amax >> 23);  // biased; 0 for subnormals
  const int s = e - (FP4 ? 2 : 8) + ((amax & 0x7fffffu) > (FP4 ? 0x400000u : 0x600000u) ? 1 : 0);
  return (uint32_t)max(s, 1);
}
// 2^s and 2^-s of a scale byte in [1, 253].
__device__ __forceinline__ float scale_of(uint32_t b) { return __uint_as_float(b << 23); }
__device__ __forceinline__ float inv_scale_of(uint32_t b) { return __uint_as_float((254u - b) << 23); }
// 2^s of any scale byte a tensor may hold: 0 is 2^-127, 255 is NaN.
__device__ __forceinline__ float scale_any(uint32_t b) {
  return b == 0 ? 0x1p-127f : (b == kNanScale ? __uint_as_float(0x7fc00000u) : scale_of(b));
}

// Eight E2M1 codes (low nibble first) of v[0..7] in a block with scale byte b.
// v_cvt_scalef32_pk_fp4_f32 divides by the scale and rounds to nearest even,
// sign kept (checked at every midpoint and its neighbours, zeros, subnormals);
// its scale operand is the fp32 number 2^s.
__device__ __forceinline__ uint32_t pack8_fp4(const float* v, uint32_t b) {
  const float s = scale_of(b == kNanScale ? 127u : b);
  uint32_t r = 0;
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[0], v[1], s, 0);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[2], v[3], s, 1);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[4], v[5], s, 2);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[6], v[7], s, 3);
  return r;
}
// Four E4M3 codes of v[0..3] times inv = 2^-s (magnitudes at most 448, where
// v_cvt_pk_fp8_f32 rounds to nearest even).
__device__ __forceinline__ uint32_t pack4_fp8(const float* v, float inv) {
  uint32_t r = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[0] * inv, v[1] * inv, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[2] * inv, v[3] * inv, (int)r, true);
}

}  // namespace mx
}  // namespace tre
