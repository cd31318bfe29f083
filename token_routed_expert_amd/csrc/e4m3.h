// The e4m3 block rule: one fp32 scale per block, OCP E4M3FN codes (shared by the
// quantisers and by the norm that writes quantised rows).
#pragma once

#include "common.h"

namespace tre {
namespace e4m3 {

constexpr float kE4M3Max = 448.0f;

// E4M3FN code of a finite fp32 value, from the format: sign bit, 4 exponent
// bits with bias 7, 3 mantissa bits; normals from 2^-6 to 448, subnormals
// m * 2^-9.  Round to nearest, ties to even; |v| >= 448 gives 448 (0x7e).
// gfx950's v_cvt_pk_fp8_f32 produces exactly these codes for |v| < 464 (a
// comparison over every fp32 value of magnitude below 2^9, both signs,
// subnormals and ties included) and NaN above, so the value is clamped to
// +-448 first (the sign of -0 is kept).
__device__ __forceinline__ uint32_t e4m3_code(float v) {
  const float c = __builtin_amdgcn_fmed3f(v, -448.0f, 448.0f);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, 0.0f, 0, false) & 0xffu;
}

__device__ __forceinline__ float block_scale(float amax) {
  return amax == 0.0f ? 1.0f : amax / kE4M3Max;
}

// Code of v in a block with scale `scale` (zero_block: the block's amax is 0).
__device__ __forceinline__ uint32_t quant1(float v, float scale, bool zero_block) {
  return zero_block ? 0u : e4m3_code(v / scale);
}

// The quotient v / s without a division per value.  With y = fp32(1 / s),
// the product q0 = fp32(v y) is corrected once by the remainder v - s q0,
// which one FMA gives exactly (the correction step of Markstein's division
// method).  For s >= kFastDivMin this equals the IEEE quotient fp32(v / s)
// whenever that quotient is at least 2^-14 in magnitude -- checked on the CPU
// over every bf16 pair |v| <= 448 s and over 1.3e9 fp32 pairs, among them
// values placed on and next to the midpoints between e4m3 codes.  Smaller
// quotients may differ in their last bits but give code +0 or -0 either way,
// and the sign is taken from v (the FMAs turn -0 into +0).
constexpr float kFastDivMin = 0x1p-90f;
__device__ __forceinline__ float div_by_scale(float v, float s, float y) {
  const float q0 = v * y;
  return __builtin_copysignf(__builtin_fmaf(__builtin_fmaf(-q0, s, v), y, q0), v);
}
// quant1 through div_by_scale (FAST) or the IEEE division.
template <bool FAST>
__device__ __forceinline__ uint32_t quant1s(float v, float s, float y, bool zero_block) {
  return zero_block ? 0u : e4m3_code(FAST ? div_by_scale(v, s, y) : v / s);
}

}  // namespace e4m3
}  // namespace tre
