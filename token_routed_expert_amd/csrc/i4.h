// 4-bit integer weights with a scale and a zero point for each group of rows.
//
// The weight of code q (0 .. 15) is bf16(s (q - z)).  A group's scale word is the
// fp32 number s (20 significant bits) whose low four bits hold the zero point z, so
// s q - s z = s (q - z) is exact in fp32 (4 bits times 20) and the weight is rounded
// once: products and moe_dequantize_weights_i4 use the same numbers.
//
// A tile of 128 rows x 16 columns is 1 KB: byte 4 j + b of (row group g, column c)
// holds rows 32 j + 8 g + b (low nibble) and + 4 (high nibble), so the four bytes j
// of lane 16 g + c are that lane's eight values of the j-th 32 rows as a bf16 matrix
// operand.
#pragma once

#include "common.h"

namespace tre {
namespace i4 {

constexpr uint32_t kNanWord = 0x7fc00008u;
// Scales stay below 2^124, so that s z is finite: groups above are NaN.
constexpr uint32_t kTooLarge = 0x7d800000u;

__device__ __forceinline__ float scale_of(uint32_t word) { return __uint_as_float(word & ~15u); }
// s and -s z of a scale word.
__device__ __forceinline__ void unpack(uint32_t word, float& s, float& nzs) {
  s = scale_of(word);
  nzs = -s * (float)(word & 15u);
}

// Four weights from the nibbles in the low halves of t's bytes.  A byte 0 .. 15 is
// the E4M3 number q 2^-9 (the code is linear there), so one conversion gives two
// exact q.
__device__ __forceinline__ void values4(uint32_t t, float s, float nzs, float* v) {
  const f32x2_t a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(t, 512.0f, false);
  const f32x2_t b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(t, 512.0f, true);
  v[0] = fmaf(a[0], s, nzs);
  v[1] = fmaf(a[1], s, nzs);
  v[2] = fmaf(b[0], s, nzs);
  v[3] = fmaf(b[1], s, nzs);
}
// Eight weights, in row order, from one lane's four bytes.
__device__ __forceinline__ void values8(uint32_t w, float s, float nzs, float* v) {
  values4(w & 0x0f0f0f0fu, s, nzs, v);
  values4((w >> 4) & 0x0f0f0f0fu, s, nzs, v + 4);
}
__device__ __forceinline__ bf16x8_t operand(uint32_t w, float s, float nzs) {
  float v[8];
  values8(w, s, nzs, v);
  const u32x4_t r = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                     pack_bf16x2(v[6], v[7])};
  return __builtin_bit_cast(bf16x8_t, r);
}

}  // namespace i4
}  // namespace tre
