// Integer weights in groups (i4.h): quantiser, packing of a checkpoint's codes, and
// the bf16 weights back.
//
// Every kernel takes a 128 x 128 tile of one matrix per block: wavefront j the rows
// 32 j .. 32 j + 31, a lane two adjacent columns, so that a memory instruction covers
// one row's 128 columns.  The codes of a tile (8 KB) pass through LDS, between the
// lanes' own columns and the 16-byte pieces in which they are stored.
//
// Bound by memory: a pair of 64 x 4096 x 1536 fp32 is quantised in 613-651 us (5.6-5.9
// TB/s) and read back in 331-345 us (5.9-6.2); a pair's codes, scales and zero points are
// packed in 231 us (5.5), 8 x 4096 x 14336 with groups of 32 in 171 (4.9); 8 x 384 x 512 bf16,
// 96 blocks, quantised in 9.0 and read back in 3.3 us, most of it one block's way through
// its 64 codes a lane.
#include "i4.h"
#include "internal.h"
#include "mx4.h"

namespace tre {

namespace {

// The tile of this block and where its 16-column groups and scales are stored: the
// groups of a pair of matrices alternate.
struct Tile {
  int cb, kt, e, which, npair, KT;
  size_t NG;  // 16-column groups of the stored matrix
  __device__ __forceinline__ Tile(int npair_, int R, int C) : npair(npair_) {
    cb = blockIdx.x;
    kt = blockIdx.y;
    e = blockIdx.z / npair;
    which = blockIdx.z % npair;
    KT = R >> 7;
    NG = (size_t)npair * (C >> 4);
  }
  __device__ __forceinline__ int group(int nt) const { return npair * (cb * 8 + nt) + which; }
  // first byte of the codes of the tile's nt-th 16 columns
  __device__ __forceinline__ size_t codes_at(int nt) const {
    return (((size_t)e * NG + group(nt)) * KT + kt) * 1024;
  }
  // scale word of column c of the nt-th 16, row group u of U
  __device__ __forceinline__ size_t word_at(int nt, int c, int u, int U) const {
    const int G = group(nt);
    return ((((size_t)e * (NG >> 2) + (G >> 2)) * KT + kt) * U + u) * 64 + 4 * c + (G & 3);
  }
};

// A lane's codes (32 rows of two columns, four dwords each) to the stored tiles.
__device__ __forceinline__ void store_codes(const Tile& t, const uint32_t (&q0)[4], const uint32_t (&q1)[4],
                                            uint32_t* lds, uint8_t* codes) {
  const int lane = threadIdx.x & 63, j = threadIdx.x >> 6;
  const int nt = lane >> 3, c = (2 * lane) & 15;
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    lds[nt * 256 + (16 * g + c) * 4 + j] = q0[g];
    lds[nt * 256 + (16 * g + c + 1) * 4 + j] = q1[g];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int p = i * 256 + (int)threadIdx.x;  // 16-byte piece
    *(u32x4_t*)(codes + t.codes_at(p >> 6) + (size_t)(p & 63) * 16) = *(const u32x4_t*)(lds + p * 4);
  }
}

__device__ __forceinline__ float2 load2(const float* p) {
  const f32x2_t v = __builtin_nontemporal_load((const f32x2_t*)p);
  return make_float2(v[0], v[1]);
}
__device__ __forceinline__ float2 load2(const bf16_t* p) {
  const uint32_t w = __builtin_nontemporal_load((const uint32_t*)p);
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

struct Range {
  uint32_t mag;  // largest magnitude bits: non-finite values show here
  float lo, hi;  // smallest and largest value, zero among them
};

// The group's scale word: the smallest scale of 20 significant bits, 2^-126 or more,
// that reaches its largest value (in 64 bits: the span of two fp32 numbers need not
// be one), 1 for a group of zeros, NaN for one that is not finite or too large.
__device__ __forceinline__ uint32_t scale_word(const Range& r, bool asym) {
  if (r.mag >= 0x7f800000u) return i4::kNanWord;
  const double span = asym ? (double)r.hi - (double)r.lo : (double)__uint_as_float(r.mag);
  const double n = asym ? 15.0 : 7.0;
  if (span == 0.0) return 0x3f800000u | (asym ? 0u : 8u);
  uint32_t bits = max(__float_as_uint((float)(span / n)) & ~15u, 0x00800000u);
  if ((double)__uint_as_float(bits) * n < span) bits += 16;
  if (bits >= i4::kTooLarge) return i4::kNanWord;
  if (!asym) return bits | 8u;
  const double z = rint(-(double)r.lo / (double)__uint_as_float(bits));
  return bits | (uint32_t)fmin(fmax(z, 0.0), 15.0);
}

// Code of w: round(w / s) + z, held to 0 .. 15, ties to even.  The product with 1 / s
// is at most one off, next to a half; the remainder w - q s is exact (|q s| <= 2 |w| or
// q = 0) and decides.
__device__ __forceinline__ uint32_t code_of(float w, float s, float rs, float z) {
  float q = rintf(w * rs);
  const float r = fmaf(-q, s, w), twice = 2.0f * fabsf(r);
  const bool odd = ((int)q & 1) != 0;
  if (twice > s || (twice == s && odd)) q += r > 0.0f ? 1.0f : -1.0f;
  return (uint32_t)fminf(fmaxf(q + z, 0.0f), 15.0f);
}

template <typename T>
__global__ __launch_bounds__(256) void quant_weights_i4_kernel(const T* __restrict__ W0, const T* __restrict__ W1,
                                                               int npair, int R, int C, int group, int asym,
                                                               uint8_t* __restrict__ codes,
                                                               uint32_t* __restrict__ words) {
  __shared__ __attribute__((aligned(16))) uint32_t lds[2048];
  __shared__ Range part[4][128];
  const Tile t(npair, R, C);
  const int lane = threadIdx.x & 63, j = threadIdx.x >> 6;
  const T* src = (t.which ? W1 : W0) + ((size_t)t.e * R + (size_t)t.kt * 128 + 32 * j) * C + t.cb * 128 + 2 * lane;
  float v[2][32];
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    const float2 x = load2(src + (size_t)i * C);
    v[0][i] = x.x;
    v[1][i] = x.y;
  }
  Range r[2];
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    r[p] = Range{0u, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      r[p].mag = max(r[p].mag, mx::mag(v[p][i]));
      r[p].lo = fminf(r[p].lo, v[p][i]);
      r[p].hi = fmaxf(r[p].hi, v[p][i]);
    }
  }
  const int U = 128 / group, per = 4 / U;  // wavefronts that share a group
  if (per > 1) {
#pragma unroll
    for (int p = 0; p < 2; ++p) part[j][2 * lane + p] = r[p];
    __syncthreads();
    for (int i = 1; i < per; ++i) {
      const int o = (j & ~(per - 1)) + ((j + i) & (per - 1));
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const Range x = part[o][2 * lane + p];
        r[p].mag = max(r[p].mag, x.mag);
        r[p].lo = fminf(r[p].lo, x.lo);
        r[p].hi = fmaxf(r[p].hi, x.hi);
      }
    }
  }
  uint32_t q[2][4];
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const uint32_t word = scale_word(r[p], asym != 0);
    const float s = i4::scale_of(word), rs = 1.0f / s, z = (float)(word & 15u);
    if ((j & (per - 1)) == 0) words[t.word_at(lane >> 3, ((2 * lane) & 15) + p, j / per, U)] = word;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      q[p][g] = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        q[p][g] |= code_of(v[p][8 * g + i], s, rs, z) << (8 * (i & 3) + 4 * (i >> 2));
    }
  }
  store_codes(t, q[0], q[1], lds, codes);
}

// A checkpoint's codes (one to a byte), scales and zero points (NULL: 8).
__global__ __launch_bounds__(256) void pack_weights_i4_kernel(I4Source a, I4Source b, int npair, int R, int C,
                                                              int group, uint8_t* __restrict__ codes,
                                                              uint32_t* __restrict__ words) {
  __shared__ __attribute__((aligned(16))) uint32_t lds[2048];
  const Tile t(npair, R, C);
  const I4Source in = t.which ? b : a;
  const int lane = threadIdx.x & 63, j = threadIdx.x >> 6;
  const int col = t.cb * 128 + 2 * lane;
  const uint8_t* src = in.q + ((size_t)t.e * R + (size_t)t.kt * 128 + 32 * j) * C + col;
  uint32_t q[2][4] = {};
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    const uint32_t x = *(const uint16_t*)(src + (size_t)i * C);
    const int at = 8 * (i & 3) + 4 * ((i >> 2) & 1);
    q[0][i >> 3] |= (x & 15u) << at;
    q[1][i >> 3] |= (x >> 8 & 15u) << at;
  }
  const int U = 128 / group, per = 4 / U;
  if ((j & (per - 1)) == 0) {
    const int u = j / per;
    const size_t row = ((size_t)t.e * (R / group) + (size_t)t.kt * U + u) * C + col;
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      // the scale to 20 significant bits, to nearest even (the carry of a finite number
      // stays within its magnitude bits), then the border of what a scale may be
      const uint32_t given = __float_as_uint(in.s[row + p]);
      uint32_t bits = (given + 7u + (given >> 4 & 1u)) & ~15u;
      if ((given & 0x7fffffffu) >= 0x7f800000u || (bits & 0x7fffffffu) >= i4::kTooLarge) bits = 0x7fc00000u;
      words[t.word_at(lane >> 3, ((2 * lane) & 15) + p, u, U)] = bits | (in.z ? in.z[row + p] & 15u : 8u);
    }
  }
  store_codes(t, q[0], q[1], lds, codes);
}

__global__ __launch_bounds__(256) void dequant_weights_i4_kernel(const uint8_t* __restrict__ codes,
                                                                 const uint32_t* __restrict__ words, int npair, int R,
                                                                 int C, int group, bf16_t* __restrict__ D0,
                                                                 bf16_t* __restrict__ D1) {
  __shared__ __attribute__((aligned(16))) uint32_t lds[2048];
  const Tile t(npair, R, C);
  const int lane = threadIdx.x & 63, j = threadIdx.x >> 6;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int p = i * 256 + (int)threadIdx.x;
    *(u32x4_t*)(lds + p * 4) =
        __builtin_nontemporal_load((const u32x4_t*)(codes + t.codes_at(p >> 6) + (size_t)(p & 63) * 16));
  }
  const int U = 128 / group, u = j * U / 4;
  const int nt = lane >> 3, c = (2 * lane) & 15;
  float s[2], nzs[2];
#pragma unroll
  for (int p = 0; p < 2; ++p) i4::unpack(words[t.word_at(nt, c + p, u, U)], s[p], nzs[p]);
  __syncthreads();
  bf16_t* dst = (t.which ? D1 : D0) + ((size_t)t.e * R + (size_t)t.kt * 128 + 32 * j) * C + t.cb * 128 + 2 * lane;
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    float v[2][8];
#pragma unroll
    for (int p = 0; p < 2; ++p) i4::values8(lds[nt * 256 + (16 * g + c + p) * 4 + j], s[p], nzs[p], v[p]);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      __builtin_nontemporal_store(pack_bf16x2(v[0][i], v[1][i]), (uint32_t*)(dst + (size_t)(8 * g + i) * C));
  }
}

dim3 tiles_of(int64_t E, int64_t R, int64_t C, int npair) {
  return dim3((unsigned)(C / 128), (unsigned)(R / 128), (unsigned)(E * npair));
}

}  // namespace

int quant_weights_i4_launch(const void* W, const void* Wp, bool src_f32, int64_t E, int64_t R, int64_t C, int group,
                            bool asym, uint8_t* codes, uint32_t* words, hipStream_t s) {
  if (E * R * C == 0) return MOE_OK;
  const int npair = Wp ? 2 : 1;
  const dim3 grid = tiles_of(E, R, C, npair);
  if (src_f32)
    quant_weights_i4_kernel<float><<<grid, 256, 0, s>>>((const float*)W, (const float*)Wp, npair, (int)R, (int)C, group,
                                                        asym, codes, words);
  else
    quant_weights_i4_kernel<bf16_t><<<grid, 256, 0, s>>>((const bf16_t*)W, (const bf16_t*)Wp, npair, (int)R, (int)C,
                                                         group, asym, codes, words);
  TRE_LAUNCH_CHECK();
  return MOE_OK;
}

int pack_weights_i4_launch(const I4Source& a, const I4Source& b, int64_t E, int64_t R, int64_t C, int group,
                           uint8_t* codes, uint32_t* words, hipStream_t s) {
  if (E * R * C == 0) return MOE_OK;
  const int npair = b.q ? 2 : 1;
  pack_weights_i4_kernel<<<tiles_of(E, R, C, npair), 256, 0, s>>>(a, b, npair, (int)R, (int)C, group, codes, words);
  TRE_LAUNCH_CHECK();
  return MOE_OK;
}

int dequant_weights_i4_launch(const uint8_t* codes, const uint32_t* words, int64_t E, int64_t R, int64_t C, int group,
                              void* W, void* Wp, hipStream_t s) {
  if (E * R * C == 0) return MOE_OK;
  const int npair = Wp ? 2 : 1;
  dequant_weights_i4_kernel<<<tiles_of(E, R, C, npair), 256, 0, s>>>(codes, words, npair, (int)R, (int)C, group,
                                                                    (bf16_t*)W, (bf16_t*)Wp);
  TRE_LAUNCH_CHECK();
  return MOE_OK;
}

}  // namespace tre
