// MXFP4 quantisers: E2M1 codes, two to a byte, with one E8M0 scale byte per 32
// values (block rule in mx4.h).
//
// Activations are quantised row by row (blocks along the row, the contraction
// of the expert products).  Expert weights are quantised once, along their
// rows' axis (the forward products' contraction), into the layout that the
// products read: a 16-column x 128-k tile is 1 KB in a row, in the order in
// which the 64 lanes of a wavefront hold it as a matrix operand (lane
// 16 g + r: column r, the 32 k of group g), so a wavefront fetches one operand
// fragment as 64 x 16 consecutive bytes, from memory or from LDS, without a
// swizzle.  Scale bytes follow the same order, four 16-column tiles to a
// 32-bit word (the matrix instruction picks the byte).
#include "internal.h"
#include "mx4.h"

namespace tre {

namespace {

// Eight consecutive values as fp32.
__device__ __forceinline__ void load8(const bf16_t* p, float* v) {
  const u32x4_t w = *(const u32x4_t*)p;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void load8(const float* p, float* v) {
  const f32x4_t a = *(const f32x4_t*)p, b = *(const f32x4_t*)(p + 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = a[i];
    v[4 + i] = b[i];
  }
}

// 1 x 32 blocks along rows; block g covers values [32 g, 32 g + 32) of the
// row-major matrix.  4 lanes per block, 8 values each: a wavefront's load
// covers 16 blocks in one piece.
template <typename T>
__global__ __launch_bounds__(256) void quant_rows_mx4_kernel(const T* __restrict__ src, int64_t nblk,
                                                             uint8_t* __restrict__ codes,
                                                             uint8_t* __restrict__ sb) {
  const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t g = t >> 2;
  const int sub = (int)(t & 3);
  float v[8] = {};
  if (g < nblk) load8(src + g * 32 + sub * 8, v);
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, mx::mag(v[i]));
  m = max(m, (uint32_t)__shfl_xor((int)m, 1, 4));
  m = max(m, (uint32_t)__shfl_xor((int)m, 2, 4));
  const uint32_t b = mx::scale_byte<true>(m);
  if (g < nblk) {
    *(uint32_t*)(codes + g * 16 + sub * 4) = mx::pack8_fp4(v, b);
    if (sub == 0) sb[g] = (uint8_t)b;
  }
}

// Two adjacent columns of a row.
__device__ __forceinline__ float2 load2(const float* p) {
  typedef float f2 __attribute__((ext_vector_type(2)));
  const f2 v = __builtin_nontemporal_load((const f2*)p);
  return make_float2(v[0], v[1]);
}
__device__ __forceinline__ float2 load2(const bf16_t* p) {
  const uint32_t w = __builtin_nontemporal_load((const uint32_t*)p);
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// The place of 16-column group `grp` of source matrix `which` among the
// stored groups: a pair's groups alternate.
__device__ __forceinline__ int stored_group(int grp, int which, int npair) {
  return npair * grp + which;
}

// Weights [E][R][C] (C columns = outputs, R rows = contraction): one block per
// 128 x 128 tile of one source matrix; wavefront g takes the 32 rows of group
// g, a lane two adjacent columns, so a load instruction reads one row's 128
// columns, and a lane holds two whole blocks of 32 values: no exchange between
// lanes.  Bound by memory: W1 and W3 of 128 experts, 4096 x 1536 fp32, take 1308 us
// (5.6 TB/s read and written, where a large copy reaches 5.2).  Grid: (C/128,
// R/128, E * npair).
template <typename T>
__global__ __launch_bounds__(256) void quant_weights_mx4_kernel(const T* __restrict__ W0,
                                                                const T* __restrict__ W1, int npair,
                                                                int R, int C,
                                                                uint8_t* __restrict__ codes,
                                                                uint8_t* __restrict__ sb) {
  const int cb = blockIdx.x, kt = blockIdx.y;
  const int e = blockIdx.z / npair, which = blockIdx.z % npair;
  const int g = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int KT = R >> 7;
  const T* src = (which ? W1 : W0) + ((size_t)e * R + (size_t)kt * 128 + 32 * g) * C + cb * 128 + 2 * lane;
  float v0[32], v1[32];
  uint32_t m0 = 0, m1 = 0;
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    const float2 x = load2(src + (size_t)i * C);
    v0[i] = x.x;
    v1[i] = x.y;
  }
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    m0 = max(m0, mx::mag(v0[i]));
    m1 = max(m1, mx::mag(v1[i]));
  }
  const uint32_t b0 = mx::scale_byte<true>(m0), b1 = mx::scale_byte<true>(m1);
  u32x4_t c0, c1;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    c0[i] = mx::pack8_fp4(v0 + 8 * i, b0);
    c1[i] = mx::pack8_fp4(v1 + 8 * i, b1);
  }
  const int r = (2 * lane) & 15;
  const int G = stored_group(cb * 8 + (lane >> 3), which, npair);
  const size_t NG = (size_t)npair * (C >> 4);
  uint8_t* ct = codes + (((size_t)e * NG + G) * KT + kt) * 1024 + (size_t)(16 * g + r) * 16;
  *(u32x4_t*)ct = c0;
  *(u32x4_t*)(ct + 16) = c1;
  uint8_t* st = sb + (((size_t)e * (NG >> 2) + (G >> 2)) * KT + kt) * 256 + (16 * g + r) * 4 + (G & 3);
  st[0] = (uint8_t)b0;
  st[4] = (uint8_t)b1;
}

// The values that the codes stand for, bf16 [E][R][C] (one matrix or a pair):
// the quantiser's lane mapping run backwards.  An E2M1 value times 2^s is exact
// in bf16 (subnormal results below 2^-133 round).  The same pair takes 754 us
// (5.4 TB/s).
__global__ __launch_bounds__(256) void dequant_weights_mx4_kernel(const uint8_t* __restrict__ codes,
                                                                  const uint8_t* __restrict__ sb,
                                                                  int npair, int R, int C,
                                                                  bf16_t* __restrict__ D0,
                                                                  bf16_t* __restrict__ D1) {
  const int cb = blockIdx.x, kt = blockIdx.y;
  const int e = blockIdx.z / npair, which = blockIdx.z % npair;
  const int g = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int KT = R >> 7;
  const int r = (2 * lane) & 15;
  const int G = stored_group(cb * 8 + (lane >> 3), which, npair);
  const size_t NG = (size_t)npair * (C >> 4);
  const uint8_t* ct = codes + (((size_t)e * NG + G) * KT + kt) * 1024 + (size_t)(16 * g + r) * 16;
  const u32x4_t c0 = __builtin_nontemporal_load((const u32x4_t*)ct);
  const u32x4_t c1 = __builtin_nontemporal_load((const u32x4_t*)(ct + 16));
  const uint8_t* st = sb + (((size_t)e * (NG >> 2) + (G >> 2)) * KT + kt) * 256 + (16 * g + r) * 4 + (G & 3);
  const float s0 = mx::scale_any(st[0]), s1 = mx::scale_any(st[4]);
  bf16_t* dst = (which ? D1 : D0) + ((size_t)e * R + (size_t)kt * 128 + 32 * g) * C + cb * 128 + 2 * lane;
  // E2M1 magnitude code c -> fp32: 0, 0.5, then 2^(c/2 - 1) (1 + (c & 1) / 2)
  auto value = [](uint32_t c, float s) -> float {
    const uint32_t m = c & 7u;
    const float a = m < 2 ? 0.5f * (float)m
                          : __uint_as_float(((126u + (m >> 1)) << 23) | ((m & 1u) << 22));
    return (c & 8u) ? -a * s : a * s;
  };
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    const float a = value((c0[i >> 3] >> (4 * (i & 7))) & 15u, s0);
    const float b = value((c1[i >> 3] >> (4 * (i & 7))) & 15u, s1);
    __builtin_nontemporal_store(pack_bf16x2(a, b), (uint32_t*)(dst + (size_t)i * C));
  }
}

}  // namespace

int quant_rows_mx4_launch(const void* src, bool src_f32, int64_t rows, int64_t cols,
                          uint8_t* codes, uint8_t* sb, hipStream_t s) {
  const int64_t nblk = rows * (cols / 32);
  constexpr int64_t kPart = (int64_t)1 << 29;  // blocks a launch: 2^31 threads
  for (int64_t at = 0; at < nblk; at += kPart) {
    const int64_t n = nblk - at < kPart ? nblk - at : kPart;
    const unsigned grid = (unsigned)((n * 4 + 255) / 256);
    if (src_f32)
      quant_rows_mx4_kernel<float><<<grid, 256, 0, s>>>((const float*)src + at * 32, n, codes + at * 16, sb + at);
    else
      quant_rows_mx4_kernel<bf16_t><<<grid, 256, 0, s>>>((const bf16_t*)src + at * 32, n, codes + at * 16, sb + at);
    TRE_LAUNCH_CHECK();
  }
  return MOE_OK;
}

int quant_weights_mx4_launch(const void* W, const void* Wp, bool src_f32, int64_t E, int64_t R,
                             int64_t C, uint8_t* codes, uint8_t* sb, hipStream_t s) {
  if (E * R * C == 0) return MOE_OK;
  const int npair = Wp ? 2 : 1;
  const dim3 grid((unsigned)(C / 128), (unsigned)(R / 128), (unsigned)(E * npair));
  if (src_f32)
    quant_weights_mx4_kernel<float><<<grid, 256, 0, s>>>((const float*)W, (const float*)Wp, npair,
                                                         (int)R, (int)C, codes, sb);
  else
    quant_weights_mx4_kernel<bf16_t><<<grid, 256, 0, s>>>((const bf16_t*)W, (const bf16_t*)Wp, npair,
                                                          (int)R, (int)C, codes, sb);
  TRE_LAUNCH_CHECK();
  return MOE_OK;
}

int dequant_weights_mx4_launch(const uint8_t* codes, const uint8_t* sb, int64_t E, int64_t R,
                               int64_t C, void* W, void* Wp, hipStream_t s) {
  if (E * R * C == 0) return MOE_OK;
  const int npair = Wp ? 2 : 1;
  const dim3 grid((unsigned)(C / 128), (unsigned)(R / 128), (unsigned)(E * npair));
  dequant_weights_mx4_kernel<<<grid, 256, 0, s>>>(codes, sb, npair, (int)R, (int)C, (bf16_t*)W,
                                                  (bf16_t*)Wp);
  TRE_LAUNCH_CHECK();
  return MOE_OK;
}

}  // namespace tre
