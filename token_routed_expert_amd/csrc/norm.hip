// The root-mean-square norm in front of a layer, with the residual's addition and
// the rows that the layer's products read quantised on the way, and its gradients.
//
//   s = x + residual (rounded to the storage type: the norm is that of the s that
//   is stored, which the backward reads again)
//   rstd = 1 / sqrt(mean s^2 + eps), y = s rstd gamma
//
// The quantised rows come from the fp32 y, not from the stored one: one rounding
// each.  Block rules as in quant.hip (E4M3, 128 values) and mx4.h (32 values).
//
// Bound by memory: a row is read once, held in registers as fp32, and everything
// that is asked for of it leaves in one pass.  16384 rows of 7168 bf16 with residual,
// sum, y and MXFP8 rows 184 us (5.8 TB/s), with MXFP4 rows 176 (5.7); 8200 of 4096 fp32
// with E4M3 rows 112 us (5.1); 8192 of 16384 bf16 without rows 190 (5.7); one row 3.0 us.
#include <type_traits>

#include "common.h"
#include "e4m3.h"
#include "internal.h"
#include "mx4.h"

namespace tre {

namespace {

// Eight consecutive values in storage form.
template <typename T>
struct Raw;
template <>
struct Raw<bf16_t> {
  u32x4_t w;
  __device__ __forceinline__ void load(const bf16_t* p) { w = *(const u32x4_t*)p; }
  __device__ __forceinline__ void zero() { w = u32x4_t{0, 0, 0, 0}; }
  __device__ __forceinline__ float at(int i) const {
    return __uint_as_float((i & 1) ? (w[i >> 1] & 0xffff0000u) : (w[i >> 1] << 16));
  }
};
template <>
struct Raw<float> {
  f32x4_t a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = *(const f32x4_t*)p;
    b = *(const f32x4_t*)(p + 4);
  }
  __device__ __forceinline__ void zero() { a = b = f32x4_t{0.f, 0.f, 0.f, 0.f}; }
  __device__ __forceinline__ float at(int i) const { return i < 4 ? a[i & 3] : b[i & 3]; }
};
__device__ __forceinline__ void store8(bf16_t* p, const float* v) {
  *(u32x4_t*)p = u32x4_t{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                         pack_bf16x2(v[6], v[7])};
}
__device__ __forceinline__ void store8(float* p, const float* v) {
  *(f32x4_t*)p = f32x4_t{v[0], v[1], v[2], v[3]};
  *(f32x4_t*)(p + 4) = f32x4_t{v[4], v[5], v[6], v[7]};
}
// The same past the caches, for what is too large for them.
__device__ __forceinline__ void stream8(bf16_t* p, const float* v) {
  __builtin_nontemporal_store((u32x4_t{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                                       pack_bf16x2(v[6], v[7])}), (u32x4_t*)p);
}
__device__ __forceinline__ void stream8(float* p, const float* v) {
  __builtin_nontemporal_store((f32x4_t{v[0], v[1], v[2], v[3]}), (f32x4_t*)p);
  __builtin_nontemporal_store((f32x4_t{v[4], v[5], v[6], v[7]}), (f32x4_t*)(p + 4));
}
template <bool PAST, typename T>
__device__ __forceinline__ void put8(T* p, const float* v) {
  if constexpr (PAST) stream8(p, v);
  else store8(p, v);
}
// Four consecutive values.
__device__ __forceinline__ f32x4_t four(const float* p) { return *(const f32x4_t*)p; }
__device__ __forceinline__ f32x4_t four(const bf16_t* p) {
  const uint2 w = *(const uint2*)p;
  return f32x4_t{__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                 __uint_as_float(w.y & 0xffff0000u)};
}
__device__ __forceinline__ float rounded(float v, bf16_t) { return bf16_to_f32(f32_to_bf16(v)); }
__device__ __forceinline__ float rounded(float v, float) { return v; }

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false);
}
// Largest v over 4 or 16 consecutive lanes, in each of them.
template <int N>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
  v = max(v, dpp<0xB1>(v));   // lane ^ 1
  v = max(v, dpp<0x4E>(v));   // lane ^ 2
  if constexpr (N == 16) {
    v = max(v, dpp<0x141>(v));  // the other four of eight
    v = max(v, dpp<0x140>(v));  // the other eight of sixteen
  }
  return v;
}
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}

// Sum over the WPR wavefronts of a row, in wavefront order; `red` holds WPR
// floats and is not written again before every wavefront has read it.
template <int WPR>
__device__ __forceinline__ float row_sum(float v, int w, float* red) {
  v = wave_sum(v);
  if constexpr (WPR > 1) {
    if ((threadIdx.x & 63) == 0) red[w] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int i = 1; i < WPR; ++i) v += red[i];
  }
  return v;
}

// Quantised form of a lane's eight values (vector `at` of the row matrix in
// eights); the lanes of a block are neighbours.  Every lane of the wavefront
// calls it; `ok`: the values exist.
template <int Q>
__device__ __forceinline__ void quant8(const float* v, bool ok, size_t at, uint8_t* codes, void* scales) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, mx::mag(v[i]));
  if constexpr (Q == MOE_E4M3) {
    m = lanes_max<16>(m);
    const bool finite = m < 0x7f800000u;
    const float sc = e4m3::block_scale(finite ? __uint_as_float(m) : 0.0f);
    uint32_t lo = 0, hi = 0;
    auto pack = [&](auto fast) __attribute__((always_inline)) {
      constexpr bool F = decltype(fast)::value;
      const float inv = F ? 1.0f / sc : 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        lo |= e4m3::quant1s<F>(v[i], sc, inv, m == 0) << (8 * i);
        hi |= e4m3::quant1s<F>(v[4 + i], sc, inv, m == 0) << (8 * i);
      }
    };
    if (__all(sc >= e4m3::kFastDivMin)) pack(std::true_type{});
    else pack(std::false_type{});
    if (!ok) return;
    *(uint2*)(codes + at * 8) = make_uint2(lo, hi);
    // a block with a NaN or an infinity reads back as NaN
    if ((at & 15) == 0) ((float*)scales)[at >> 4] = finite ? sc : __uint_as_float(0x7fc00000u);
  } else {
    constexpr bool F4 = Q == MOE_MXFP4;
    m = lanes_max<4>(m);
    const uint32_t b = mx::scale_byte<F4>(m);
    if constexpr (F4) {
      if (!ok) return;
      *(uint32_t*)(codes + at * 4) = mx::pack8_fp4(v, b);
    } else {
      const float inv = mx::inv_scale_of(b == mx::kNanScale ? 127u : b);
      if (!ok) return;
      // (an all-zero block has +0 codes, whatever its signs)
      *(uint2*)(codes + at * 8) = m == 0 ? make_uint2(0, 0) : make_uint2(mx::pack4_fp8(v, inv), mx::pack4_fp8(v + 4, inv));
    }
    if ((at & 3) == 0) ((uint8_t*)scales)[at >> 2] = (uint8_t)b;
  }
}

// WPR wavefronts take one row (WPR == 1: a block has four rows), vector i of
// lane l of wavefront w being number (i WPR + w) 64 + l of the row's d / 8.
// x, residual, sum and y may be the same memory: a lane reads all its values of a
// row before it writes any.
template <typename T, int Q, int WPR, int NV, bool PAST>
__global__ __launch_bounds__(WPR == 1 ? 256 : 64 * WPR) void norm_kernel(NormArgs a) {
  __shared__ float red[2][WPR];
  const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6;
  const int w = WPR == 1 ? 0 : wid;
  const int64_t row = WPR == 1 ? (int64_t)blockIdx.x * 4 + wid : blockIdx.x;
  if (WPR == 1 && row >= a.T) return;
  const int nvec = a.d >> 3;
  const size_t base = (size_t)row * (size_t)nvec;  // in vectors
  const T* x = (const T*)a.x + base * 8;
  const T* res = a.residual ? (const T*)a.residual + base * 8 : nullptr;
  Raw<T> xr[NV], rr[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int at = (i * WPR + w) * 64 + lane;
    if (at < nvec) xr[i].load(x + (size_t)at * 8);
    else xr[i].zero();
  }
  if (res) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int at = (i * WPR + w) * 64 + lane;
      if (at < nvec) rr[i].load(res + (size_t)at * 8);
      else rr[i].zero();
    }
  }
  // Eight sums a lane, then a tree, and the root in 64 bits: an error of rstd moves a
  // whole row's values towards rounding borders of the codes.  Its relative error is
  // 3.5e-8 (root mean square over 16384 rows of 7168; elementwise fp32 operations: 4.4e-8).
  // MXFP8 codes that differ from those of the exact v are next to a tie: 57, 70 and 84 of
  // those 117 million values over three inputs (elementwise: 55, 81, 112).
  float v[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int q = 0; q < 8; ++q) v[i][q] = res ? rounded(xr[i].at(q) + rr[i].at(q), T{}) : xr[i].at(q);
  auto squares = [&](float scale, float* r) __attribute__((always_inline)) {
    float sq[8] = {};
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const float t = v[i][q] * scale;
        sq[q] = fmaf(t, t, sq[q]);
      }
    return (double)row_sum<WPR>(((sq[0] + sq[1]) + (sq[2] + sq[3])) + ((sq[4] + sq[5]) + (sq[6] + sq[7])), w, r);
  };
  // Rows whose squares leave fp32's range at either end (the same for all lanes of a
  // row) are added again, scaled.
  double ss = squares(1.0f, red[0]);
  if (!(ss >= 0x1p-60 && ss <= 0x1p120)) ss = ss < 1.0 ? squares(0x1p90f, red[1]) * 0x1p-180 : squares(0x1p-90f, red[1]) * 0x1p180;
  const float rstd = (float)(1.0 / sqrt(ss / (double)a.d + (double)a.eps));
  if (a.rstd && w == 0 && lane == 0) a.rstd[row] = rstd;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if ((i * WPR) * 64 >= nvec) break;
    const int at = (i * WPR + w) * 64 + lane;
    const bool ok = at < nvec;
    Raw<T> g;
    if (ok) g.load((const T*)a.gamma + (size_t)at * 8);
    else g.zero();
    if (ok && a.sum) put8<PAST>((T*)a.sum + (base + at) * 8, v[i]);
#pragma unroll
    for (int q = 0; q < 8; ++q) v[i][q] = v[i][q] * rstd * g.at(q);
    if (ok && a.y) put8<PAST>((T*)a.y + (base + at) * 8, v[i]);
    if constexpr (Q >= 0) quant8<Q>(v[i], ok, base + at, a.codes, a.scales);
  }
}

// a b, rounded by itself (never part of a fused addition).
__device__ __forceinline__ float product(float a, float b) {
#pragma clang fp contract(off)
  return a * b;
}

// dgamma of THREADS / 4 columns from dy, sum and rstd: a thread takes every 16th row of
// four columns, and the 16 parts meet in LDS.  The sums are those of the two kernels
// below, where a team has one row, in the same order.
template <typename T, int THREADS>
__device__ __forceinline__ void few_dgamma(const NormBwdArgs& a, int block) {
  constexpr int L = THREADS / 16;
  __shared__ f32x4_t part[16][L];
  const int l = threadIdx.x % L, w = threadIdx.x / L;
  const int col = (block * L + l) * 4;
  f32x4_t v = {0.f, 0.f, 0.f, 0.f};
  if (col < a.d) {
#pragma unroll 8
    for (int r = w; r < (int)a.T; r += 16) {
      const size_t at = (size_t)r * (size_t)a.d + (size_t)col;
      const f32x4_t dy = four((const T*)a.dy + at), s = four((const T*)a.sum + at);
      const float rstd = a.rstd[r];
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] += product(dy[q], s[q] * rstd);
    }
  }
  part[w][l] = v;
  __syncthreads();
  if (w != 0 || col >= a.d) return;
  v = part[0][l];
#pragma unroll
  for (int i = 1; i < 16; ++i)
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] += part[i][l][q];
#pragma unroll
  for (int q = 0; q < 4; ++q) Elem<T>::store((T*)a.dgamma + col + q, v[q]);
}

// The backward: with g = dy gamma and c = rstd / d sum(g s),
//   dx = dsum + rstd (g - s rstd c),  dgamma = sum over rows of dy s rstd.
// Teams of WPR wavefronts walk the rows with a stride of the number of teams and
// keep their part of dgamma in registers; the parts, [teams][d] fp32, are summed
// in order by a second kernel.  PRE: the next row is on its way while the current
// one is worked on.  dx may be dy, sum or dsum.  Bound by memory: 16384 rows of 7168 bf16 with
// dsum 178 us (5.3 TB/s) and 5 for dgamma.
//
// Rows of more than 8192 values take sixteen wavefronts, whose 128 registers a lane do not
// hold the row, the next one and dgamma: 19 (bf16, two vectors a lane) to 229 (bf16, four)
// of them lie in scratch memory, which bounds these rows: 8192 of 16384 bf16 299 us (3.6
// TB/s), 4096 of 16384 fp32 488 (2.2), 2048 of 32768 fp32 468 (2.3), 4096 of 32768 bf16
// 1090 (1.0).
//
// FEW: one launch for few rows.  Every team has one row, and blocks after theirs take
// dgamma from dy, sum and rstd again.
template <typename T, int WPR, int NV, bool PRE, bool FEW>
__global__ __launch_bounds__(WPR == 1 ? 256 : 64 * WPR) void norm_bwd_kernel(NormBwdArgs a) {
  __shared__ float red[2][WPR];
  if constexpr (FEW) {
    const int rows = WPR == 1 ? (int)(a.T + 3) / 4 : (int)a.T;  // blocks for the rows
    if ((int)blockIdx.x >= rows) {
      few_dgamma<T, WPR == 1 ? 256 : 64 * WPR>(a, (int)blockIdx.x - rows);
      return;
    }
  }
  const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6;
  const int w = WPR == 1 ? 0 : wid;
  const int64_t team = WPR == 1 ? (int64_t)blockIdx.x * 4 + wid : blockIdx.x;
  if (team >= a.teams) return;
  const int nvec = a.d >> 3;
  int at[NV];
  bool ok[NV];
  Raw<T> gm[NV];
  float acc[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    at[i] = (i * WPR + w) * 64 + lane;
    ok[i] = at[i] < nvec;
    if (ok[i]) gm[i].load((const T*)a.gamma + (size_t)at[i] * 8);
    else gm[i].zero();
#pragma unroll
    for (int q = 0; q < 8; ++q) acc[i][q] = 0.0f;
  }
  struct Row {
    Raw<T> s[NV], dy[NV], ds[NV];
    float rstd;
  };
  auto fetch = [&](int64_t r, Row& o) __attribute__((always_inline)) {
    const size_t base = (size_t)r * (size_t)a.d;
    o.rstd = a.rstd[r];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (ok[i]) {
        o.s[i].load((const T*)a.sum + base + (size_t)at[i] * 8);
        o.dy[i].load((const T*)a.dy + base + (size_t)at[i] * 8);
      } else {
        o.s[i].zero();
        o.dy[i].zero();
      }
    }
    if (a.dsum) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (ok[i]) o.ds[i].load((const T*)a.dsum + base + (size_t)at[i] * 8);
        else o.ds[i].zero();
      }
    }
  };
  Row cur, nxt;
  int par = 0;
  if constexpr (PRE) fetch(team, nxt);
  for (int64_t r = team; r < a.T; r += a.teams, par ^= 1) {
    if constexpr (PRE) {
      cur = nxt;
      if (r + a.teams < a.T) fetch(r + a.teams, nxt);
    } else {
      fetch(r, cur);
    }
    float c = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int q = 0; q < 8; ++q) c = fmaf(cur.dy[i].at(q) * gm[i].at(q), cur.s[i].at(q) * cur.rstd, c);
    c = row_sum<WPR>(c, w, red[par]) / (float)a.d;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float o[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const float dy = cur.dy[i].at(q), xhat = cur.s[i].at(q) * cur.rstd;
        // (every fused operation by name: the same bits from every form of this kernel)
        const float v = fmaf(-xhat, c, dy * gm[i].at(q));
        o[q] = a.dsum ? fmaf(cur.rstd, v, cur.ds[i].at(q)) : cur.rstd * v;
        acc[i][q] = fmaf(dy, xhat, acc[i][q]);
      }
      if (ok[i]) store8((T*)a.dx + (size_t)r * (size_t)a.d + (size_t)at[i] * 8, o);
    }
  }
  if constexpr (FEW) return;
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (ok[i]) store8(a.part + (size_t)team * (size_t)a.d + (size_t)at[i] * 8, acc[i]);
}

// dgamma from the teams' parts: a block has 64 columns, its 16 wavefronts take
// the parts in turn and meet in LDS, in wavefront order.
template <typename T>
__global__ __launch_bounds__(1024) void norm_dgamma_kernel(const float* __restrict__ part, int teams, int d,
                                                           T* __restrict__ dgamma) {
  __shared__ float red[16][64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int col = blockIdx.x * 64 + lane;
  float v = 0.0f;
  if (col < d) {
#pragma unroll 8
    for (int t = w; t < teams; t += 16) v += part[(size_t)t * d + col];
  }
  red[w][lane] = v;
  __syncthreads();
  if (w != 0 || col >= d) return;
  v = red[0][lane];
#pragma unroll
  for (int i = 1; i < 16; ++i) v += red[i][lane];
  Elem<T>::store(dgamma + col, v);
}

// The values that rows of codes stand for: a thread takes eight.  16384 rows of 7168
// MXFP8 -> bf16 65 us (5.5 TB/s).
template <int Q, typename T, bool PAST>
__global__ __launch_bounds__(256) void dequant_rows_kernel(const uint8_t* __restrict__ codes,
                                                           const void* __restrict__ scales, int64_t nvec,
                                                           T* __restrict__ dst) {
  const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (at >= nvec) return;
  float v[8];
  if constexpr (Q == MOE_MXFP4) {
    const float s = mx::scale_any(((const uint8_t*)scales)[at >> 2]);
    const uint32_t c = *(const uint32_t*)(codes + at * 4);
    const f32x2_t p[4] = {__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 0),
                          __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 1),
                          __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 2),
                          __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 3)};
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = p[i >> 1][i & 1] * s;
  } else {
    const float s = Q == MOE_E4M3 ? ((const float*)scales)[at >> 4] : mx::scale_any(((const uint8_t*)scales)[at >> 2]);
    const uint2 c = *(const uint2*)(codes + at * 8);
    const f32x2_t p[4] = {__builtin_amdgcn_cvt_pk_f32_fp8((int)c.x, false), __builtin_amdgcn_cvt_pk_f32_fp8((int)c.x, true),
                          __builtin_amdgcn_cvt_pk_f32_fp8((int)c.y, false), __builtin_amdgcn_cvt_pk_f32_fp8((int)c.y, true)};
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = p[i >> 1][i & 1] * s;
  }
  put8<PAST>(dst + at * 8, v);
}

template <typename T, int Q, int WPR, int NV, bool PAST = false>
int fwd_as(const NormArgs& a, hipStream_t s) {
  const int64_t grid = WPR == 1 ? (a.T + 3) / 4 : a.T;
  if (!launch_fits(grid, WPR == 1 ? 256 : 64 * WPR)) return MOE_ERR_UNSUPPORTED;
  norm_kernel<T, Q, WPR, NV, PAST><<<(unsigned)grid, WPR == 1 ? 256 : 64 * WPR, 0, s>>>(a);
  TRE_LAUNCH_CHECK();
  return MOE_OK;
}
template <typename T, int Q>
int fwd_of(const NormArgs& a, hipStream_t s) {
  // Wavefronts to a row: one where it has no more than 1024 values, else four (one,
  // 16384 rows of 7168: 214 us against 187; 8200 of 4096, fp32: 123 against 111), and
  // sixteen where there are too few rows for the chip (177 of 7168: 5.4 us against 7.2)
  // or a row is longer than four hold.
  // sum and y of 32 MB and more, all L2s together, are written past the caches by the
  // forms of one and four wavefronts: 5000 rows of 4096 36.0 us against 28.1, 4096 of 7168
  // 56 / 46, 40000 of 512 34.8 / 28.2.  (Sixteen wavefronts store through them: 8192 rows of
  // 16384 190 us, 5.7 TB/s, which is what the others reach past them.  The codes, which
  // the layer reads next, are not written past them either: it would cost their reader
  // more than it saves here.)
  const int nvec = a.d / 8;
  const bool past = a.T * a.d * (int64_t)sizeof(T) >= (int64_t)1 << 25;
  if (nvec <= 128) return past ? fwd_as<T, Q, 1, 2, true>(a, s) : fwd_as<T, Q, 1, 2>(a, s);
  if (nvec <= 512 && a.T >= 1024) return past ? fwd_as<T, Q, 4, 2, true>(a, s) : fwd_as<T, Q, 4, 2>(a, s);
  if (nvec <= 1024 && a.T >= 1024) return past ? fwd_as<T, Q, 4, 4, true>(a, s) : fwd_as<T, Q, 4, 4>(a, s);
  return nvec <= 1024 ? fwd_as<T, Q, 16, 1>(a, s) : fwd_as<T, Q, 16, 4>(a, s);
}
template <typename T>
int fwd_type(const NormArgs& a, hipStream_t s) {
  if (!a.codes) return fwd_of<T, -1>(a, s);
  if (a.q_dtype == MOE_E4M3) return fwd_of<T, MOE_E4M3>(a, s);
  if (a.q_dtype == MOE_MXFP8) return fwd_of<T, MOE_MXFP8>(a, s);
  return fwd_of<T, MOE_MXFP4>(a, s);
}

// One launch where a row is a team: two launches and one, calls in a row, us: 257 rows of
// 512 fp32 10.4 and 8.0, 512 of 4096 13.0 / 9.9, 512 of 8192 19.8 / 16.9, 1024 of 1024 11.5 /
// 10.0, 2048 of 512 14.2 / 15.2; bf16 256 of 16384 19.8 / 12.2.  (Its blocks for dgamma read
// dy and sum while others write dx, so dx may be neither.)
bool few_rows(const NormBwdArgs& a, size_t bytes) {
  auto apart = [&](const void* p) { return (char*)a.dx + bytes <= (char*)p || (char*)p + bytes <= (char*)a.dx; };
  return a.T > 0 && a.T <= 1024 && a.teams == a.T && apart(a.dy) && apart(a.sum);
}

// PRE where a lane has 64 bytes of each tensor or less: without it and with it, us: 16384
// rows of 4096 bf16 103.7 and 100.3, fp32 207.4 / 204.6, 4096 of 7168 bf16 44.0 / 42.9, 16384
// of 1024 as long; fp32 of 8192 (not taken) 400 / 396.
template <typename T, int WPR, int NV>
int bwd_as(const NormBwdArgs& a, hipStream_t s) {
  constexpr int THREADS = WPR == 1 ? 256 : 64 * WPR;
  const int64_t grid = WPR == 1 ? (a.teams + 3) / 4 : a.teams;
  if (a.few)
    norm_bwd_kernel<T, WPR, NV, false, true><<<(unsigned)(grid + (a.d + THREADS / 4 - 1) / (THREADS / 4)), THREADS, 0, s>>>(a);
  else
    norm_bwd_kernel<T, WPR, NV, (sizeof(T) * NV <= 8), false><<<(unsigned)grid, THREADS, 0, s>>>(a);
  TRE_LAUNCH_CHECK();
  return MOE_OK;
}
template <typename T>
int bwd_of(NormBwdArgs a, hipStream_t s) {
  const int nvec = a.d / 8;
  int st = MOE_OK;
  a.few = few_rows(a, (size_t)a.T * (size_t)a.d * sizeof(T));
  if (a.T > 0) {
    if (nvec <= 128) st = bwd_as<T, 1, 2>(a, s);
    else if (nvec <= 512) st = bwd_as<T, 4, 2>(a, s);
    else if (nvec <= 1024) st = bwd_as<T, 4, 4>(a, s);
    else if (nvec <= 2048) st = bwd_as<T, 16, 2>(a, s);
    else st = bwd_as<T, 16, 4>(a, s);
  }
  if (st || a.few) return st;
  norm_dgamma_kernel<T><<<(unsigned)((a.d + 63) / 64), 1024, 0, s>>>(a.part, (int)a.teams, a.d, (T*)a.dgamma);
  TRE_LAUNCH_CHECK();
  return MOE_OK;
}

template <int Q, typename T>
int dequant_as(const uint8_t* codes, const void* scales, int64_t rows, int64_t cols, void* dst, hipStream_t s) {
  const int64_t nvec = rows * (cols / 8);
  // values of 128 MB and more past the caches (16384 rows of 7168: 71 us against 65)
  const bool past = nvec * 8 * (int64_t)sizeof(T) >= (int64_t)1 << 27;
  constexpr int64_t kPart = (int64_t)1 << 31;  // vectors a launch
  for (int64_t at = 0; at < nvec; at += kPart) {
    const int64_t n = nvec - at < kPart ? nvec - at : kPart;
    const void* sc = Q == MOE_E4M3 ? (const void*)((const float*)scales + at / 16)
                                   : (const void*)((const uint8_t*)scales + at / 4);
    const uint8_t* c = codes + at * (Q == MOE_MXFP4 ? 4 : 8);
    const unsigned grid = (unsigned)((n + 255) / 256);
    if (past) dequant_rows_kernel<Q, T, true><<<grid, 256, 0, s>>>(c, sc, n, (T*)dst + at * 8);
    else dequant_rows_kernel<Q, T, false><<<grid, 256, 0, s>>>(c, sc, n, (T*)dst + at * 8);
    TRE_LAUNCH_CHECK();
  }
  return MOE_OK;
}

}  // namespace

// Teams of the backward: as many as keep the chip busy, each with as many rows as
// the others or one fewer.
static int64_t most_teams(int64_t d) { return d <= 1024 ? 2048 : d <= 8192 ? 512 : 256; }
int64_t norm_bwd_most_teams(int64_t T, int64_t d) { return T < most_teams(d) ? T : most_teams(d); }
int64_t norm_bwd_teams(int64_t T, int64_t d) {
  if (T < 1) return 0;
  const int64_t most = most_teams(d);
  const int64_t rows = (T + most - 1) / most;
  return (T + rows - 1) / rows;
}

int norm_launch(const NormArgs& a, bool f32, hipStream_t s) {
  if (a.T == 0) return MOE_OK;
  return f32 ? fwd_type<float>(a, s) : fwd_type<bf16_t>(a, s);
}

int norm_bwd_launch(const NormBwdArgs& a, bool f32, hipStream_t s) {
  return f32 ? bwd_of<float>(a, s) : bwd_of<bf16_t>(a, s);
}

int dequant_rows_launch(const uint8_t* codes, const void* scales, int q_dtype, int64_t rows, int64_t cols, void* dst,
                        bool f32, hipStream_t s) {
  if (q_dtype == MOE_E4M3)
    return f32 ? dequant_as<MOE_E4M3, float>(codes, scales, rows, cols, dst, s)
               : dequant_as<MOE_E4M3, bf16_t>(codes, scales, rows, cols, dst, s);
  if (q_dtype == MOE_MXFP8)
    return f32 ? dequant_as<MOE_MXFP8, float>(codes, scales, rows, cols, dst, s)
               : dequant_as<MOE_MXFP8, bf16_t>(codes, scales, rows, cols, dst, s);
  return f32 ? dequant_as<MOE_MXFP4, float>(codes, scales, rows, cols, dst, s)
             : dequant_as<MOE_MXFP4, bf16_t>(codes, scales, rows, cols, dst, s);
}

}  // namespace tre
