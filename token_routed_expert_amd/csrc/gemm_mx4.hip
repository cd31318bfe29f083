// The experts' forward with MXFP4 weights (E2M1 codes, one E8M0 scale per 32
// values along the contraction) and MXFP4 or MXFP8 activations:
//
//   fc1:  [a | b] = x W13,  h = silu(a) b, quantised in the epilogue
//   fc2:  o = h W2                                          (bf16)
//
// on v_mfma_scale_f32_16x16x128_f8f6f4, fp32 accumulation.  The instruction
// takes the weights as its first operand (rows of D = C^T: four consecutive
// output columns per lane) and the activations as its second.  Operand layouts
// (measured with a probe): lane 16 g + r supplies row r; E2M1: the 32 values
// of K group g, low nibble first; E4M3: values [16 g, 16 g + 16) and
// [64 + 16 g, 64 + 16 g + 16); the E8M0 byte of 32-value group g of a row
// comes from lane 16 g + r for both.  Its sums (measured): products of two E2M1
// numbers are added exactly to the fp32 accumulator's rounding; with an E4M3
// operand the products of each 8 consecutive k of a lane are first cut, toward
// zero, to multiples of 2^-13 of the largest one's binade.  W13 holds W1's and W3's 16-column groups
// alternately, so a lane holds a and b of the same element.
//
// h is quantised straight from the fp32 products: silu(a) b is rounded once,
// to the format fc2 reads, and neither a, b nor an unquantised h leaves the
// registers.
#include "gemm_common.h"

namespace tre {

namespace {
using namespace gemm;

typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef int i32x4_t __attribute__((ext_vector_type(4)));

// D += W X for one 16 x 16 x 128 block: w fp4, x fp4 or fp8; WSEL: byte of ws.
template <bool A8, int WSEL>
__device__ __forceinline__ f32x4_t mma(const i32x4_t& w, const i32x8_t& x, const f32x4_t& c, int ws,
                                       int xs) {
  const i32x8_t w8 = {w[0], w[1], w[2], w[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w8, x, c, 4, A8 ? 0 : 4, WSEL, ws, 0, xs);
}

// Epilogue of fc1 for one 16-row fragment: acc = [a0 b0 a1 b1] (16 columns of
// f each; lane l: row l & 15, columns 4 (l >> 4)..+3) -> h of the 32 columns
// as one block per row, its codes to hq and its scale byte to hs.  `row`: the
// row's index in the permuted buffers; col: the block's first column.
template <bool A8>
__device__ __forceinline__ void store_h(const f32x4_t (&acc)[4], bool ok, size_t row, int col, int f,
                                        int lane, uint8_t* hq, uint8_t* hs) {
  f32x4_t h0, h1;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    h0[q] = silu_f32(acc[0][q]) * acc[1][q];
    h1[q] = silu_f32(acc[2][q]) * acc[3][q];
  }
  pair_f32(h0, h1);  // the lane's 8 consecutive columns, from pc on
  const int pc = ((lane >> 4) & 1) * 16 + (lane >> 5) * 8;
  float v[8];
  uint32_t m = 0;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    v[q] = h0[q];
    v[4 + q] = h1[q];
  }
#pragma unroll
  for (int q = 0; q < 8; ++q) m = max(m, mx::mag(v[q]));
  m = row_max(m);
  const uint32_t b = mx::scale_byte<!A8>(m);
  if (!ok) return;
  if constexpr (A8) {
    const float inv = mx::inv_scale_of(b == mx::kNanScale ? 127u : b);
    *(uint2*)(hq + row * (size_t)f + col + pc) = make_uint2(mx::pack4_fp8(v, inv), mx::pack4_fp8(v + 4, inv));
  } else {
    *(uint32_t*)(hq + row * (size_t)(f / 2) + (col + pc) / 2) = mx::pack8_fp4(v, b);
  }
  if (lane < 16) hs[row * (size_t)(f / 32) + col / 32] = (uint8_t)b;
}

// Epilogue of fc2 for one 16-row fragment: 64 columns from col on as bf16.
__device__ __forceinline__ void store_o(const f32x4_t (&acc)[4], bool ok, size_t row, int col, int d,
                                        int lane, bf16_t* o) {
  const int pc = ((lane >> 4) & 1) * 16 + (lane >> 5) * 8;
  const u32x4_t v0 = pair_bf16(acc[0], acc[1]), v1 = pair_bf16(acc[2], acc[3]);
  if (!ok) return;
  bf16_t* p = o + row * (size_t)d + col + pc;
  *(u32x4_t*)p = v0;
  *(u32x4_t*)(p + 32) = v1;
}

// Few rows per expert: the product is bound by reading the weights.  A block
// of four wavefronts takes 64 stored columns of one expert (one scale group)
// and all its rows, 16 at a time; the wavefronts split K (wavefront w takes
// the 128-K steps w, w + 4, ...), read the weight fragments from memory into
// registers as they are stored, and their partial sums meet in LDS, added in
// wavefront order.  Blocks take the experts that have rows, in order, so a
// call with few rows launches few blocks.
template <int FC, bool A8>
__global__ __launch_bounds__(256) void gemm_mx4_rows_kernel(Mx4Args args) {
  constexpr int U = 4;  // K steps whose loads are in flight together
  __shared__ f32x4_t part[4][4][64];
  const int lane = threadIdx.x & 63, g = lane >> 4, r = lane & 15;
  const int w = uniform((int)threadIdx.x >> 6);
  const int K = FC == 1 ? args.d : args.f, N = FC == 1 ? 2 * args.f : args.d;
  const int KT = K >> 7, NB = N >> 6;
  const int nb = (int)blockIdx.x % NB;
  // the expert: the (blockIdx / NB)-th one that has rows
  int e = -1, row0 = 0, rows = 0;
  {
    int want = (int)blockIdx.x / NB;
    for (int base = 0; base < args.E; base += 64) {
      const int x = base + lane;
      const int o0 = x < args.E ? args.offsets[x] : 0, o1 = x < args.E ? args.offsets[x + 1] : 0;
      const uint64_t has = __ballot(o1 > o0);
      const int n = __popcll(has);
      if (want < n) {
        uint64_t m = has;
        for (int i = 0; i < want; ++i) m &= m - 1;
        const int at = __builtin_ctzll(m);
        e = base + at;
        row0 = __shfl(o0, at, 64);
        rows = __shfl(o1, at, 64) - row0;
        break;
      }
      want -= n;
    }
  }
  e = uniform(e);
  if (e < 0) return;
  row0 = uniform(row0);
  rows = uniform(rows);
  const uint8_t* wt = args.w + ((size_t)e * (N >> 4) + (size_t)nb * 4) * KT * 1024 + lane * 16;
  const uint8_t* wst = args.ws + ((size_t)e * NB + nb) * KT * 256 + lane * 4;
  const size_t a_ld = A8 ? (size_t)K : (size_t)(K >> 1), as_ld = (size_t)(K >> 5);
  const size_t wstride = (size_t)KT * 1024;  // from one 16-column group to the next
  for (int m0 = 0; m0 < rows; m0 += 16) {
    // rows past the last are read as the last one and not stored
    const int pr = row0 + min(m0 + r, rows - 1);
    const size_t ar = FC == 1 && args.token_of ? (size_t)args.token_of[pr] : (size_t)pr;
    const uint8_t* at = args.a + ar * a_ld + g * 16;
    const uint8_t* ast = args.as + ar * as_ld + g;
    f32x4_t acc[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    for (int k0 = w; k0 < KT; k0 += 4 * U) {
      i32x4_t wf[U][4];
      i32x8_t xf[U];
      int sw[U], sx[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int kt = k0 + 4 * u;
        if (kt < KT) {
#pragma unroll
          for (int j = 0; j < 4; ++j) wf[u][j] = *(const i32x4_t*)(wt + j * wstride + (size_t)kt * 1024);
          sw[u] = *(const int*)(wst + (size_t)kt * 256);
          sx[u] = ast[kt * 4];
          if constexpr (A8) {
            const i32x4_t lo = *(const i32x4_t*)(at + (size_t)kt * 128);
            const i32x4_t hi = *(const i32x4_t*)(at + (size_t)kt * 128 + 64);
            xf[u] = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
          } else {
            const i32x4_t lo = *(const i32x4_t*)(at + (size_t)kt * 64);
            xf[u] = __builtin_shufflevector(lo, i32x4_t{0, 0, 0, 0}, 0, 1, 2, 3, 4, 5, 6, 7);
          }
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (k0 + 4 * u < KT) {
          static_for<0, 4>([&](auto J) __attribute__((always_inline)) {
            acc[J.value] = mma<A8, J.value>(wf[u][J.value], xf[u], acc[J.value], sw[u], sx[u]);
          });
        }
      }
    }
    __syncthreads();  // the previous rows' partial sums have been read
#pragma unroll
    for (int j = 0; j < 4; ++j) part[w][j][lane] = acc[j];
    __syncthreads();
    if (w != 0) continue;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f32x4_t s = part[0][j][lane];
#pragma unroll
      for (int i = 1; i < 4; ++i) {
        const f32x4_t p = part[i][j][lane];
#pragma unroll
        for (int q = 0; q < 4; ++q) s[q] += p[q];
      }
      acc[j] = s;
    }
    const bool ok = m0 + r < rows;
    const size_t row = (size_t)(row0 + m0 + r);
    if constexpr (FC == 1) store_h<A8>(acc, ok, row, nb * 32, args.f, lane, args.hq, args.hs);
    else store_o(acc, ok, row, nb * 64, args.d, lane, (bf16_t*)args.o);
  }
}

template <int FC, bool A8>
int launch_rows(const Mx4Args& a, hipStream_t s) {
  const int64_t NB = (FC == 1 ? 2 * (int64_t)a.f : (int64_t)a.d) / 64;
  const int64_t grid = NB * (a.P < a.E ? a.P : a.E);
  if (grid > 0x7fffffff) return MOE_ERR_UNSUPPORTED;
  gemm_mx4_rows_kernel<FC, A8><<<(unsigned)grid, 256, 0, s>>>(a);
  TRE_LAUNCH_CHECK();
  return MOE_OK;
}

}  // namespace

int gemm_mx4_launch(int fc, bool a8, const Mx4Args& a, hipStream_t s) {
  if (fc == 1) return a8 ? launch_rows<1, true>(a, s) : launch_rows<1, false>(a, s);
  return a8 ? launch_rows<2, true>(a, s) : launch_rows<2, false>(a, s);
}

}  // namespace tre
