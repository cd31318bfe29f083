// The experts' forward with 4-bit integer weights in scaled groups (i4.h) and bf16
// activations:
//
//   fc1:  [a | b] = x W13,  h = silu(a) b, rounded to bf16 in the epilogue
//   fc2:  o = h W2
//
// on v_mfma_f32_16x16x32_bf16, fp32 accumulation.  The weights are the first operand
// (rows of D = C^T: four consecutive output columns per lane), decoded to bf16 in
// registers: a lane's 16 bytes of a 128-row tile are its operands of four products.
// W13 holds W1's and W3's 16-column groups alternately, so a lane holds a and b of
// the same element.
#include "gemm_common.h"
#include "i4.h"

namespace tre {

namespace {
using namespace gemm;

typedef int i32x4_t __attribute__((ext_vector_type(4)));

__device__ __forceinline__ f32x4_t mma(const bf16x8_t& w, const bf16x8_t& x, const f32x4_t& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, x, c, 0, 0, 0);
}

// Epilogue of fc1 for one 16-row fragment: acc = [a0 b0 a1 b1] (16 columns of f each;
// lane l: row l & 15, columns 4 (l >> 4)..+3) -> h of the 32 columns from col on.
__device__ __forceinline__ void store_h(const f32x4_t (&acc)[4], bool ok, size_t row, int col, int f, int lane,
                                        bf16_t* h) {
  f32x4_t h0, h1;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    h0[q] = silu_f32(acc[0][q]) * acc[1][q];
    h1[q] = silu_f32(acc[2][q]) * acc[3][q];
  }
  const int pc = ((lane >> 4) & 1) * 16 + (lane >> 5) * 8;
  const u32x4_t v = pair_bf16(h0, h1);
  if (ok) *(u32x4_t*)(h + row * (size_t)f + col + pc) = v;
}

// Epilogue of fc2 for one 16-row fragment: 64 columns from col on.
__device__ __forceinline__ void store_o(const f32x4_t (&acc)[4], bool ok, size_t row, int col, int d, int lane,
                                        bf16_t* o) {
  const int pc = ((lane >> 4) & 1) * 16 + (lane >> 5) * 8;
  const u32x4_t v0 = pair_bf16(acc[0], acc[1]), v1 = pair_bf16(acc[2], acc[3]);
  if (!ok) return;
  bf16_t* p = o + row * (size_t)d + col + pc;
  *(u32x4_t*)p = v0;
  *(u32x4_t*)(p + 32) = v1;
}

// Few rows: a block of NW wavefronts takes 64 stored columns of one expert and up to
// 32 of its rows; the wavefronts split K (wavefront w takes the 128-row steps w,
// w + NW, ...) and their partial sums meet in LDS, added in wavefront order.  Blocks
// take the pieces of 32 rows that the experts have, in order, so a call with few rows
// launches few blocks.  U: groups of a 128-row step.
constexpr int NW = 4;
template <int FC, int U>
__global__ __launch_bounds__(NW * 64) void gemm_i4_rows_kernel(I4Args args) {
  __shared__ f32x4_t part[2][NW][4][64];
  const int lane = threadIdx.x & 63, g = lane >> 4, r = lane & 15;
  const int w = uniform((int)threadIdx.x >> 6);
  const int K = FC == 1 ? args.d : args.f, N = FC == 1 ? 2 * args.f : args.d;
  const int KT = K >> 7, NB = N >> 6;
  const int nb = (int)blockIdx.x % NB;
  // the piece: the (blockIdx / NB)-th of the experts' pieces of 32 rows, in order
  int e = -1, row0 = 0, rows = 0;
  {
    int want = (int)blockIdx.x / NB;
    for (int base = 0; base < args.E; base += 64) {
      const int x = base + lane;
      const int o0 = x < args.E ? args.offsets[x] : 0, o1 = x < args.E ? args.offsets[x + 1] : 0;
      const int n = (o1 - o0 + 31) >> 5;
      int end = n;  // pieces of this expert and of those before it
#pragma unroll
      for (int i = 1; i < 64; i *= 2) {
        const int v = __shfl_up(end, i, 64);
        end += lane >= i ? v : 0;
      }
      const uint64_t past = __ballot(end > want);
      if (past) {
        const int at = __builtin_ctzll(past);
        const int first = 32 * (want - __shfl(end - n, at, 64));
        e = base + at;
        row0 = __shfl(o0, at, 64) + first;
        rows = min(__shfl(o1, at, 64) - row0, 32);
        break;
      }
      want -= __shfl(end, 63, 64);
    }
  }
  e = uniform(e);
  if (e < 0) return;
  row0 = uniform(row0);
  rows = uniform(rows);
  const uint8_t* wt = args.w + ((size_t)e * (N >> 4) + (size_t)nb * 4) * KT * 1024 + lane * 16;
  const uint32_t* wst = args.ws + (((size_t)e * NB + nb) * KT * U) * 64 + r * 4;
  const size_t wstride = (size_t)KT * 1024;  // from one 16-column group to the next
  // the rows as MT fragments of 16, UF steps' loads of a wavefront in flight together
  auto run = [&](auto MTC, auto UFC) __attribute__((always_inline)) {
    constexpr int MT = decltype(MTC)::value, UF = decltype(UFC)::value;
    const bf16_t* at[MT];
    bool known[MT], all_known = true;
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      // rows past the last are read as the last one and not stored; a token that
      // there is not counts as a row of zeros (not its results: 0 times a NaN is NaN)
      const int pr = row0 + min(16 * t + r, rows - 1);
      size_t ar = (size_t)pr;
      known[t] = true;
      if (FC == 1 && args.token_of) {
        const uint32_t token = (uint32_t)args.token_of[pr];
        known[t] = token < (uint32_t)args.T;
        ar = known[t] ? token : 0;
        all_known = all_known && known[t];
      }
      at[t] = args.a + ar * (size_t)K + g * 8;
    }
    all_known = __all(all_known);
    f32x4_t acc[MT][4];
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[t][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    for (int k0 = w; k0 < KT; k0 += NW * UF) {
      i32x4_t wf[UF][4], sw[UF][U], xf[UF][MT][4];
#pragma unroll
      for (int u = 0; u < UF; ++u) {
        const int kt = k0 + NW * u;
        if (kt < KT) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            wf[u][j] = __builtin_nontemporal_load((const i32x4_t*)(wt + j * wstride + (size_t)kt * 1024));
#pragma unroll
          for (int i = 0; i < U; ++i) sw[u][i] = *(const i32x4_t*)(wst + ((size_t)kt * U + i) * 64);
#pragma unroll
          for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int j = 0; j < 4; ++j) xf[u][t][j] = *(const i32x4_t*)(at[t] + (size_t)kt * 128 + j * 32);
        }
      }
#pragma unroll
      for (int u = 0; u < UF; ++u) {
        if (k0 + NW * u < KT) {
          if (!all_known) {
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
              for (int j = 0; j < 4; ++j) xf[u][t][j] = known[t] ? xf[u][t][j] : i32x4_t{0, 0, 0, 0};
          }
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            float s = 0.f, nzs = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              if (j * U % 4 == 0) i4::unpack((uint32_t)sw[u][j * U / 4][c], s, nzs);
              const bf16x8_t wv = i4::operand((uint32_t)wf[u][c][j], s, nzs);
#pragma unroll
              for (int t = 0; t < MT; ++t) acc[t][c] = mma(wv, __builtin_bit_cast(bf16x8_t, xf[u][t][j]), acc[t][c]);
            }
          }
        }
      }
    }
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int j = 0; j < 4; ++j) part[t][w][j][lane] = acc[t][j];
    __syncthreads();
    if (w >= MT) return;  // wavefront t stores rows 16 t ..
    f32x4_t sum[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f32x4_t s = part[w][0][j][lane];
#pragma unroll
      for (int i = 1; i < NW; ++i) {
        const f32x4_t p = part[w][i][j][lane];
#pragma unroll
        for (int q = 0; q < 4; ++q) s[q] += p[q];
      }
      sum[j] = s;
    }
    const int m = 16 * w + r;
    const size_t row = (size_t)(row0 + m);
    if constexpr (FC == 1) store_h(sum, m < rows, row, nb * 32, args.f, lane, args.h);
    else store_o(sum, m < rows, row, nb * 64, args.d, lane, args.o);
  };
  if (rows <= 16) run(IntC<1>{}, IntC<2>{});
  else run(IntC<2>{}, IntC<1>{});
}

template <int FC, int U>
int launch_rows(const I4Args& a, hipStream_t s) {
  const int64_t NB = (FC == 1 ? 2 * (int64_t)a.f : (int64_t)a.d) / 64;
  // at most sum_e ceil(m_e / 32) pieces, P with fewer rows than experts
  const int64_t grid = NB * (a.P / 32 + (a.P < a.E ? a.P : a.E));
  if (!launch_fits(grid, NW * 64)) return MOE_ERR_UNSUPPORTED;
  gemm_i4_rows_kernel<FC, U><<<(unsigned)grid, NW * 64, 0, s>>>(a);
  TRE_LAUNCH_CHECK();
  return MOE_OK;
}

template <int FC>
int launch_fc(const I4Args& a, hipStream_t s) {
  if (a.group == 128) return launch_rows<FC, 1>(a, s);
  if (a.group == 64) return launch_rows<FC, 2>(a, s);
  return launch_rows<FC, 4>(a, s);
}

}  // namespace

int gemm_i4_launch(int fc, const I4Args& a, hipStream_t s) {
  return fc == 1 ? launch_fc<1>(a, s) : launch_fc<2>(a, s);
}

}  // namespace tre
