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

// A row's 128 values of one K step in registers: E2M1 or E4M3.
template <bool A8>
struct Frag {
  typedef i32x4_t type;
};
template <>
struct Frag<true> {
  typedef i32x8_t type;
};

// The registers an E2M1 operand does not use (the instruction reads four).
__device__ __forceinline__ i32x8_t widen(const i32x4_t& v) {
  return __builtin_shufflevector(v, v, 0, 1, 2, 3, -1, -1, -1, -1);
}
__device__ __forceinline__ i32x8_t widen(const i32x8_t& v) { return v; }

// D += W X for one 16 x 16 x 128 block: w fp4, x fp4 or fp8; WSEL: byte of ws.
template <bool A8, int WSEL>
__device__ __forceinline__ f32x4_t mma(const i32x4_t& w, const typename Frag<A8>::type& xf, const f32x4_t& c,
                                       int ws, int xs) {
  const i32x8_t w8 = widen(w), x = widen(xf);
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w8, x, c, 4, A8 ? 0 : 4, WSEL, ws, 0, xs);
}

// Epilogue of fc1 for one 16-row fragment: acc = [a0 b0 a1 b1] (16 columns of
// f each; lane l: row l & 15, columns 4 (l >> 4)..+3) -> h of the 32 columns
// as one block per row, its codes to hq and its scale byte to hs.  `row`: the
// row's index in the permuted buffers; col: the block's first column.
//
// The quantised h lies in panels of 128 columns, [f/128][P] rows of 64 (E2M1)
// or 128 (E4M3) code bytes and of one scale word: what fc2 reads of 128 rows in
// one K step is then one piece of memory.
template <bool A8>
__device__ __forceinline__ void store_h(const f32x4_t (&acc)[4], bool ok, size_t row, int col, size_t P,
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
  const size_t at = (size_t)(col >> 7) * P + row;
  const int c = (col & 127) + pc;
  if constexpr (A8) {
    const float inv = mx::inv_scale_of(b == mx::kNanScale ? 127u : b);
    *(uint2*)(hq + at * 128 + c) = make_uint2(mx::pack4_fp8(v, inv), mx::pack4_fp8(v + 4, inv));
  } else {
    *(uint32_t*)(hq + at * 64 + c / 2) = mx::pack8_fp4(v, b);
  }
  if (lane < 16) hs[at * 4 + (col & 127) / 32] = (uint8_t)b;
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

// Few rows: the product is bound by reading the weights, or by latency where
// there are few of them.  A block of NW wavefronts takes 64 stored columns of one
// expert (one scale group) and up to 32 of its rows; the wavefronts split K
// (wavefront w takes the 128-K steps w, w + NW, ...), read the weight fragments
// from memory into registers as they are stored, and their partial sums meet in
// LDS, added in wavefront order.  Blocks take the pieces of 32 rows that the
// experts have, in order, so a call with few rows launches few blocks, and a
// call whose rows all went to one expert spreads them (2048 rows on one of 128
// experts, d 4096, f 1536, E2M1 rows: 117 us; one block per column group that
// walked them all took 599 us).  The weights are read with non-temporal loads
// (23 tokens of 8 of those experts: fc1 107 -> 100 us, fc2 58 -> 55 us,
// 6.4 TB/s).  Eight wavefronts, or eight K steps in flight, are slower by 5-40 %.
constexpr int NW = 4;  // wavefronts of a block, which split K
template <int FC, bool A8>
__global__ __launch_bounds__(NW * 64) void gemm_mx4_rows_kernel(Mx4Args args) {
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
  const uint8_t* wst = args.ws + ((size_t)e * NB + nb) * KT * 256 + lane * 4;
  // A row: fc1 row-major, fc2 in panels; a K step is a_step / as_step bytes on
  constexpr int ARB = A8 ? 128 : 64;
  const size_t a_ld = FC == 1 ? (size_t)KT * ARB : ARB, as_ld = FC == 1 ? (size_t)KT * 4 : 4;
  const uint32_t a_step = FC == 1 ? ARB : (uint32_t)args.P * ARB;  // (the whole of A: below 2^31 bytes)
  const uint32_t as_step = FC == 1 ? 4 : (uint32_t)args.P * 4;
  const size_t wstride = (size_t)KT * 1024;  // from one 16-column group to the next
  // the rows as MT fragments of 16, U K steps' loads of a wavefront in flight together
  auto run = [&](auto MTC, auto UC) __attribute__((always_inline)) {
    constexpr int MT = decltype(MTC)::value, U = decltype(UC)::value;
    const uint8_t *at[MT], *ast[MT];
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
      at[t] = args.a + ar * a_ld + g * 16;
      ast[t] = args.as + ar * as_ld + g;
    }
    all_known = __all(all_known);
    f32x4_t acc[MT][4];
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[t][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    for (int k0 = w; k0 < KT; k0 += NW * U) {
      i32x4_t wf[U][4];
      typename Frag<A8>::type xf[U][MT];
      int sw[U], sx[U][MT];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int kt = k0 + NW * u;
        if (kt < KT) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            wf[u][j] = __builtin_nontemporal_load((const i32x4_t*)(wt + j * wstride + (size_t)kt * 1024));
          sw[u] = *(const int*)(wst + (size_t)kt * 256);
#pragma unroll
          for (int t = 0; t < MT; ++t) {
            const uint8_t* a = at[t] + (uint32_t)kt * a_step;
            sx[u][t] = ast[t][(uint32_t)kt * as_step];
            if constexpr (A8) {
              const i32x4_t lo = *(const i32x4_t*)a, hi = *(const i32x4_t*)(a + 64);
              xf[u][t] = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
            } else {
              xf[u][t] = *(const i32x4_t*)a;
            }
          }
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (k0 + NW * u < KT) {
          if (!all_known) {
#pragma unroll
            for (int t = 0; t < MT; ++t) {
              xf[u][t] = known[t] ? xf[u][t] : typename Frag<A8>::type{};
              sx[u][t] = known[t] ? sx[u][t] : 127;
            }
          }
#pragma unroll
          for (int t = 0; t < MT; ++t)
            static_for<0, 4>([&](auto J) __attribute__((always_inline)) {
              acc[t][J.value] = mma<A8, J.value>(wf[u][J.value], xf[u][t], acc[t][J.value], sw[u], sx[u][t]);
            });
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
    if constexpr (FC == 1) store_h<A8>(sum, m < rows, row, nb * 32, (size_t)args.P, lane, args.hq, args.hs);
    else store_o(sum, m < rows, row, nb * 64, args.d, lane, (bf16_t*)args.o);
  };
  if (rows <= 16) run(IntC<1>{}, IntC<4>{});
  else run(IntC<2>{}, IntC<2>{});
}

template <int FC, bool A8>
int launch_rows(const Mx4Args& a, hipStream_t s) {
  const int64_t NB = (FC == 1 ? 2 * (int64_t)a.f : (int64_t)a.d) / 64;
  // at most sum_e ceil(m_e / 32) pieces, P with fewer rows than experts
  const int64_t grid = NB * (a.P / 32 + (a.P < a.E ? a.P : a.E));
  if (!launch_fits(grid, NW * 64)) return MOE_ERR_UNSUPPORTED;
  gemm_mx4_rows_kernel<FC, A8><<<(unsigned)grid, NW * 64, 0, s>>>(a);
  TRE_LAUNCH_CHECK();
  return MOE_OK;
}

// Many rows per expert: tiles of 128 rows x 256 stored columns, four
// wavefronts side by side (each all 128 rows x 64 columns, one scale group, as
// 8 x 4 fragments), two blocks to a compute unit, so that one block's prologue,
// epilogue and barrier waits run under the other's products.  K advances 128 a
// stage through two LDS slots; every byte of a stage arrives by buffer_load ...
// lds.  What bounds the kernel beside the matrix cores is the number of cache
// lines that a compute unit can have on the way from L2 (a build whose loads all
// hit L1 took 407 us where this tiling's first form took 557, 65536 rows, 128
// experts, d 4096, f 1536, fc1 with E2M1 rows; one more slot of look-ahead changed
// nothing).  As it is the kernel takes 477-534 us there and fc2 334-363 us (best
// and mean of calls in a row: 3.5 and 2.5 PFLOP/s at best), with E4M3 rows 641-732
// and 409-462 us (the matrix cores alone: 7.2 and 4.3 PFLOP/s).  So every load
// takes whole 128-byte lines where the layout allows it:
//  * B: the wavefronts' 4 fragments each, 1 KB as stored: a lane reads back its
//    own 16 bytes;
//  * A: 128 rows of 128 bytes, the 16-byte chunk c of row r stored at chunk
//    c ^ ((r >> 1) & 7), which spreads the 16 rows of a fragment read over all
//    banks.  That is one stage of E4M3 rows.  E2M1 rows have 64 bytes a stage:
//    fc1, whose rows lie anywhere (token_of), loads two stages together (PAIR);
//    fc2's lie in panels, row next to row, and take 128 rows of 64 bytes a
//    stage, chunk c at c ^ ((r >> 1) & 3);
//  * scales: one word per lane and column group for B, one per row (its four
//    group bytes) for fc2's A.  fc1's A scales are row-major in memory, where a
//    word per row and stage would be as many lines as the codes themselves:
//    they come 16 bytes a row, for four stages together, into one of two
//    buffers (the first two stages of four load the next four's).
// A slot is free once every wavefront has its last fragments in registers: with
// the reads of stage kt done, a wait for stage kt + 1's loads and one barrier,
// the loads of stage kt + 2 that the block shares go there.  A wavefront's own
// B fragments need no barrier: they are loaded as soon as the registers hold
// the stage's, so they have almost two stages to arrive.
template <int FC, bool A8>
__global__ __launch_bounds__(256, 2) void gemm_mx4_tile_kernel(Mx4Args args, int NT) {
  constexpr int BM = 128, BN = 256, FM = BM / 16;
  constexpr bool PAIR = FC == 1 && !A8;         // A loads of two stages
  constexpr int KB = A8 ? 128 : 64;             // bytes of an A row and stage
  constexpr int ARB = PAIR ? 128 : KB;          // bytes of an A row in LDS
  constexpr int A_BYTES = BM * ARB, B_BYTES = 16 * 1024, BS_BYTES = 1024;
  constexpr int AS_BYTES = FC == 1 ? 0 : BM * 4;        // fc2: A scales in the stage
  constexpr int AS4_BYTES = FC == 1 ? BM * 16 : 0;      // fc1: of four stages
  constexpr int STAGE = B_BYTES + AS_BYTES + BS_BYTES;
  constexpr int B_AT = 2 * A_BYTES, AS4_AT = B_AT + 2 * STAGE;
  constexpr int NA = A_BYTES / 4096;            // a wavefront's 1 KB loads of an A slot
  __shared__ __attribute__((aligned(1024))) char lds[AS4_AT + 2 * AS4_BYTES];
  __shared__ int sched[8];
  TileInfo ti;
  if (!decode_ragged_m<BM, 4, 32>(args.offsets, args.E, NT, sched, ti)) return;
  const int lane = threadIdx.x & 63, g = lane >> 4, r = lane & 15;
  const int w = uniform((int)threadIdx.x >> 6);
  const int e = uniform(ti.e), row0 = uniform(ti.row0), rows = uniform(ti.rows);
  const int n0 = uniform(ti.n0) * BN;
  const int K = FC == 1 ? args.d : args.f, N = FC == 1 ? 2 * args.f : args.d;
  const int KT = K >> 7;

  // ---- sources: rows past the expert's end and columns past N read as zero.
  // A row: fc1 row-major, a slot is ARB bytes on; fc2 in panels
  const bool gather = FC == 1 && args.token_of != nullptr;
  const uint32_t a_rows = (uint32_t)(gather ? args.T : args.P);
  const uint32_t a_ld = FC == 1 ? (uint32_t)KT * KB : KB, as_ld = FC == 1 ? (uint32_t)KT * 4u : 4u;
  const uint32_t a_step = FC == 1 ? ARB : (uint32_t)args.P * KB, as_step = (uint32_t)args.P * 4u;
  const rsrc_t a_src = make_rsrc(args.a, a_rows * (uint32_t)KT * KB);
  const rsrc_t as_src = make_rsrc(args.as, a_rows * (uint32_t)KT * 4u);
  const int col = n0 + 64 * w;                  // this wavefront's 64 columns
  const uint32_t b_size = col < N ? 4096u * (uint32_t)KT : 0u;
  const int colc = min(col, N - 64);
  const rsrc_t b_src = make_rsrc(args.w + ((size_t)e * (N >> 4) + (size_t)(colc >> 4)) * KT * 1024, b_size);
  const rsrc_t bs_src = make_rsrc(args.ws + ((size_t)e * (N >> 6) + (size_t)(colc >> 6)) * KT * 256, b_size / 16);
  constexpr uint32_t kPast = 0x80000000u;       // past every range
  // offset of tile row m's source row; none for rows past the last and for a
  // token that there is not
  auto row_at = [&](int m, uint32_t ld, uint32_t at) __attribute__((always_inline)) -> uint32_t {
    const int pr = row0 + min(m, rows - 1);
    const uint32_t row = gather ? (uint32_t)args.token_of[pr] : (uint32_t)pr;
    return m < rows && row < a_rows ? row * ld + at : kPast;
  };
  uint32_t a_off[NA];
#pragma unroll
  for (int q = 0; q < NA; ++q) {
    const int t = w * NA + q;                   // load t: 1 KB of A rows
    const int m = ARB == 128 ? 8 * t + (lane >> 3) : 16 * t + (lane >> 2);
    const int c = ARB == 128 ? (lane & 7) ^ ((m >> 1) & 7) : (lane & 3) ^ ((m >> 1) & 3);
    a_off[q] = row_at(m, a_ld, (uint32_t)c * 16u);
  }
  // A scales.  fc1: the wavefront's 16 rows of either half of the tile, a lane
  // one of a row's four words; fc2: wavefronts 0 and 1, 64 rows each
  uint32_t as_off[FC == 1 ? 2 : 1];
#pragma unroll
  for (int q = 0; q < (FC == 1 ? 2 : 1); ++q) {
    const int m = FC == 1 ? 64 * q + 16 * w + (lane >> 2) : 64 * (w & 1) + lane;
    as_off[q] = row_at(m, as_ld, FC == 1 ? (uint32_t)(lane & 3) * 4u : 0u);
  }
  const uint32_t lane16 = (uint32_t)lane * 16u, lane4 = (uint32_t)lane * 4u;
  const uint32_t lds_base = (uint32_t)uniform((int)(uint32_t)(size_t)LDS_PTR(lds));

  // Loads of stage s (slot s & 1); past the last stage nothing is read and
  // zeros land.
  auto src = [&](rsrc_t v, bool live) __attribute__((always_inline)) {
    v[2] = live ? v[2] : 0;
    return uniform_rsrc(v);
  };
  auto issue_bs = [&](int s, int slot) __attribute__((always_inline)) {
    const bool live = s < KT;
    dma4(src(bs_src, live), lane4, (uint32_t)(live ? s : 0) * 256u,
         lds_base + (uint32_t)(B_AT + slot * STAGE + B_BYTES + AS_BYTES + w * 256));
  };
  auto issue_b = [&](int s, int slot, int j) __attribute__((always_inline)) {
    const bool live = s < KT;
    dma16(src(b_src, live), lane16, (uint32_t)(j * KT + (live ? s : 0)) * 1024u,
          lds_base + (uint32_t)(B_AT + slot * STAGE + (4 * w + j) * 1024));
  };
  // load q of A slot content u: stage u, or (PAIR) stages 2 u and 2 u + 1.  The
  // pair of an odd last stage reaches past its row: the rows' own part of the
  // offset carries u, so that the range check sees the sum.
  auto issue_a = [&](int u, int slot, int q) __attribute__((always_inline)) {
    const bool live = (PAIR ? 2 * u : u) < KT;
    const uint32_t dst = lds_base + (uint32_t)(slot * A_BYTES + (w * NA + q) * 1024);
    if constexpr (PAIR) dma16(src(a_src, live), a_off[q] + (uint32_t)u * a_step, dst);
    else dma16(src(a_src, live), a_off[q], (uint32_t)(live ? u : 0) * a_step, dst);
  };
  // fc1: half `half` of the A scales of stages 4 grp .. 4 grp + 3 (words past a
  // row's end are not used)
  auto issue_as4 = [&](int grp, int half) __attribute__((always_inline)) {
    dma4(as_src, (half ? as_off[FC == 1 ? 1 : 0] : as_off[0]) + (uint32_t)grp * 16u,
         lds_base + (uint32_t)(AS4_AT + (grp & 1) * AS4_BYTES + (64 * half + 16 * w) * 16));
  };
  // A scales loaded during stage kt: fc1, half of the next four stages' in the
  // first two of four; fc2, stage kt + 2's.  Who has none to load repeats its B
  // scales, so that all wavefronts issue as many loads.
  // (Without a branch: one would split the stage, and the compiler then sinks
  // the products in front of it past the barrier, with all their operands live.)
  auto issue_as = [&](int kt, int slot) __attribute__((always_inline)) {
    const bool live = kt + 2 < KT;
    const int sc = live ? kt + 2 : 0;
    const uint32_t bs_dst = lds_base + (uint32_t)(B_AT + slot * STAGE + B_BYTES + AS_BYTES + w * 256);
    const bool as = FC == 1 ? (kt & 3) < 2 : w < 2;
    rsrc_t v = pick(as, as_src, bs_src);
    uint32_t dst, off;
    if constexpr (FC == 1) {
      const int grp = (kt >> 2) + 1, half = kt & 1;
      v[2] = as || live ? v[2] : 0;
      off = as ? (half ? as_off[FC == 1 ? 1 : 0] : as_off[0]) + (uint32_t)grp * 16u : lane4 + (uint32_t)sc * 256u;
      dst = as ? lds_base + (uint32_t)(AS4_AT + (grp & 1) * AS4_BYTES + (64 * half + 16 * w) * 16) : bs_dst;
    } else {
      v[2] = live ? v[2] : 0;
      off = as ? as_off[0] + (uint32_t)sc * as_step : lane4 + (uint32_t)sc * 256u;
      dst = as ? lds_base + (uint32_t)(B_AT + slot * STAGE + B_BYTES + w * 256) : bs_dst;
    }
    dma4(uniform_rsrc(v), off, (uint32_t)uniform((int)dst));
  };

  // ---- fragments of stage s
  const uint32_t sw = (uint32_t)(r >> 1) & (ARB == 128 ? 7u : 3u);
  const uint32_t a_lo = (uint32_t)r * ARB + (((uint32_t)g ^ sw) << 4);
  const uint32_t a_hi = (uint32_t)r * ARB + (((uint32_t)(4 + g) ^ sw) << 4);
  auto ld16 = [&](const char* p) __attribute__((always_inline)) -> i32x4_t {
    return *(const __attribute__((address_space(3))) i32x4_t*)p;
  };
  // par = s & 1 (a constant); s itself for what is kept longer than two stages
  auto read_a = [&](int s, auto PAR, int i) __attribute__((always_inline)) -> typename Frag<A8>::type {
    constexpr int par = decltype(PAR)::value;
    if constexpr (A8) {
      const char* st = lds + par * A_BYTES + i * 16 * ARB;
      return __builtin_shufflevector(ld16(st + a_lo), ld16(st + a_hi), 0, 1, 2, 3, 4, 5, 6, 7);
    } else if constexpr (PAIR) {
      return ld16(lds + ((s >> 1) & 1) * A_BYTES + i * 16 * ARB + (par ? a_hi : a_lo));
    } else {
      return ld16(lds + par * A_BYTES + i * 16 * ARB + a_lo);
    }
  };
  auto read_as = [&](int s, auto PAR, int i) __attribute__((always_inline)) -> int {
    constexpr int par = decltype(PAR)::value;
    const char* p = FC == 1 ? lds + AS4_AT + ((s >> 2) & 1) * AS4_BYTES + (16 * i + r) * 16 + (s & 3) * 4 + g
                            : lds + B_AT + par * STAGE + B_BYTES + (16 * i + r) * 4 + g;
    return *(const __attribute__((address_space(3))) uint8_t*)p;
  };
  auto read_b = [&](auto PAR, int j) __attribute__((always_inline)) -> i32x4_t {
    constexpr int par = decltype(PAR)::value;
    return ld16(lds + B_AT + par * STAGE + (4 * w + j) * 1024 + lane * 16);
  };
  auto read_bs = [&](auto PAR) __attribute__((always_inline)) -> int {
    constexpr int par = decltype(PAR)::value;
    return *(const __attribute__((address_space(3))) int*)(lds + B_AT + par * STAGE + B_BYTES + AS_BYTES +
                                                          w * 256 + lane * 4);
  };

  f32x4_t acc[FM][4];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  // both slots, in the order and number in which the stages issue them (PAIR: the
  // B scales of stage 1 twice, in the place of the load that a stage issues after
  // them: the waits count it)
  if constexpr (FC == 1) {
    issue_as4(0, 0);
    issue_as4(0, 1);
  }
  static_for<0, 2>([&](auto S) __attribute__((always_inline)) {
    static_for<0, 4>([&](auto J) __attribute__((always_inline)) { issue_b(S.value, S.value, J.value); });
    issue_bs(S.value, S.value);
    if constexpr (FC == 2) issue_as(S.value - 2, S.value);
    if constexpr (PAIR && S.value == 1) issue_bs(S.value, S.value);
    static_for<0, NA>([&](auto Q) __attribute__((always_inline)) { issue_a(S.value, S.value, Q.value); });
  });
  constexpr int OWN = 5;                        // a stage's loads before the barrier
  wait_vmcnt<OWN + NA + (FC == 2 || PAIR ? 1 : 0)>();
  block_barrier();

  typename Frag<A8>::type xf[4];                // A fragments in flight: i & 3
  int sx[4];
  // a B fragment is replaced by the next stage's after its last product
  i32x4_t wf[4];
  int wsc;
  static_for<0, 4>([&](auto J) __attribute__((always_inline)) { wf[J.value] = read_b(IntC<0>{}, J.value); });
  wsc = read_bs(IntC<0>{});
  static_for<0, 2>([&](auto I) __attribute__((always_inline)) {
    xf[I.value] = read_a(0, IntC<0>{}, I.value);
    sx[I.value] = read_as(0, IntC<0>{}, I.value);
  });
  const int nfr = min(FM, (rows + 15) >> 4);    // fragments with rows
  constexpr int BAR = 5;                        // the barrier follows step BAR
  auto stage = [&](int kt, auto PAR, auto SKIP) __attribute__((always_inline)) {
    constexpr int p = decltype(PAR)::value;
    constexpr bool skip = decltype(SKIP)::value;
    constexpr IntC<1 - p> NEXT{};
    static_for<0, FM>([&](auto I) __attribute__((always_inline)) {
      constexpr int i = I.value;
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (i >= 1 && i < BAR) issue_b(kt + 2, p, i - 1);
      if constexpr (i == BAR) issue_bs(kt + 2, p);
      if constexpr (i > BAR) {
        // shared loads: the A scales, then A (PAIR: the pair after next, in the
        // second stage of a pair)
        if constexpr (i == BAR + 1) issue_as(kt, p);
        if constexpr (!PAIR || p == 1) {
          constexpr int q0 = (i - BAR - 1) * NA / 2, q1 = (i - BAR) * NA / 2;
          static_for<q0, q1>([&](auto Q) __attribute__((always_inline)) {
            issue_a(PAIR ? (kt >> 1) + 2 : kt + 2, PAIR ? (kt >> 1) & 1 : p, Q.value);
          });
        }
      }
      if constexpr (i + 2 < FM) {
        if (!skip || i + 2 < nfr) {
          xf[(i + 2) & 3] = read_a(kt, PAR, i + 2);
          sx[(i + 2) & 3] = read_as(kt, PAR, i + 2);
        }
      } else {
        xf[(i + 2) & 3] = read_a(kt + 1, NEXT, i + 2 - FM);
        sx[(i + 2) & 3] = read_as(kt + 1, NEXT, i + 2 - FM);
      }
      __builtin_amdgcn_sched_barrier(0);
      if (!skip || i < nfr) {
        static_for<0, 4>([&](auto J) __attribute__((always_inline)) {
          acc[i][J.value] = mma<A8, J.value>(wf[J.value], xf[i & 3], acc[i][J.value], wsc, sx[i & 3]);
          if constexpr (i == FM - 1 && !skip) {
            __builtin_amdgcn_sched_barrier(0);
            wf[J.value] = read_b(NEXT, J.value);
          }
        });
      }
      // The products stay in their step: without a use here the compiler sinks
      // them to the end of the stage, past the barrier, with every fragment live.
      stay(acc[i]);
      if constexpr (i == FM - 1) {
        if constexpr (skip)
          static_for<0, 4>([&](auto J) __attribute__((always_inline)) { wf[J.value] = read_b(NEXT, J.value); });
        wsc = read_bs(NEXT);
      }
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (i == BAR) {
        __builtin_amdgcn_s_waitcnt(0xc07f);     // lgkmcnt(0): this stage's reads are in registers
        // stage kt + 1 has landed for this wavefront: newer than its B loads are
        // the shared loads issued in stage kt - 1 and this stage's B loads; its A
        // loads (not PAIR, or the next pair's when p is 1) are the last of those
        if constexpr (PAIR && p == 0) wait_vmcnt<OWN + 1 + NA>();
        else if constexpr (PAIR) wait_vmcnt<OWN + 1>();
        else wait_vmcnt<OWN>();
        block_barrier();
      }
    });
  };
  auto run = [&](auto SKIP) __attribute__((always_inline)) {
    int kt = 0;
    for (; kt + 1 < KT; kt += 2) {
      stage(kt, IntC<0>{}, SKIP);
      stage(kt + 1, IntC<1>{}, SKIP);
    }
    if (kt < KT) stage(kt, IntC<0>{}, SKIP);
  };
  if (nfr == FM) run(IntC<0>{});
  else run(IntC<1>{});
  wait_vmcnt<0>();  // no LDS write may be in flight when the block ends

  if (col >= N) return;
  static_for<0, FM>([&](auto I) __attribute__((always_inline)) {
    constexpr int i = I.value;
    const int m = 16 * i + r;
    const size_t row = (size_t)(row0 + m);
    if constexpr (FC == 1) store_h<A8>(acc[i], m < rows, row, col >> 1, (size_t)args.P, lane, args.hq, args.hs);
    else store_o(acc[i], m < rows, row, col, args.d, lane, (bf16_t*)args.o);
  });
}

template <int FC, bool A8>
int launch_tiles(const Mx4Args& a, hipStream_t s) {
  const int64_t NT = ((FC == 1 ? 2 * (int64_t)a.f : (int64_t)a.d) + 255) / 256;
  // at most sum_e ceil(m_e / 128) row tiles; a block past the device-side count ends at once
  const int64_t grid = ((int64_t)a.P / 128 + a.E) * NT;
  if (!launch_fits(grid, 256)) return MOE_ERR_UNSUPPORTED;
  gemm_mx4_tile_kernel<FC, A8><<<(unsigned)grid, 256, 0, s>>>(a, (int)NT);
  TRE_LAUNCH_CHECK();
  return MOE_OK;
}

}  // namespace

// Which kernel: the rows kernel reads a column group's weights once per 32 rows of
// an expert and wins while they are read once or hardly more.  Calls with their
// quantiser, E2M1 and E4M3 rows, against the tile kernel, us: 128 experts, d 4096,
// f 1536: 16 rows an expert 229 and 250 against 243 and 245, 20 rows 239 and 265
// against 244 and 249, 24 rows 254 and 284 against 251 and 257; 8 experts, f 14336:
// 16 rows 127 and 139 against 170 and 177, 32 rows 193 and 224 against 173 and 185
// (at 24 rows, hardly an expert with a second piece, it would still win: 132 and
// 149 against 170 and 178).
// It also wins while the latency of a block's K steps counts, of which it has a
// quarter: while its blocks (pieces of 32 rows, an expert's last one half full on
// average, times groups of 64 columns), in rounds of two to a compute unit, each
// weighted with K, come to 1.5 rounds.  4 experts, d 384, f 2560: 97 rows an
// expert (1.16 rounds) 19 and 24 against 30 and 36 us, 300 rows (1.67) 30 and 40
// against 29 and 34 us; 8 experts, d = f = 1024: 64 rows (1.12) 19 and 22 against
// 24 and 28 us, 256 rows (3.19) 36 and 46 against 26 and 31 us.
bool gemm_mx4_few_rows(const Mx4Args& a) {
  if ((int64_t)a.P <= 20 * (int64_t)a.E) return true;
  const double pieces = a.P / 32.0 + 0.5 * (a.P < a.E ? a.P : a.E);
  auto steps = [&](int64_t n, int64_t k) {
    const double rounds = pieces * (double)(n / 64) / 512.0;
    return (rounds > 1.0 ? rounds : 1.0) * (double)k;
  };
  return steps(2 * (int64_t)a.f, a.d) + steps(a.d, a.f) <= 1.5 * ((double)a.d + (double)a.f);
}

int gemm_mx4_launch(int fc, bool a8, const Mx4Args& a, hipStream_t s) {
  if (!gemm_mx4_few_rows(a)) {
    if (fc == 1) return a8 ? launch_tiles<1, true>(a, s) : launch_tiles<1, false>(a, s);
    return a8 ? launch_tiles<2, true>(a, s) : launch_tiles<2, false>(a, s);
  }
  if (fc == 1) return a8 ? launch_rows<1, true>(a, s) : launch_rows<1, false>(a, s);
  return a8 ? launch_rows<2, true>(a, s) : launch_rows<2, false>(a, s);
}

}  // namespace tre
