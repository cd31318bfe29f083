// The experts' forward with 4-bit integer weights in scaled groups (i4.h) and bf16
// activations:
//
//   fc1:  [a | b] = x W13,  h = silu(a) b, rounded to bf16 in the epilogue
//   fc2:  o = h W2
//
// on v_mfma_f32_16x16x32_bf16 (many rows: 32x32x16), fp32 accumulation.  The weights
// are the first operand (rows of D = C^T: four consecutive output columns per lane),
// decoded to bf16 in registers: a lane's 16 bytes of a 128-row tile are its operands
// of four products.  W13 holds W1's and W3's 16-column groups alternately, so a lane
// holds a and b of the same element.  h is rounded to bf16 because fc2's instructions
// read it so, and the bf16 layers store it so: one rounding of the fp32 product.
#include "gemm_common.h"
#include "i4.h"

namespace tre {

namespace {
using namespace gemm;

typedef int i32x2_t __attribute__((ext_vector_type(2)));
typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));

__device__ __forceinline__ f32x4_t mma(const bf16x8_t& w, const bf16x8_t& x, const f32x4_t& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, x, c, 0, 0, 0);
}

// Epilogue of fc1 for one 16-row fragment: acc = [a0 b0 ..] (16 columns of f each; lane
// l: row l & 15, columns 4 (l >> 4)..+3) -> h of the 8 CF columns from col on.
template <int CF>
__device__ __forceinline__ void store_h(const f32x4_t (&acc)[CF], bool ok, size_t row, int col, int f, int lane,
                                        bf16_t* h) {
  f32x4_t v[CF / 2];
#pragma unroll
  for (int i = 0; i < CF / 2; ++i)
#pragma unroll
    for (int q = 0; q < 4; ++q) v[i][q] = silu_f32(acc[2 * i][q]) * acc[2 * i + 1][q];
  bf16_t* p = h + row * (size_t)f + col;
  if constexpr (CF == 4) {
    const u32x4_t x = pair_bf16(v[0], v[1]);
    if (ok) *(u32x4_t*)(p + ((lane >> 4) & 1) * 16 + (lane >> 5) * 8) = x;
  } else {
    if (ok) *(uint2*)(p + (lane >> 4) * 4) = make_uint2(pack_bf16x2(v[0][0], v[0][1]), pack_bf16x2(v[0][2], v[0][3]));
  }
}

// Epilogue of fc2 for one 16-row fragment: 16 CF columns from col on.
template <int CF>
__device__ __forceinline__ void store_o(const f32x4_t (&acc)[CF], bool ok, size_t row, int col, int d, int lane,
                                        bf16_t* o) {
  bf16_t* p = o + row * (size_t)d + col + ((lane >> 4) & 1) * 16 + (lane >> 5) * 8;
#pragma unroll
  for (int i = 0; i < CF / 2; ++i) {
    const u32x4_t v = pair_bf16(acc[2 * i], acc[2 * i + 1]);
    if (ok) *(u32x4_t*)(p + 32 * i) = v;
  }
}

// 16 bytes a lane at byte offset voff + soff (soff uniform); zeros past the end.
__device__ __forceinline__ i32x4_t load16(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t soff) {
  return __builtin_bit_cast(i32x4_t, __builtin_amdgcn_raw_buffer_load_b128(r, voff, soff, 0));
}
// The same for what is read once (non-temporal).
__device__ __forceinline__ i32x4_t load16_once(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t soff) {
  return __builtin_bit_cast(i32x4_t, __builtin_amdgcn_raw_buffer_load_b128(r, voff, soff, 2));
}
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const void* p, uint32_t bytes) {
  const uint64_t a = (uint64_t)p;
  const uint32_t lo = (uint32_t)uniform((int)(uint32_t)a), hi = (uint32_t)uniform((int)(uint32_t)(a >> 32));
  return __builtin_amdgcn_make_buffer_rsrc((void*)((uint64_t)hi << 32 | lo), 0, (int)bytes, 0x00020000);
}

// A lane's scale words of CF 16-column groups.
template <int CF>
struct Words {
  typedef i32x4_t type;
  static __device__ __forceinline__ type load(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t soff) {
    return load16(r, voff, soff);
  }
};
template <>
struct Words<2> {
  typedef i32x2_t type;
  static __device__ __forceinline__ type load(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t soff) {
    return __builtin_bit_cast(i32x2_t, __builtin_amdgcn_raw_buffer_load_b64(r, voff, soff, 0));
  }
};

// Few rows: a block of NW wavefronts takes CF 16-column groups of one expert and up to
// 32 of its rows; the wavefronts split K (wavefront w takes the 128-row steps w,
// w + NW, ...) and their partial sums meet in LDS, added in wavefront order.  Blocks
// take the pieces of 32 rows that the experts have, in order, so a call with few rows
// launches few blocks.  U: groups of a 128-row step.
//
// With up to 16 rows a step's operands are on their way while the step before it is
// decoded and multiplied (23 tokens of 8 of 128 experts, d 4096, f 1536: 212 -> 197
// us), and registers are kept to four wavefronts a SIMD (groups of 128: 197 -> 182 us)
// or three.  Reading the weights and decoding them take turns as the bound: without
// the decoding (19 instructions for 8 weights, 65 cycles of a SIMD for a wavefront's)
// the same call takes 152 us, 6.6 TB/s, with it 5.5; 177 tokens, groups of 64, 241 us
// against 274, 5.0 TB/s, of which reading x from L2 costs 14.
template <int FC, int U, int NW, int CF>
__global__ __launch_bounds__(NW * 64, U == 1 ? 4 : 3) void gemm_i4_rows_kernel(I4Args args) {
  __shared__ f32x4_t part[2][NW][CF][64];
  const int lane = threadIdx.x & 63, g = lane >> 4, r = lane & 15;
  const int w = uniform((int)threadIdx.x >> 6);
  const int K = FC == 1 ? args.d : args.f, N = FC == 1 ? 2 * args.f : args.d;
  const int KT = K >> 7, NB = N / (16 * CF);
  const int nb = (int)blockIdx.x % NB;
  // the piece: the (blockIdx / NB)-th of the experts' pieces of 32 rows, in order
  int e = -1, row0 = 0, rows = 0;
  {
    int want = (int)blockIdx.x / NB;
    int o0[4], o1[4];
    const __amdgpu_buffer_rsrc_t ob = buffer(args.offsets, 4u * (uint32_t)args.E + 4u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // (at most 256 experts; every load before the first use)
      o0[i] = (int)__builtin_amdgcn_raw_buffer_load_b32(ob, (uint32_t)(64 * i + lane) * 4u, 0, 0);
      o1[i] = (int)__builtin_amdgcn_raw_buffer_load_b32(ob, (uint32_t)(64 * i + lane) * 4u + 4u, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (e >= 0 || 64 * i >= args.E) break;
      const int n = 64 * i + lane < args.E ? (o1[i] - o0[i] + 31) >> 5 : 0;
      int end = n;  // pieces of this expert and of those before it
#pragma unroll
      for (int k = 1; k < 64; k *= 2) {
        const int v = __shfl_up(end, k, 64);
        end += lane >= k ? v : 0;
      }
      const uint64_t past = __ballot(end > want);
      if (past) {
        const int at = __builtin_ctzll(past);
        const int first = 32 * (want - __shfl(end - n, at, 64));
        e = 64 * i + at;
        row0 = __shfl(o0[i], at, 64) + first;
        rows = min(__shfl(o1[i], at, 64) - row0, 32);
      }
      want -= __shfl(end, 63, 64);
    }
  }
  e = uniform(e);
  if (e < 0) return;
  row0 = uniform(row0);
  rows = uniform(rows);
  const __amdgpu_buffer_rsrc_t wb = buffer(args.w + ((size_t)e * (N >> 4) + (size_t)nb * CF) * KT * 1024, 1024u * CF * (uint32_t)KT);
  const __amdgpu_buffer_rsrc_t sb = buffer(args.ws + ((size_t)e * (N >> 6) + nb * CF / 4) * KT * (U * 64), 256u * U * (uint32_t)KT);
  const bool gather = FC == 1 && args.token_of != nullptr;
  const uint32_t a_rows = (uint32_t)(gather ? args.T : args.P), a_ld = (uint32_t)K * 2u;
  const __amdgpu_buffer_rsrc_t ab = buffer(args.a, a_rows * a_ld);
  const uint32_t lane16 = (uint32_t)lane * 16u, r16 = (uint32_t)r * 16u + (CF == 2 ? (uint32_t)(nb & 1) * 8u : 0u);
  const uint32_t wstride = (uint32_t)KT * 1024u;  // from one 16-column group to the next
  // the rows as MT fragments of 16
  auto run = [&](auto MTC) __attribute__((always_inline)) {
    constexpr int MT = decltype(MTC)::value;
    f32x4_t acc[MT][CF];
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int j = 0; j < CF; ++j) acc[t][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    struct Step {
      i32x4_t wf[CF], xf[MT][4];
      typename Words<CF>::type sw[U];
    };
    auto load_w = [&](Step& o, int kt) __attribute__((always_inline)) {
#pragma unroll
      for (int j = 0; j < CF; ++j) o.wf[j] = load16_once(wb, lane16, (uint32_t)j * wstride + (uint32_t)kt * 1024u);
#pragma unroll
      for (int i = 0; i < U; ++i) o.sw[i] = Words<CF>::load(sb, r16, (uint32_t)(kt * U + i) * 256u);
    };
    // the first weights are on their way while the rows' token ids arrive
    uint32_t ids[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) ids[t] = gather ? (uint32_t)args.token_of[row0 + min(16 * t + r, rows - 1)] : 0u;
    Step a, b;
    load_w(a, min(w, KT - 1));
    // rows past the last read as zero, and so does a token that there is not
    uint32_t at[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      const int m = 16 * t + r;
      const uint32_t row = gather ? ids[t] : (uint32_t)(row0 + min(m, rows - 1));
      at[t] = m < rows && row < a_rows ? row * a_ld + (uint32_t)g * 16u : 0x80000000u;
    }
    auto load_x = [&](Step& o, int kt) __attribute__((always_inline)) {
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j) o.xf[t][j] = load16(ab, at[t] + (uint32_t)j * 64u, (uint32_t)kt * 256u);
    };
    auto load = [&](Step& o, int kt) __attribute__((always_inline)) {
      load_w(o, kt);
      load_x(o, kt);
    };
    auto multiply = [&](const Step& o) __attribute__((always_inline)) {
#pragma unroll
      for (int c = 0; c < CF; ++c) {
        float s = 0.f, nzs = 0.f;
        __builtin_amdgcn_sched_barrier(0);  // one column group's decoded weights at a time
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (j * U % 4 == 0) i4::unpack((uint32_t)o.sw[j * U / 4][c], s, nzs);
          const bf16x8_t wv = i4::operand((uint32_t)o.wf[c][j], s, nzs);
#pragma unroll
          for (int t = 0; t < MT; ++t) acc[t][c] = mma(wv, __builtin_bit_cast(bf16x8_t, o.xf[t][j]), acc[t][c]);
        }
      }
    };
    if (w < KT) {
      load_x(a, w);
      if constexpr (MT == 1) {
        for (int kt = w;; kt += 2 * NW) {
          if (kt + NW < KT) load(b, kt + NW);
          multiply(a);
          if (kt + NW >= KT) break;
          if (kt + 2 * NW < KT) load(a, kt + 2 * NW);
          multiply(b);
          if (kt + 2 * NW >= KT) break;
        }
      } else {
        for (int kt = w;;) {
          multiply(a);
          if ((kt += NW) >= KT) break;
          load(a, kt);
        }
      }
    }
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int j = 0; j < CF; ++j) part[t][w][j][lane] = acc[t][j];
    __syncthreads();
    if (w >= MT) return;  // wavefront t stores rows 16 t ..
    f32x4_t sum[CF];
#pragma unroll
    for (int j = 0; j < CF; ++j) {
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
    if constexpr (FC == 1) store_h<CF>(sum, m < rows, row, nb * CF * 8, args.f, lane, args.h);
    else store_o<CF>(sum, m < rows, row, nb * CF * 16, args.d, lane, args.o);
  };
  if (rows <= 16) run(IntC<1>{});
  else run(IntC<2>{});
}

template <int FC, int U, int NW, int CF>
int launch_rows(const I4Args& a, hipStream_t s) {
  const int64_t NB = (FC == 1 ? 2 * (int64_t)a.f : (int64_t)a.d) / (16 * CF);
  // at most sum_e ceil(m_e / 32) pieces, P with fewer rows than experts
  const int64_t grid = NB * (a.P / 32 + (a.P < a.E ? a.P : a.E));
  if (!launch_fits(grid, NW * 64)) return MOE_ERR_UNSUPPORTED;
  gemm_i4_rows_kernel<FC, U, NW, CF><<<(unsigned)grid, NW * 64, 0, s>>>(a);
  TRE_LAUNCH_CHECK();
  return MOE_OK;
}

// D += W X for a block of 32 columns of W x 32 rows x 16 k.  Lane l: column / row l &
// 31, the eight k from 8 (l >> 5) on; D: row l & 31, column 8 (i >> 2) + 4 (l >> 5) +
// (i & 3) in register i.
__device__ __forceinline__ f32x16_t mma32(const u32x4_t& w, const bf16x8_t& x, const f32x16_t& c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, w), x, c, 0, 0, 0);
}
__device__ __forceinline__ void stay32(f32x16_t (&a)[2]) { asm volatile("" : "+v"(a[0]), "+v"(a[1])); }

// Four columns each of x (4 (l >> 5) on) and y (8 further on) -> eight consecutive ones
// as bf16, from column 8 (l >> 5) on.
__device__ __forceinline__ u32x4_t pair32(const f32x4_t& x, const f32x4_t& y) {
  const uint32_t x0 = pack_bf16x2(x[0], x[1]), x1 = pack_bf16x2(x[2], x[3]);
  const uint32_t y0 = pack_bf16x2(y[0], y[1]), y1 = pack_bf16x2(y[2], y[3]);
  const auto a = __builtin_amdgcn_permlane32_swap(x0, y0, false, false);
  const auto b = __builtin_amdgcn_permlane32_swap(x1, y1, false, false);
  return u32x4_t{(uint32_t)a[0], (uint32_t)b[0], (uint32_t)a[1], (uint32_t)b[1]};
}
template <int Q>
__device__ __forceinline__ f32x4_t quad(const f32x16_t& a) {
  return f32x4_t{a[4 * Q], a[4 * Q + 1], a[4 * Q + 2], a[4 * Q + 3]};
}

// Many rows per expert: tiles of 128 rows x 256 stored columns, four wavefronts side
// by side (each all 128 rows x 64 columns as 4 x 2 fragments of 32 x 32), two blocks
// to a compute unit, so that one block's prologue, epilogue and barrier waits run under
// the other's products.  A wavefront decodes its own 64 columns, one step of 32 k
// ahead of the products that take them, between those products: 19 vector
// instructions for 8 weights a lane, 76 a step of 16 products.
//
// Bound by the matrix unit with that decoding beside it: 8192 tokens through 8 of 128
// experts (d 4096, f 1536) take 2.23 ms, 1.11 PFLOP/s; the same without decoding 1.91,
// with half of it 1.99.  Loads that all hit take 2-3 % off, fragments read further
// ahead nothing; a wavefront tile of 256 rows, which would decode half as often,
// spills (3.1 ms), and decoded weights shared through LDS would be bound by its
// bandwidth.  Where there are too few tiles for the chip, blockIdx.y takes parts of K
// and gemm_i4_join_kernel adds them.
//
// A (activations): stages of 64 k through three LDS slots, 128 rows of 128 bytes, the
// 16-byte chunk c of row r stored at chunk c ^ ((r >> 1) & 7), which spreads the rows
// of a fragment read over all banks.  B: 128 k (two stages, four steps) as stored, 4
// KB of codes and 256 bytes of scales for each group of a wavefront's 64 columns; only
// that wavefront reads them, into registers half by half, so one slot is enough and no
// barrier guards it.  Every byte arrives by buffer_load ... lds.  One barrier a stage:
// it follows the stage's last fragment read, so the slot that the loads of the stage
// after next go to (issued in the next stage) is free.
template <int FC, int U>
__global__ __launch_bounds__(256, 2) void gemm_i4_tile_kernel(I4Args args, int NT) {
  constexpr int BM = 128, BN = 256, FM = BM / 32, SUB = 2 * FM;   // a step: two halves of 16 k, FM fragments each
  constexpr int A_BYTES = BM * 128, BW = 4096 + U * 256;   // an A slot; a wavefront's part of B
  constexpr int B_AT = 3 * A_BYTES;
  constexpr int NA = A_BYTES / 4096, NBL = 4 + U;          // a wavefront's loads of a stage's A and of B
  __shared__ __attribute__((aligned(1024))) char lds[B_AT + 4 * BW];
  __shared__ int sched[8];
  TileInfo ti;
  if (!decode_ragged_m<BM, 4, 32>(args.offsets, args.E, NT, sched, ti)) return;
  const int lane = threadIdx.x & 63, kg = lane >> 5, r = lane & 31;
  const int w = uniform((int)threadIdx.x >> 6);
  const int e = uniform(ti.e), row0 = uniform(ti.row0), rows = uniform(ti.rows);
  const int n0 = uniform(ti.n0) * BN;
  const int K = FC == 1 ? args.d : args.f, N = FC == 1 ? 2 * args.f : args.d;
  const int KT = K >> 7;
  // this block's part of K, in 128 k
  const int P0 = KT * (int)blockIdx.y / (int)gridDim.y, P1 = KT * ((int)blockIdx.y + 1) / (int)gridDim.y;

  // ---- sources: rows past the expert's end and columns past N read as zero
  const bool gather = FC == 1 && args.token_of != nullptr;
  const uint32_t a_rows = (uint32_t)(gather ? args.T : args.P), a_ld = (uint32_t)K * 2u;
  const rsrc_t a_src = make_rsrc(args.a, a_rows * a_ld);
  const int col = n0 + 64 * w;                  // this wavefront's 64 columns
  const uint32_t b_size = col < N ? 4096u * (uint32_t)KT : 0u;
  const int colc = min(col, N - 64);
  const rsrc_t b_src = make_rsrc(args.w + ((size_t)e * (N >> 4) + (size_t)(colc >> 4)) * KT * 1024, b_size);
  const rsrc_t bs_src = make_rsrc(args.ws + ((size_t)e * (N >> 6) + (size_t)(colc >> 6)) * KT * (U * 64), b_size / 16 * U);
  constexpr uint32_t kPast = 0x80000000u;       // past every range
  uint32_t a_off[NA];
#pragma unroll
  for (int q = 0; q < NA; ++q) {
    const int m = 8 * (w * NA + q) + (lane >> 3);   // a load: 8 rows
    const int c = (lane & 7) ^ ((m >> 1) & 7);
    const int pr = row0 + min(m, rows - 1);
    const uint32_t row = gather ? (uint32_t)args.token_of[pr] : (uint32_t)pr;
    a_off[q] = m < rows && row < a_rows ? row * a_ld + (uint32_t)c * 16u : kPast;
  }
  const uint32_t lane16 = (uint32_t)lane * 16u, lane4 = (uint32_t)lane * 4u;
  const uint32_t lds_base = (uint32_t)uniform((int)(uint32_t)(size_t)LDS_PTR(lds));
  const uint32_t b_dst = lds_base + (uint32_t)(B_AT + w * BW);

  // Loads; past the last stage nothing is read and zeros land.
  auto src = [&](rsrc_t v, bool live) __attribute__((always_inline)) {
    v[2] = live ? v[2] : 0;
    return uniform_rsrc(v);
  };
  auto issue_a = [&](int kt, int slot, int q) __attribute__((always_inline)) {
    const bool live = kt < 2 * P1;
    dma16(src(a_src, live), a_off[q], (uint32_t)(live ? kt : 0) * 128u,
          lds_base + (uint32_t)(slot * A_BYTES + (w * NA + q) * 1024));
  };
  auto issue_b = [&](int P, int j) __attribute__((always_inline)) {
    const bool live = P < P1;
    dma16(src(b_src, live), lane16, (uint32_t)(j * KT + (live ? P : 0)) * 1024u, b_dst + (uint32_t)(j * 1024));
  };
  auto issue_bs = [&](int P, int u) __attribute__((always_inline)) {
    const bool live = P < P1;
    dma4(src(bs_src, live), lane4, (uint32_t)((live ? P : 0) * U + u) * 256u, b_dst + (uint32_t)(4096 + u * 256));
  };

  // ---- fragments.  A: half m of 16 k of the stage's four, fragment i of 32 rows
  const uint32_t sw = (uint32_t)(r >> 1) & 7u;
  uint32_t a_at[4];
#pragma unroll
  for (int m = 0; m < 4; ++m) a_at[m] = (uint32_t)r * 128u + (((uint32_t)(2 * m + kg) ^ sw) << 4);
  auto read_a = [&](int slot, auto M, int i) __attribute__((always_inline)) -> bf16x8_t {
    return *(const __attribute__((address_space(3))) bf16x8_t*)(lds + (uint32_t)slot * A_BYTES + a_at[decltype(M)::value] +
                                                                 i * 4096);
  };
  // B: 64 k of the wavefront's weights as stored: half HB of the slot's 128 k, and the
  // scale words of the groups that start there.  Fragment F has the 16-column tiles 2 F
  // and 2 F + 1 (lane bit 4); the k of a lane's half m lie in row group 2 m + kg of them.
  constexpr int UH = U == 4 ? 2 : 1;
  i32x2_t raw[2][2];
  uint32_t words[UH][2];
  const char* const b_codes = lds + B_AT + w * BW + ((lane >> 4) & 1) * 1024 + (16 * kg + (lane & 15)) * 16;
  const char* const b_words = lds + B_AT + w * BW + 4096 + (lane & 15) * 16 + ((lane >> 4) & 1) * 4;
  auto read_b = [&](auto HB) __attribute__((always_inline)) {
    constexpr int hb = decltype(HB)::value;
    if constexpr (hb == 0 || U > 1)
      static_for<0, 2 * UH>([&](auto I) __attribute__((always_inline)) {
        constexpr int u = I.value / 2, f = I.value % 2;
        words[u][f] = *(const __attribute__((address_space(3))) uint32_t*)(b_words + (hb * (U / 2) + u) * 256 + f * 8);
      });
    static_for<0, 4>([&](auto J) __attribute__((always_inline)) {
      constexpr int f = J.value / 2, m = J.value % 2;
      raw[f][m] = *(const __attribute__((address_space(3))) i32x2_t*)(b_codes + f * 2048 + m * 512 + hb * 8);
    });
  };
  float sc[2], nz[2];
  u32x4_t wd[2][2][2];                          // decoded: [step & 1][half][fragment]
  // piece X (of 8: fragment, half, 4 of a lane's 8 k) of step S
  auto decode = [&](auto S, auto X) __attribute__((always_inline)) {
    constexpr int s = decltype(S)::value, x = decltype(X)::value;
    constexpr int f = x >> 2, m = (x >> 1) & 1, p = x & 1;
    if constexpr ((x & 3) == 0 && s * U % 4 == 0) i4::unpack(words[U == 4 ? s & 1 : 0][f], sc[f], nz[f]);
    const uint32_t t = (uint32_t)raw[f][m][s & 1];
    float v[4];
    i4::values4((p ? t >> 4 : t) & 0x0f0f0f0fu, sc[f], nz[f], v);
    uint32_t a = pack_bf16x2(v[0], v[1]), b = pack_bf16x2(v[2], v[3]);
    asm volatile("" : "+v"(a), "+v"(b));        // decoded here, between these products
    wd[s & 1][m][f][2 * p] = a;
    wd[s & 1][m][f][2 * p + 1] = b;
  };

  f32x16_t acc[FM][2];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int f = 0; f < 2; ++f) acc[i][f] = f32x16_t{};
  static_for<0, 4>([&](auto J) __attribute__((always_inline)) { issue_b(P0, J.value); });
  static_for<0, U>([&](auto I) __attribute__((always_inline)) { issue_bs(P0, I.value); });
  static_for<0, 2>([&](auto S) __attribute__((always_inline)) {
    static_for<0, NA>([&](auto Q) __attribute__((always_inline)) { issue_a(2 * P0 + S.value, S.value, Q.value); });
  });
  wait_vmcnt<NA>();
  block_barrier();
  read_b(IntC<0>{});
  static_for<0, 8>([&](auto X) __attribute__((always_inline)) { decode(IntC<0>{}, X); });
  bf16x8_t xf[4];                               // A fragments in flight
  int slot = 0;                                 // of the current stage
  xf[0] = read_a(0, IntC<0>{}, 0);
  xf[1] = read_a(0, IntC<0>{}, 1);
  const int nfr = min(FM, (rows + 31) >> 5);    // fragments with rows

  // Step S (of 4) of the 128 k P: 32 k, half S & 1 of stage 2 P + S / 2.
  auto step = [&](int P, auto S, auto SKIP) __attribute__((always_inline)) {
    constexpr int s = decltype(S)::value, h = s & 1;
    constexpr bool skip = decltype(SKIP)::value;
    const int kt = 2 * P + (s >> 1);
    const int next = slot == 2 ? 0 : slot + 1, after = next == 2 ? 0 : next + 1;
    static_for<0, SUB>([&](auto I) __attribute__((always_inline)) {
      constexpr int x = I.value, m = x / FM, i = x % FM;
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (h == 0 && x >= 1 && x <= NA) issue_a(kt + 2, after, x - 1);
      // The second half of B's slot, then the next 128 k into it: its reads are in
      // registers, as the last products waited for a fragment read after them (where
      // products are skipped: an explicit wait).
      if constexpr (s == 1 && x == 0) read_b(IntC<1>{});
      if constexpr (s == 1 && x == 4) {
        if constexpr (skip) __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0)
        static_for<0, U>([&](auto Q) __attribute__((always_inline)) { issue_bs(P + 1, Q.value); });
        issue_b(P + 1, 0);
        issue_b(P + 1, 1);
      }
      if constexpr (s == 1 && x == 5) {
        issue_b(P + 1, 2);
        issue_b(P + 1, 3);
      }
      if constexpr (s == 3 && x == 0) {
        // the next 128 k of B have landed (and A's next stage, older): newer are this stage's A loads
        wait_vmcnt<NA>();
        asm volatile("" ::: "memory");
        read_b(IntC<0>{});
      }
      constexpr int y = x + 2, yi = y % FM;     // the fragment read ahead: of the stage's 4 FM, or the next one's
      constexpr int ym = (2 * h + y / FM) % 4;
      if constexpr (h == 1 && y >= SUB) xf[y & 3] = read_a(next, IntC<ym>{}, yi);
      else if (!skip || yi < nfr) xf[y & 3] = read_a(slot, IntC<ym>{}, yi);
      __builtin_amdgcn_sched_barrier(0);
      if (!skip || i < nfr) {
        static_for<0, 2>([&](auto F) __attribute__((always_inline)) {
          acc[i][F.value] = mma32(wd[h][m][F.value], xf[x & 3], acc[i][F.value]);
        });
      }
      // the next step's weights, a piece at a time (those that come out of the reads
      // above one place later)
      constexpr IntC<(s + 1) & 3> SN{};
      if constexpr (h == 0) {
        decode(SN, I);
      } else {
        if constexpr (x == 1) decode(SN, IntC<0>{});
        if constexpr (x >= 1) decode(SN, I);
      }
      stay32(acc[i]);
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (h == 1 && x == SUB - 3) {
        __builtin_amdgcn_s_waitcnt(0xc07f);     // lgkmcnt(0): this stage's reads are in registers
        // the next stage has landed: newer are the stage after next and, first stage, B
        if constexpr (s == 1) wait_vmcnt<NA + NBL>();
        block_barrier();
      }
    });
    if constexpr (h == 1) slot = next;
  };
  auto run = [&](auto SKIP) __attribute__((always_inline)) {
    for (int P = P0; P < P1; ++P)
      static_for<0, 4>([&](auto S) __attribute__((always_inline)) { step(P, S, SKIP); });
  };
  if (nfr == FM) run(IntC<0>{});
  else run(IntC<1>{});
  wait_vmcnt<0>();  // no LDS write may be in flight when the block ends

  if (col >= N) return;
  static_for<0, FM>([&](auto I) __attribute__((always_inline)) {
    constexpr int i = I.value;
    const int m = 32 * i + r;
    const size_t row = (size_t)(row0 + m);
    static_for<0, 2>([&](auto F) __attribute__((always_inline)) {
      constexpr int f = F.value;
      const f32x4_t q0 = quad<0>(acc[i][f]), q1 = quad<1>(acc[i][f]), q2 = quad<2>(acc[i][f]), q3 = quad<3>(acc[i][f]);
      if (gridDim.y > 1) {                      // sums over a part of K, as they are
        float* p = args.part + ((size_t)blockIdx.y * args.P + row) * (size_t)N + col + 32 * f + 4 * kg;
        if (m < rows) {
          *(f32x4_t*)p = q0;
          *(f32x4_t*)(p + 8) = q1;
          *(f32x4_t*)(p + 16) = q2;
          *(f32x4_t*)(p + 24) = q3;
        }
      } else if constexpr (FC == 1) {           // columns 0..15 of W1 and the same of W3
        f32x4_t h0, h1;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          h0[q] = silu_f32(q0[q]) * q2[q];
          h1[q] = silu_f32(q1[q]) * q3[q];
        }
        const u32x4_t v = pair32(h0, h1);
        if (m < rows) *(u32x4_t*)(args.h + row * (size_t)args.f + (col >> 1) + 16 * f + 8 * kg) = v;
      } else {
        const u32x4_t v0 = pair32(q0, q1), v1 = pair32(q2, q3);
        bf16_t* p = args.o + row * (size_t)args.d + col + 32 * f + 8 * kg;
        if (m < rows) {
          *(u32x4_t*)p = v0;
          *(u32x4_t*)(p + 16) = v1;
        }
      }
    });
  });
}

// The parts of K (fp32 [parts][P][N]) added in order, and the epilogue: a thread takes
// eight columns of h or o.  Rows outside the experts' are left as they were.
template <int FC>
__global__ __launch_bounds__(256) void gemm_i4_join_kernel(I4Args args, int parts) {
  const int C = FC == 1 ? args.f : args.d;
  const int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8, row = at / C;
  if (row < args.offsets[0] || row >= min(args.offsets[args.E], args.P)) return;
  const int64_t all = (int64_t)args.P * (FC == 1 ? 2 * C : C);
  auto sum8 = [&](const float* p, f32x4_t (&v)[2]) __attribute__((always_inline)) {
    v[0] = *(const f32x4_t*)p;
    v[1] = *(const f32x4_t*)(p + 4);
    for (int i = 1; i < parts; ++i) {
      v[0] += *(const f32x4_t*)(p + i * all);
      v[1] += *(const f32x4_t*)(p + i * all + 4);
    }
  };
  f32x4_t v[2];
  if constexpr (FC == 1) {                      // 16 columns of W1, then the same of W3
    const int c = (int)(at - row * C);
    const float* p = args.part + row * 2 * C + 2 * (c & ~15) + (c & 15);
    f32x4_t b[2];
    sum8(p, v);
    sum8(p + 16, b);
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q >> 2][q & 3] = silu_f32(v[q >> 2][q & 3]) * b[q >> 2][q & 3];
  } else {
    sum8(args.part + at, v);
  }
  *(u32x4_t*)((FC == 1 ? args.h : args.o) + at) =
      u32x4_t{pack_bf16x2(v[0][0], v[0][1]), pack_bf16x2(v[0][2], v[0][3]), pack_bf16x2(v[1][0], v[1][1]),
              pack_bf16x2(v[1][2], v[1][3])};
}

template <int FC, int U>
int launch_tiles(const I4Args& a, hipStream_t s) {
  const int64_t NT = ((FC == 1 ? 2 * (int64_t)a.f : (int64_t)a.d) + 255) / 256;
  // at most sum_e ceil(m_e / 128) row tiles; a block past the device-side count ends at once
  const int64_t grid = ((int64_t)a.P / 128 + a.E) * NT;
  const int parts = gemm_i4_parts(a, FC);
  if (!launch_fits(grid * parts, 256)) return MOE_ERR_UNSUPPORTED;
  gemm_i4_tile_kernel<FC, U><<<dim3((unsigned)grid, (unsigned)parts), 256, 0, s>>>(a, (int)NT);
  TRE_LAUNCH_CHECK();
  if (parts == 1) return MOE_OK;
  const int64_t n = (int64_t)a.P * (FC == 1 ? a.f : a.d) / 8;
  gemm_i4_join_kernel<FC><<<(unsigned)((n + 255) / 256), 256, 0, s>>>(a, parts);
  TRE_LAUNCH_CHECK();
  return MOE_OK;
}

// The blocks of the rows kernel: 64 columns and four wavefronts each where there are
// four of them for each of 256 compute units, else 32 columns, and eight wavefronts
// where those would be one to a compute unit.  64 columns, 32 columns, 32 columns with
// eight wavefronts, us, by the number of the first: 384 (8 experts, K 4096) 18.0,
// 15.6, 16.6; 896 (2 experts, K 4096) 29.2, 26.6, 30.6; 1024 (16, K 1536) 13.4, 15.0,
// 19.5; 128 (2, K 14336) 30.9, 21.6, 16.7; 64 (4, K 1024) 5.6, 4.8, 4.6.
template <int FC, int U>
int launch(const I4Args& a, hipStream_t s) {
  if (!gemm_i4_few_rows(a)) return launch_tiles<FC, U>(a, s);
  const int64_t blocks = (FC == 1 ? 2 * (int64_t)a.f : (int64_t)a.d) / 64 * (a.P / 32 + (a.P < a.E ? a.P : a.E));
  if (blocks >= 1024) return launch_rows<FC, U, 4, 4>(a, s);
  return blocks > 128 ? launch_rows<FC, U, 4, 2>(a, s) : launch_rows<FC, U, 8, 2>(a, s);
}
template <int FC>
int launch_fc(const I4Args& a, hipStream_t s) {
  if (a.group == 128) return launch<FC, 1>(a, s);
  if (a.group == 64) return launch<FC, 2>(a, s);
  return launch<FC, 4>(a, s);
}

}  // namespace

static int64_t stored_columns(const I4Args& a, int fc) { return fc == 1 ? 2 * (int64_t)a.f : a.d; }
static int64_t contraction(const I4Args& a, int fc) { return fc == 1 ? a.d : a.f; }

// Blocks of m rows x n columns of a product, as the host can tell: an expert has about
// 0.35 of them down its rows more than the rows fill, and one at least.
static double blocks_of(const I4Args& a, int fc, double m, double n) {
  const double experts = a.P < a.E ? a.P : a.E, have = a.P / experts / m + 0.35;
  return experts * (have > 1.0 ? have : 1.0) * ((double)stored_columns(a, fc) / n);
}

// The tiles' time, in k that a full chip of them (two blocks to each of 256 compute
// units) goes through, and the parts of K, one block each, that make it least: half a
// chip of blocks takes three quarters of a full one's time a step, and the parts' sums
// cost a launch and their way through memory.  One part against these, us, rows an
// expert: 8 experts, d 4096, f 14336: 36 rows 372 against 267 (four parts in fc2), 64:
// 413 / 315, 100: 447 / 361, 150: 562 / 550 (two), 259: 802 / 794; 1, d 2048, f 8192: 512
// rows 133 / 76 (two, four); 2, d 7168, f 2048: 200 rows 157 / 95; 4, d 384, f 2560: 400
// rows 58 / 38.
struct TileCost {
  int parts;
  double time;
};
// `room`: bytes for the parts' sums; where the best number does not fit, the best that does.
static TileCost tile_cost(const I4Args& a, int fc, size_t room) {
  const double K = (double)contraction(a, fc), tiles = blocks_of(a, fc, 128, 256);
  const double values = (double)a.P * (double)stored_columns(a, fc);
  TileCost best = {1, 0.0};
  for (int parts = 1; parts <= 4 && parts * 128 <= K; ++parts) {
    if (parts > 1 && (size_t)parts * (size_t)a.P * (size_t)stored_columns(a, fc) * 4 > room) break;
    const double r = tiles * parts / 512;
    const double time = (r < 1.0 ? 0.5 + 0.5 * r : r) * K / parts + (parts > 1 ? 160 + 1e-4 * values * parts : 0.0);
    if (parts == 1 || time < best.time) best = {parts, time};
  }
  return best;
}

int gemm_i4_parts(const I4Args& a, int fc) { return gemm_i4_few_rows(a) ? 1 : tile_cost(a, fc, a.part_bytes).parts; }

// Which kernel.  The rows kernel's time goes with the rounds of its pieces of 32 rows x
// 64 columns, three to a compute unit; a step of a chip of tiles takes three times as
// long as one of theirs.  Both kernels, us, rows an expert:
//   128 experts, d 4096, f 1536: 16 rows 298 against 386, 32: 467 / 415, 64: 808 / 508;
//   8, d 4096, f 14336: 16 rows 185 / 232, 20: 211 / 237, 28: 272 / 250, 64: 490 / 315;
//   8, d = f = 1024: 64 rows 22 / 41, 256: 40 / 38, 512: 72 / 42; 4, d 384, f 2560: 200
//   rows 32 / 34, 400: 47 / 38; 16, d 2048, f 8192: 24 rows 144 / 143, 32: 177 / 155; 32, d
//   2048, f 1408: 32 rows 72 / 75, 64: 107 / 84.
bool gemm_i4_few_rows(const I4Args& a) {
  double rows = 0, tiles = 0;
  for (int fc = 1; fc <= 2; ++fc) {
    const double r = blocks_of(a, fc, 32, 64) / 768;
    rows += (r > 0.35 ? r : 0.35) * (double)contraction(a, fc);
    tiles += tile_cost(a, fc, SIZE_MAX).time;  // (whatever this call's workspace: the choice is the shape's)
  }
  return rows <= 3.0 * tiles;
}

int gemm_i4_launch(int fc, const I4Args& a, hipStream_t s) {
  return fc == 1 ? launch_fc<1>(a, s) : launch_fc<2>(a, s);
}

}  // namespace tre
