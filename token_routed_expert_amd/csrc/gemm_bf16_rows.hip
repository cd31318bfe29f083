// Grouped expert GEMMs in bf16 for few rows per expert (the ragged-M products of
// gemm_bf16.hip: same operands, same epilogues, fp32 accumulation).
//
// With few rows a 256 x 256 tile is mostly padding, the tiles do not fill the
// chip, and each walks the whole contraction a K step of 32 at a time, bound by
// the latency of its loads (64 rows, d 384, f 3840, 4 experts: fc1's data
// gradient has 8 tiles of 240 steps).  A training step's products of 1028 rows,
// 16 experts, d 512, f 384 take 54 us with these kernels for the ragged-M ones
// (7-12 us each, a launch and a few K steps of latency), 93 us without.  Here a
// tile is 64 rows x 128 columns and K advances 128 a stage: 8 wavefronts in 4 K
// groups of 2, K group q taking columns 32 q .. 32 q + 31 of every stage for all
// 64 rows and one half of the tile's columns each.  The four partial sums meet in
// LDS, added in K-group order, and wavefront (q, half) applies the epilogue to
// rows 16 q .. + 15.
// Stages arrive by buffer_load ... lds, three slots of 48 KB, whole 128-byte
// lines throughout:
//  * K-contiguous operands: rows of 256 bytes; 16-byte chunk c of row r at chunk
//    c ^ (r & 15), so the 16 rows of a fragment read cover all banks;
//  * MN-contiguous operands (the forward weights): two halves of 64 columns (fc1:
//    W1's and W3's), each [128 k][128 bytes]; 32-byte unit u of k-row k at
//    u ^ swz(k), swz(k) = bit 1 of k | bit 3 of k << 1, which spreads the 16 k-rows
//    of a transposing read over all banks.
#include "gemm_common.h"

namespace tre {

namespace {
using namespace gemm;

constexpr int BM = 64, BN = 128, BK = 128, NS = 3;
constexpr int A_BYTES = BM * 256, B_BYTES = BN * 256, STAGE = A_BYTES + B_BYTES;
constexpr int NA = A_BYTES / 1024 / 8, NB = B_BYTES / 1024 / 8, LOADS = NA + NB;  // a wavefront's of a stage
constexpr uint32_t kPast = 0x80000000u;  // past every operand's range

__device__ __forceinline__ int swz(int k) { return ((k >> 1) & 1) | (((k >> 3) & 1) << 1); }

__device__ __forceinline__ bf16x8_t read16(const char* p) {
  return *(const __attribute__((address_space(3))) bf16x8_t*)p;
}
// k-rows kr .. kr + 3 and kr + 4 .. kr + 7 of 16 columns, transposed
__device__ __forceinline__ bf16x8_t read_tr(const char* p) {
  const i16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) i16x4_t*)p);
  const i16x4_t hi =
      __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) i16x4_t*)(p + 4 * 128));
  return __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

template <int OP, bool RS, bool CK>
__global__ __launch_bounds__(512, 1) void gemm_bf16_rows_kernel(GemmArgs args, int NT) {
  constexpr bool B_KC = OP == OP_FC2_DGRAD || OP == OP_FC1_DGRAD;  // B K-contiguous
  __shared__ __attribute__((aligned(1024))) char lds[NS * STAGE];
  __shared__ int sched[16];
  __shared__ float dp_red[2 * 256];
  TileInfo ti;
  if (!decode_ragged_m<BM, 8>(args.offsets, args.E, NT, sched, ti)) return;
  ti.e = uniform(ti.e);
  ti.row0 = uniform(ti.row0);
  ti.rows = uniform(ti.rows);
  ti.n0 = uniform(ti.n0) * BN;
  const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, sl = lane & 15;
  const int w = uniform(tid >> 6);
  const int kg = w >> 1, wn = w & 1;
  const int d = args.d, f = args.f;
  const int K = (OP == OP_FC1_FWD || OP == OP_FC2_DGRAD) ? d : (OP == OP_FC2_FWD ? f : 2 * f);
  const int N = OP == OP_FC1_FWD ? 2 * f : (OP == OP_FC2_DGRAD ? f : d);
  const int KT = K / BK;  // d and f are multiples of 128

  // ---- sources
  const bool gather = OP == OP_FC1_FWD && args.gather != nullptr;
  const uint32_t a_ld = (uint32_t)K * 2u;
  const void* a_base = OP == OP_FC1_FWD ? (gather ? args.gx : args.xp)
                                        : (OP == OP_FC2_FWD ? args.h : (OP == OP_FC2_DGRAD ? args.dO : args.dab));
  // (K = d for the gathered product, so a row of x is a_ld bytes too)
  const rsrc_t a_src = gather ? make_rsrc(a_base, (uint32_t)args.gT * a_ld)
                              : make_rsrc((const char*)a_base + (size_t)ti.row0 * a_ld, (uint32_t)ti.rows * a_ld);
  const size_t mat = (size_t)ti.e * (size_t)d * (size_t)f;
  const uint32_t b_size = (uint32_t)d * (uint32_t)f * 2u;
  const bool w2 = OP == OP_FC2_FWD || OP == OP_FC2_DGRAD;
  const rsrc_t b_src = make_rsrc((const bf16_t*)(w2 ? args.W2 : args.W1) + mat, b_size);
  const rsrc_t b_src2 = w2 ? b_src : make_rsrc((const bf16_t*)args.W3 + mat, b_size);
  // row length of the weights in bytes: W1, W3 [d][f], W2 [f][d]
  const uint32_t b_ld = (uint32_t)((OP == OP_FC1_FWD || OP == OP_FC1_DGRAD) ? f : d) * 2u;

  uint32_t a_off[NA], b_off[NB];
#pragma unroll
  for (int q = 0; q < NA; ++q) {
    const int m = 4 * (w * NA + q) + (lane >> 4);
    const int c = (lane & 15) ^ (m & 15);
    const int src_row = gather ? args.gather[ti.row0 + min(m, ti.rows - 1)] : m;
    // (a token that there is not reads as a row of zeros)
    const bool ok = m < ti.rows && (!gather || (uint32_t)src_row < (uint32_t)args.gT);
    a_off[q] = ok ? (uint32_t)src_row * a_ld + (uint32_t)c * 16u : kPast;
  }
#pragma unroll
  for (int q = 0; q < NB; ++q) {
    const int t = w * NB + q;  // 1 KB instruction of the B operand, 0 .. 31
    if constexpr (B_KC) {
      const int n = 4 * t + (lane >> 4);
      const int c = (lane & 15) ^ (n & 15);
      b_off[q] = ti.n0 + n < N ? (uint32_t)(ti.n0 + n) * b_ld + (uint32_t)c * 16u : kPast;
    } else {
      const int half = t >> 4, k = 8 * (t & 15) + (lane >> 3);
      const int unit = ((lane & 7) >> 1) ^ swz(k);
      const int col = (OP == OP_FC1_FWD ? ti.n0 / 2 : ti.n0 + 64 * half) + unit * 16 + (lane & 1) * 8;
      b_off[q] = (uint32_t)k * b_ld + (uint32_t)col * 2u;
    }
  }
  const uint32_t lds_base = (uint32_t)uniform((int)(uint32_t)(size_t)LDS_PTR(lds));
  // the loads of stage s into slot s % NS (past the last stage: nothing is read)
  auto issue = [&](int s) __attribute__((always_inline)) {
    const uint32_t base = lds_base + (uint32_t)(s % NS) * (uint32_t)STAGE;
    const bool live = s < KT;
    const int k0 = s * BK;
    static_for<0, NA>([&](auto Q) __attribute__((always_inline)) {
      rsrc_t v = a_src;
      v[2] = live ? v[2] : 0;
      dma16(uniform_rsrc(v), a_off[Q.value] + (uint32_t)k0 * 2u, base + (uint32_t)((w * NA + Q.value) * 1024));
    });
    static_for<0, NB>([&](auto Q) __attribute__((always_inline)) {
      const int t = w * NB + Q.value;
      rsrc_t v = b_src;
      uint32_t k = (uint32_t)k0;
      if constexpr (OP == OP_FC1_DGRAD) {  // K = [da | db]: the first f rows multiply W1, the rest W3
        const bool first = k0 < f;
        v = pick(first, b_src, b_src2);
        k = (uint32_t)(first ? k0 : k0 - f);
      }
      if constexpr (OP == OP_FC1_FWD) v = pick(t < 16, b_src, b_src2);
      v[2] = live ? v[2] : 0;
      dma16(uniform_rsrc(v), b_off[Q.value] + k * (B_KC ? 2u : b_ld),
            base + (uint32_t)(A_BYTES + t * 1024));
    });
  };

  // ---- fragment addresses inside a stage
  const uint32_t kc = (uint32_t)sl * 256u + (uint32_t)(((4 * kg + g) ^ sl) << 4);
  const int kr = 32 * kg + 8 * g + (sl >> 2);  // MN-contiguous: the lane's first k-row
  auto read_a = [&](const char* st, int i) __attribute__((always_inline)) -> bf16x8_t {
    return read16(st + i * 16 * 256 + kc);
  };
  auto read_b = [&](const char* st, int j) __attribute__((always_inline)) -> bf16x8_t {
    if constexpr (B_KC) {
      return read16(st + A_BYTES + (64 * wn + 16 * j) * 256 + kc);
    } else {
      const int half = OP == OP_FC1_FWD ? j >> 1 : wn;
      const int unit = OP == OP_FC1_FWD ? 2 * wn + (j & 1) : j;
      return read_tr(st + A_BYTES + half * 16384 + kr * 128 + ((unit ^ swz(kr)) << 5) + (sl & 3) * 8);
    }
  };

  f32x4_t acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  issue(0);
  issue(1);
  for (int kt = 0; kt < KT; ++kt) {
    wait_vmcnt<LOADS>();  // stage kt has landed for this wavefront, and with the barrier for all;
    block_barrier();      // every wavefront has stage kt - 1 in registers: its slot takes kt + 2
    issue(kt + 2);
    const char* st = lds + (kt % NS) * STAGE;
    bf16x8_t a[4], b[4];
    static_for<0, 4>([&](auto J) __attribute__((always_inline)) { b[J.value] = read_b(st, J.value); });
    static_for<0, 4>([&](auto I) __attribute__((always_inline)) { a[I.value] = read_a(st, I.value); });
    static_for<0, 4>([&](auto I) __attribute__((always_inline)) {
      static_for<0, 4>([&](auto J) __attribute__((always_inline)) {
        acc[I.value][J.value] =
            __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[J.value], a[I.value], acc[I.value][J.value], 0, 0, 0);
      });
      stay(acc[I.value]);
    });
  }
  wait_vmcnt<0>();  // no load may still be writing LDS
  block_barrier();

  // ---- the K groups' sums: wavefront (kg, wn) adds up fragment row kg of its half
  f32x4_t* const red = (f32x4_t*)lds;  // [kg][wn][fragment][lane]
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) red[(((kg * 2 + wn) * 16) + i * 4 + j) * 64 + lane] = acc[i][j];
  __syncthreads();
  f32x4_t sum[1][4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f32x4_t s = red[((wn * 16) + kg * 4 + j) * 64 + lane];
#pragma unroll
    for (int q = 1; q < 4; ++q) {
      const f32x4_t p = red[(((q * 2 + wn) * 16) + kg * 4 + j) * 64 + lane];
#pragma unroll
      for (int x = 0; x < 4; ++x) s[x] += p[x];
    }
    sum[0][j] = s;
  }
  store_tile<OP, 1, 4, 16, 64, true, RS, false, CK, BN>(args, sum, ti, ti.rows, N, kg, wn, lane, dp_red);
}

template <int OP, bool RS, bool CK>
int launch(const GemmArgs& a, hipStream_t s) {
  const int N = OP == OP_FC1_FWD ? 2 * a.f : (OP == OP_FC2_DGRAD ? a.f : a.d);
  const int64_t NT = (N + BN - 1) / BN;
  const int64_t grid = ((int64_t)a.P / BM + a.E) * NT;
  if (!launch_fits(grid, 512)) return MOE_ERR_UNSUPPORTED;
  gemm_bf16_rows_kernel<OP, RS, CK><<<(unsigned)grid, 512, 0, s>>>(a, (int)NT);
  TRE_LAUNCH_CHECK();
  return MOE_OK;
}

}  // namespace

int gemm_bf16_rows_launch(GemmOp op, const GemmArgs& a, hipStream_t s) {
  switch (op) {
    case OP_FC1_FWD: return launch<OP_FC1_FWD, true, true>(a, s);
    case OP_FC2_FWD: return launch<OP_FC2_FWD, false, false>(a, s);
    case OP_FC2_DGRAD: return launch<OP_FC2_DGRAD, true, true>(a, s);
    case OP_FC1_DGRAD: return launch<OP_FC1_DGRAD, false, false>(a, s);
    default: return MOE_ERR_INVALID;
  }
}

}  // namespace tre
