/*
 * moe.h -- C ABI of one GPU's routed-expert (mixture-of-experts) layer on
 * AMD Instinct MI355X (gfx950).
 *
 * Method: "Scalable Training of Mixture-of-Experts Models with Megatron Core"
 * (gist.science technical summaries).  The Spanish summary, section 2.1
 * ("Arquitectura de la capa MoE"), splits the layer into four steps: route
 * each token to its k best experts, dispatch the tokens to their experts,
 * run the experts as grouped GEMMs, combine the results.  On one GPU dispatch
 * and combine are a local permutation and a weighted un-permutation.
 *
 * Conventions for every call
 * --------------------------
 *  - All tensor pointers are DEVICE pointers, owned by the caller, row-major,
 *    16-byte aligned, and not aliased with each other unless stated.  The
 *    library never allocates or frees memory and keeps no state between
 *    calls, apart from the device array of moe_permute_noalloc (a fixed
 *    1 MiB per GPU, see there) and a per-device cache of the compute-unit
 *    count; scratch space is the caller's `ws` buffer of `ws_bytes` bytes
 *    (size from moe_workspace_bytes).
 *  - `stream` is a hipStream_t (NULL = the default stream).  Calls only
 *    enqueue work on it and return: no host synchronisation, no copy of
 *    per-expert counts to the host (the German summary, section 2 D, and the
 *    Spanish summary, section 2.3 C: kernels read shape information from GPU
 *    memory, so dropless routing needs no CPU-GPU sync).  Calls are safe to
 *    capture into a HIP graph.
 *  - Return value: a moe_status.  Arguments are validated before anything is
 *    enqueued; MOE_ERR_HIP reports a launch failure.  Faults inside kernels
 *    surface at the caller's next synchronisation.  Nothing aborts or prints.
 *  - Shapes: T tokens, d hidden size, E experts, k experts per token, f
 *    expert FFN width, P = T*k routed rows (dropless: every assignment gets a
 *    row, so permuted buffers always have exactly P rows -- the worst case is
 *    known on the host; cf. the hyper.ai article on Hybrid-EP, which reserves
 *    buffers for the worst case).  Limits: 1 <= k <= E <= 256, T >= 1,
 *    P < 2^31.  The bf16 expert GEMMs need d and f to be multiples of 128,
 *    and P * max(d, 2f) * 2 and d * f * 2 below 2^32 bytes (the shared
 *    expert: T in place of P, f_shared in place of f); outside that they
 *    return MOE_ERR_UNSUPPORTED.
 *  - Expert weights: W1, W3 are [E][d][f], W2 is [E][f][d]; expert e maps a
 *    row x to o = (silu(x W1_e) * (x W3_e)) W2_e with silu(z) = z / (1+e^-z).
 *  - Dtypes: MOE_F32 (every tensor fp32), MOE_BF16 (x, weights, outputs and
 *    saved activations bf16, fp32 accumulation, one round-to-nearest-even per
 *    output element) or MOE_E4M3 (the expert GEMMs take OCP E4M3FN operands
 *    with fp32 block scales -- see "e4m3 expert GEMMs" below -- while x, dY,
 *    y, dX, the saved activations and the weight gradients are bf16) or
 *    MOE_MXFP8 (the same with MXFP8 operands: E4M3FN codes with one
 *    power-of-two E8M0 scale byte per 32 values -- see "MXFP8 expert GEMMs"
 *    below).  MOE_MXFP4 and MOE_MXFP4_A8 run the forward alone, with 4-bit
 *    expert weights ("MXFP4 experts" below) and bf16 x and y; MOE_INT4 does with
 *    integer ones ("Integer expert weights" below).  Router
 *    logits and probabilities are always fp32 (German summary, section 2 E:
 *    the router stays in high precision).
 */
#ifndef TRE_MOE_H
#define TRE_MOE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  MOE_OK = 0,
  MOE_ERR_INVALID = 1,      /* null pointer, inconsistent or out-of-range sizes */
  MOE_ERR_UNSUPPORTED = 2,  /* valid but outside this build's limits (dtype, alignment, sizes
                               whose launch would need 2^32 threads or more) */
  MOE_ERR_WORKSPACE = 3,    /* ws_bytes smaller than moe_workspace_bytes() (or than the
                               least that a call names) */
  MOE_ERR_HIP = 4           /* a HIP runtime call or kernel launch failed */
} moe_status;

typedef enum {
  MOE_F32 = 0,
  MOE_BF16 = 1,
  MOE_E4M3 = 2,
  MOE_MXFP8 = 3,
  MOE_MXFP4 = 4,    /* forward only: MXFP4 weights and activations */
  MOE_MXFP4_A8 = 5, /* forward only: MXFP4 weights, MXFP8 activations */
  MOE_INT4 = 6      /* forward only: integer weights in scaled groups, bf16 activations */
} moe_dtype;

typedef struct {
  int64_t T, d, E, k, f;
  int64_t f_shared;  /* width of an always-on shared expert, 0 = none */
  int32_t dtype;     /* moe_dtype of x, weights, activations and outputs */
  int32_t reserved;  /* must be 0 */
} moe_shape;

/* Which call a workspace size is asked for. */
typedef enum {
  MOE_WS_PERMUTE = 0,
  MOE_WS_GEMM_FWD = 1,
  MOE_WS_GEMM_BWD = 2,
  MOE_WS_LAYER_FWD = 3,
  MOE_WS_LAYER_BWD = 4,
  MOE_WS_AUX_LOSS = 5,
  MOE_WS_GEMM_BWD_ROWSCALED = 6,
  MOE_WS_LAYER_BWD_ROWSCALED = 7,
  MOE_WS_NORM_BWD = 8,     /* moe_add_rms_norm_bwd: the shape's T and d count */
  MOE_WS_NORM_BWD_MAX = 9  /* the same, enough for every T up to the shape's */
} moe_ws_kind;

/*
 * moe_route -- top-k routing (Spanish summary, section 2.1: a router assigns
 * each token to its k best experts).
 *   logits    fp32 [T][E].
 *   topk_idx  out int32 [T][k]: the k largest logits of the token in
 *             descending order; equal logits (IEEE equality, -0 == +0) are
 *             ordered by lower expert index first.  A NaN logit ranks below
 *             every number (-inf included), NaNs among themselves by index,
 *             so every token always gets k distinct experts in [0, E).
 *   topk_prob out fp32 [T][k]: softmax over the k selected logits,
 *             p_j = exp(l_j - l_0) / sum_i exp(l_i - l_0), summed in j order
 *             (NaN for every pick of a token whose picks include a NaN).
 * Errors: MOE_ERR_INVALID for null pointers, T < 1, k < 1 or k > E;
 * MOE_ERR_UNSUPPORTED for E > 256 or T * k >= 2^31.
 */
int moe_route(const float* logits, int64_t T, int64_t E, int64_t k,
              int32_t* topk_idx, float* topk_prob, void* stream);

/*
 * moe_permute -- dispatch on one GPU: copy every token row to one row per
 * assignment, in expert-contiguous order (Spanish summary, section 2.1,
 * dispatch; German summary, section 1: dropless routing).
 *   build_map = 1: from topk_idx [T][k] computes
 *       counts   out int32 [E]   rows per expert;
 *       offsets  out int32 [E+1] exclusive prefix sum, offsets[E] = P;
 *       row_of   out int32 [T][k] destination row of assignment (t, j);
 *       token_of out int32 [P]   source token of each row;
 *     rows of one expert ascend by token index (a stable counting sort), so
 *     the map is unique.  An index outside [0, E) gets no row: its row_of
 *     entry is -1 and it is not counted (offsets[E] is then below P and the
 *     rows from offsets[E] on are not written).  Needs ws_bytes >=
 *     moe_workspace_bytes(sh, MOE_WS_PERMUTE).
 *   build_map = 0: uses the caller's row_of; counts, offsets, token_of, ws
 *     may be NULL.
 *   dst NULL (build_map = 1 only): the map alone, no rows moved (src may be
 *     NULL); the experts then read x through token_of (the *_gather calls).
 *   src [T][d] and dst [P][d] are in sh->dtype.  Assignments whose row_of
 *   entry lies outside [0, P) are skipped (here and in every call that reads
 *   row_of).  row_scale NULL: dst rows are bit copies of src rows.  row_scale fp32 [T][k] non-NULL: dst[row_of[t][j]]
 *   = round(row_scale[t][j] * src[t]) computed in fp32 (the backward of the
 *   weighted combine, dO = p * dY).
 */
int moe_permute(const moe_shape* sh, const void* src, const int32_t* topk_idx,
                const float* row_scale, int build_map, int32_t* counts, int32_t* offsets,
                int32_t* row_of, int32_t* token_of, void* dst, void* ws, size_t ws_bytes,
                void* stream);

/*
 * moe_permute_noalloc -- moe_permute without a workspace argument, for
 * callers that cannot allocate device memory (code under HIP graph capture,
 * tight serving loops, harnesses that forbid hipMalloc).  With build_map = 1
 * the map's per-(expert, 256-token block) counts, E * ceil(T / 256) int32
 * (aligned up to 256 bytes), go to a 1 MiB array that the library keeps in
 * device memory, one per GPU, for the life of the process (e.g. E = 256
 * experts allow T <= 262144 tokens); larger maps return MOE_ERR_WORKSPACE
 * before anything is enqueued.  All calls on one GPU share that array: calls
 * that overlap on one GPU (other streams, other threads) race and must be
 * serialised by the caller.  Nothing in it needs to start at zero.  The first
 * call on a device looks up the array's device address (MOE_ERR_HIP if the
 * runtime cannot); no call allocates or frees memory.  Arguments, results
 * and errors otherwise as moe_permute.
 */
int moe_permute_noalloc(const moe_shape* sh, const void* src, const int32_t* topk_idx,
                        const float* row_scale, int build_map, int32_t* counts,
                        int32_t* offsets, int32_t* row_of, int32_t* token_of, void* dst,
                        void* stream);

/*
 * moe_unpermute -- combine on one GPU (Spanish summary, section 2.1):
 *   dst[t] = round( sum_{j=0..k-1} w[t][j] * src[row_of[t][j]] + add[t] )
 * with the sum in fp32 in j order, w = topk_prob (fp32 [T][k]) or 1 when
 * topk_prob is NULL (the backward of moe_permute), add [T][d] optional
 * (NULL = none; used for the shared expert).  src [P][d], dst [T][d] in
 * sh->dtype.  dst must not alias src.
 */
int moe_unpermute(const moe_shape* sh, const void* src, const int32_t* row_of,
                  const float* topk_prob, const void* add, void* dst, void* stream);

/*
 * moe_grouped_gemm_fwd -- the experts' forward as grouped GEMMs over the
 * expert-contiguous rows (German summary, section 2 D, and Spanish summary,
 * section 2.3 C: one grouped GEMM bundles the many small expert GEMMs).
 * For expert e and its rows r in [offsets[e], offsets[e+1]):
 *   a = xp_r W1_e, b = xp_r W3_e           saved: ab [P][2f] = [a | b]
 *   h = silu(a) * b                        saved: h  [P][f]
 *   o = h W2_e                             out:   o  [P][d]
 * offsets int32 [E+1] lives on the device (typically from moe_permute); the
 * kernels read it there.  Rows of experts with no tokens are not touched.
 * ws may be NULL (current kernels need no workspace).
 */
int moe_grouped_gemm_fwd(const moe_shape* sh, const int32_t* offsets, const void* xp,
                         const void* W1, const void* W3, const void* W2, void* ab, void* h,
                         void* o, void* ws, size_t ws_bytes, void* stream);

/*
 * moe_grouped_gemm_bwd -- data and weight gradients of moe_grouped_gemm_fwd,
 * as separate products (German summary, section 2 C: W/D split).  Inputs are
 * the forward's xp, ab, h and the upstream gradient dO [P][d]; outputs:
 *   dab [P][2f] = [da | db],  dH = dO W2_e^T, s = sigmoid(a),
 *                 da = dH * b * s * (1 + a (1 - s)), db = dH * silu(a)
 *   dXp [P][d]  = da W1_e^T + db W3_e^T
 *   dW2 [E][f][d] = h_e^T dO_e, dW1 = xp_e^T da_e, dW3 = xp_e^T db_e
 * (each accumulated in fp32 over all of the expert's rows, rounded once).
 * Experts with no rows get all-zero dW1, dW3, dW2.
 */
int moe_grouped_gemm_bwd(const moe_shape* sh, const int32_t* offsets, const void* xp,
                         const void* ab, const void* h, const void* dO, const void* W1,
                         const void* W3, const void* W2, void* dab, void* dXp, void* dW1,
                         void* dW3, void* dW2, void* ws, size_t ws_bytes, void* stream);

/*
 * moe_grouped_gemm_fwd_gather / moe_grouped_gemm_bwd_gather -- the same
 * products with the permutation fused into the expert GEMMs' operand loads
 * (the pages' dispatchers eliminate permutation steps: German technical
 * summary, section 2 C, and the hyper.ai article on Hybrid-EP): row r of the
 * permuted input is row token_of[r] of x [T][d] (token_of from moe_permute's
 * map), read by fc1 forward and by the fc1 weight gradient, so no permuted
 * copy xp is written or read.  An entry outside [0, T) counts as a row of
 * zeros.  Results equal moe_grouped_gemm_fwd / _bwd on
 * xp = x[token_of] bit for bit.  bf16 and fp32; MOE_ERR_UNSUPPORTED when
 * T * d * element bytes >= 2^31 - 4096.
 */
int moe_grouped_gemm_fwd_gather(const moe_shape* sh, const int32_t* offsets,
                                const int32_t* token_of, const void* x, const void* W1,
                                const void* W3, const void* W2, void* ab, void* h, void* o,
                                void* ws, size_t ws_bytes, void* stream);
int moe_grouped_gemm_bwd_gather(const moe_shape* sh, const int32_t* offsets,
                                const int32_t* token_of, const void* x, const void* ab,
                                const void* h, const void* dO, const void* W1, const void* W3,
                                const void* W2, void* dab, void* dXp, void* dW1, void* dW3,
                                void* dW2, void* ws, size_t ws_bytes, void* stream);

/*
 * Buffers of a whole layer.  Inputs are read-only; "saved" buffers are
 * written by moe_layer_fwd and read by moe_layer_bwd; the rest are outputs.
 * Shared-expert pointers are ignored when f_shared == 0.
 */
typedef struct {
  /* inputs */
  const float* logits;                    /* fp32 [T][E] */
  const void* x;                          /* [T][d] */
  const void *W1, *W3, *W2;               /* [E][d][f], [E][d][f], [E][f][d] */
  const void *Ws1, *Ws3, *Ws2;            /* shared expert [d][fs], [d][fs], [fs][d] */
  const void* dY;                         /* [T][d], backward only */
  /* routing (written by fwd) */
  int32_t* topk_idx;                      /* [T][k] */
  float* topk_prob;                       /* [T][k] */
  int32_t *counts, *offsets;              /* [E], [E+1] */
  int32_t *row_of, *token_of;             /* [T][k], [P] */
  /* saved activations (written by fwd) */
  void *xp, *ab, *h, *o;                  /* [P][d], [P][2f], [P][f], [P][d] */
  void *s_ab, *s_h, *ys;                  /* shared expert: [T][2fs], [T][fs], [T][d] */
  /* forward output */
  void* y;                                /* [T][d] */
  /* backward scratch and outputs */
  void *dO, *dab, *dXp;                   /* [P][d], [P][2f], [P][d] */
  void *s_dab, *dXs;                      /* shared expert: [T][2fs], [T][d] */
  void* dX;                               /* [T][d] */
  void *dW1, *dW3, *dW2;                  /* like W1, W3, W2 */
  void *dWs1, *dWs3, *dWs2;               /* like Ws1, Ws3, Ws2 */
  /* e4m3 layers only (sh->dtype == MOE_E4M3; ignored otherwise): the
     quantised weights replace W1, W3, W2, which may be NULL; xp is not
     used (the backward reads x and token_of instead) */
  const struct moe_e4m3_weights* wq;
  uint8_t* xq;                            /* [T][d] codes of x */
  float* xs;                              /* [T][d/128] scales of x */
  uint8_t* xpq;                           /* [P][d] permuted codes */
  float* xps;                             /* [P][d/128] permuted scales */
  /* router gradient (optional; NULL = not computed): the forward writes the
     load-balancing loss when aux_loss is set, the backward writes dprob and
     dlogits when dlogits is set (dprob is then required) */
  float* aux_loss;                        /* device scalar */
  float* dprob;                           /* [T][k] */
  float* dlogits;                         /* [T][E] */
  float aux_alpha;                        /* coefficient alpha of the loss; 0 = none */
  /* memory-efficient permutation (bf16, e4m3, MXFP8): when memory_efficient != 0
     the probabilities are applied before W2 (h and o hold p-scaled values),
     the backward reads neither o nor a scaled dO, and row_prob [P] (written
     by the forward, read by the backward) holds each permuted row's
     probability; memory_efficient == 2 also recomputes h in the backward
     (the forward's h need not be kept, io->h is then overwritten), and 3 is
     the 8-bit checkpoint below (bf16 layers; e4m3 and MXFP8 layers refuse it
     with MOE_ERR_UNSUPPORTED); other non-zero values act as 1 */
  float* row_prob;
  int32_t memory_efficient;
  /* MXFP8 layers (sh->dtype == MOE_MXFP8): the quantised weights (W1, W3, W2
     may be NULL); xq, xpq hold codes as for e4m3 and xs, xps hold E8M0 scale
     bytes, [T][d/32] and [P][d/32] (the same byte count as the e4m3 scales) */
  const struct moe_mx_weights* wmx;
  /* fused permutation (bf16 and fp32 layers): when fused_permute != 0 the
     forward builds the map alone and the experts' fc1 forward and fc1 weight
     gradient read row token_of[r] of x directly (moe_grouped_gemm_fwd_gather
     / moe_grouped_gemm_bwd_gather), so xp is neither written nor read and
     may be NULL; needs T * d * element bytes below 2^31 - 4096 */
  int32_t fused_permute;
  /* MXFP4 layers (sh->dtype == MOE_MXFP4 or MOE_MXFP4_A8; moe_layer_fwd only):
     the quantised weights; xq holds the codes of x ([T][d/2], MXFP4_A8 [T][d])
     and xs its scale bytes [T][d/32].  xp, xpq, xps, ab and h are not used */
  const struct moe_mx4_weights* wmx4;
  /* 8-bit checkpoint (bf16 layers, memory_efficient == 3): as
     memory_efficient == 2, with [a|b] kept as E4M3 codes ab_q [P][2f] and E8M0
     bytes ab_s [P][2f/32] between forward and backward; ab is not used */
  uint8_t* ab_q;
  uint8_t* ab_s;
  /* e4m3, MXFP8 and MXFP4 layers: when x_quantized != 0, xq and xs hold x's
     quantised rows already (from moe_add_rms_norm) and moe_layer_fwd reads them
     in place of quantising x (x itself is read by the backward alone and may be
     NULL in the forward); other layers ignore it */
  int32_t x_quantized;
  /* integer-weight layers (sh->dtype == MOE_INT4; moe_layer_fwd only): the packed
     weights.  xp, ab, h, xq and xs are not used; a shared expert has bf16 weights
     and its buffers s_ab, s_h, ys */
  const struct moe_i4_weights* wi4;
} moe_layer_io;

/*
 * moe_layer_fwd -- route, permute, expert forward (+ shared expert applied to
 * every token with weight 1), weighted combine into y.  Same as calling
 * moe_route, moe_permute(build_map=1), moe_grouped_gemm_fwd and
 * moe_unpermute in sequence on one stream.  For MOE_E4M3: moe_route,
 * moe_quantize_rows of x into xq/xs, moe_permute_e4m3 into xpq/xps,
 * moe_grouped_gemm_fwd_e4m3, moe_unpermute (MOE_MXFP8: the _mx calls, weights
 * io->wmx).  For MOE_MXFP4 / MOE_MXFP4_A8: moe_route, the permutation's map,
 * moe_quantize_rows_mx4 / _mx of x, moe_grouped_gemm_fwd_mx4 reading x through
 * token_of, moe_unpermute (io->memory_efficient must be 0).  For MOE_INT4:
 * moe_route, the map, moe_grouped_gemm_fwd_i4 reading x through token_of (and the
 * bf16 shared expert), moe_unpermute (no memory_efficient either).  With io->aux_loss
 * set, the routing is moe_route_aux and moe_aux_loss_final (alpha =
 * io->aux_alpha) follows the permutation; ws_bytes then needs MOE_WS_AUX_LOSS
 * more bytes.  With io->memory_efficient:
 * moe_row_probs into io->row_prob, the row-scaled expert forward (bf16:
 * moe_grouped_gemm_fwd_rowscaled; e4m3 / MXFP8: fc1's epilogue scales h by p
 * before h is quantised) and an unweighted moe_unpermute.
 */
int moe_layer_fwd(const moe_shape* sh, const moe_layer_io* io, void* ws, size_t ws_bytes,
                  void* stream);

/*
 * moe_layer_bwd -- backward of moe_layer_fwd for upstream gradient dY:
 * dO = p * dY permuted, expert backward, dX = un-permuted sum of dXp (+ the
 * shared expert's dXs), and all weight gradients.  No gradient flows to the
 * logits unless io->dlogits is set: then dO comes from moe_combine_bwd
 * (writing io->dprob) and moe_route_bwd adds the router gradient, with the
 * load-balancing term (coefficient io->aux_alpha, upstream gradient 1).  For
 * MOE_E4M3 the expert backward is moe_grouped_gemm_bwd_e4m3.  With
 * io->memory_efficient: dO = dY permuted without scaling, then
 * moe_grouped_gemm_bwd_rowscaled (io->o is not read; dprob comes from its
 * partials; e4m3 and MXFP8 layers run the same steps with their products);
 * ws_bytes >= moe_workspace_bytes(sh, MOE_WS_LAYER_BWD_ROWSCALED).
 */
int moe_layer_bwd(const moe_shape* sh, const moe_layer_io* io, void* ws, size_t ws_bytes,
                  void* stream);

/*
 * e4m3 expert GEMMs
 * -----------------
 * The pages train the experts in FP8 with blockwise scaling on Hopper and
 * quantise weights straight from fp32 masters, keeping the router in high
 * precision (German technical summary, section 2 E; French summary, section
 * 2 E).  The quantiser used for every block B of values:
 *   amax = max |v| over B; scale = 1 if amax == 0 else fp32(amax / 448);
 *   code = OCP E4M3FN(fp32(v / scale)) rounded to nearest even, saturating
 *   at +-448, subnormals kept, -0 and tiny negatives -> 0x80; an all-zero
 *   block has every code +0.  A code stands for code * scale.
 * Block shapes: 1 x 128 along the contraction for activations and
 * gradients (xp, h, dO, da|db), 128 x 128 tiles for expert weights, and for
 * the weight-gradient products (contraction over an expert's rows) 128
 * consecutive rows of one expert per column, the expert's last block short.
 * The GEMMs accumulate in fp32: each 128-long block product is added times
 * the product of its two scales.  Outputs are bf16.  d and f must be
 * multiples of 128; e4m3 layers have no shared expert.
 */

/* Quantised expert weights as written by moe_quantize_weights. */
typedef struct moe_e4m3_weights {
  const uint8_t *W1, *W3, *W2;    /* codes [E][d][f], [E][d][f], [E][f][d] */
  const uint8_t *W1t, *W3t, *W2t; /* not read (may be NULL): the products take every weight in the
                                     orientation above, the forward ones MN-contiguous */
  const float *W1s, *W3s, *W2s;   /* tile scales [E][d/128][f/128] (W1, W3), [E][f/128][d/128] (W2) */
} moe_e4m3_weights;

/*
 * moe_quantize_rows -- 1 x 128 blocks along each row of src [rows][cols]
 * (src_dtype MOE_BF16 or MOE_F32, cols a multiple of 128):
 *   codes  out uint8 [rows][cols];  scales out fp32 [rows][cols/128].
 */
int moe_quantize_rows(const void* src, int32_t src_dtype, int64_t rows, int64_t cols,
                      uint8_t* codes, float* scales, void* stream);

/*
 * moe_quantize_weights -- 128 x 128 tiles of E fp32 matrices W [E][R][C]
 * (R, C multiples of 128):
 *   codes   out uint8 [E][R][C];
 *   codes_t out uint8 [E][C][R], the same codes transposed (may be NULL);
 *   scales  out fp32 [E][R/128][C/128].
 * For a layer: W1 and W3 with (R, C) = (d, f), W2 with (f, d).
 */
int moe_quantize_weights(const float* W, int64_t E, int64_t R, int64_t C, uint8_t* codes,
                         uint8_t* codes_t, float* scales, void* stream);

/* Number of 128-row blocks that P rows over E experts can need at most
 * (P/128 + E); the token-block buffers below are sized with it. */
int64_t moe_token_block_capacity(int64_t P, int64_t E);

/*
 * moe_quantize_token_blocks -- the weight-gradient operand blocks: for every
 * expert e (rows offsets[e] .. offsets[e+1]-1 of a [P][C] matrix) and each
 * of its 128-row blocks b (the last one short), one block per column.
 * Row r of the matrix is row src_row[r] of src (src_row NULL: row r), src
 * bf16 [.][C], C a multiple of 128.  With cap = moe_token_block_capacity:
 *   blk     out int32 [E+1]: first block of each expert, blk[E] = blocks used;
 *   codes   out uint8 [P][C]: the codes of row r in row r (row-major, the
 *           matrix's own layout; the weight-gradient GEMMs read them
 *           MN-contiguous);
 *   scales  out fp32 [cap][C]: scale of the expert's block j (rows
 *           offsets[e] + 128 j ..) and column c at row blk[e] + j; rows from
 *           blk[E] on are not written.
 */
int moe_quantize_token_blocks(const int32_t* offsets, int64_t E, int64_t P, const void* src,
                              const int32_t* src_row, int64_t C, int32_t* blk, uint8_t* codes,
                              float* scales, void* stream);

/*
 * moe_quantize_token_blocks_with_rows -- moe_quantize_token_blocks and, in
 * the same pass over the matrix, moe_quantize_rows of its rows: row_codes
 * uint8 [P][C] and row_scales fp32 [P][C/128], bit-identical to
 * moe_quantize_rows (the backward's dO and [da db] feed both a data gradient
 * and a weight gradient, German §2 E / French §2 E).  Arguments and errors as
 * moe_quantize_token_blocks; row_codes and row_scales must not be NULL.
 */
int moe_quantize_token_blocks_with_rows(const int32_t* offsets, int64_t E, int64_t P,
                                        const void* src, const int32_t* src_row, int64_t C,
                                        int32_t* blk, uint8_t* codes, float* scales,
                                        uint8_t* row_codes, float* row_scales, void* stream);

/*
 * moe_permute_e4m3 -- moe_permute for rows of e4m3 codes: codes [T][d] and
 * their scales [T][d/128] (from moe_quantize_rows of x) are copied bit for
 * bit to dst_codes [P][d] and dst_scales [P][d/128] at row row_of[t][j];
 * build_map and the map arguments as in moe_permute (quantising before the
 * permutation gives the same rows as after it, as scales are per row).
 */
int moe_permute_e4m3(const moe_shape* sh, const uint8_t* codes, const float* scales,
                     const int32_t* topk_idx, int build_map, int32_t* counts, int32_t* offsets,
                     int32_t* row_of, int32_t* token_of, uint8_t* dst_codes, float* dst_scales,
                     void* ws, size_t ws_bytes, void* stream);

/*
 * moe_grouped_gemm_fwd_e4m3 -- moe_grouped_gemm_fwd with e4m3 operands:
 * [a|b] = xp W{1,3} from xpq [P][d] / xps [P][d/128] and the weight codes;
 * ab and h = silu(a) * b are stored bf16; h is quantised (1 x 128 along f)
 * into the workspace and o = h W2 is stored bf16.  sh->dtype == MOE_E4M3;
 * ws_bytes >= moe_workspace_bytes(sh, MOE_WS_GEMM_FWD).
 */
int moe_grouped_gemm_fwd_e4m3(const moe_shape* sh, const int32_t* offsets, const uint8_t* xpq,
                              const float* xps, const moe_e4m3_weights* w, void* ab, void* h,
                              void* o, void* ws, size_t ws_bytes, void* stream);

/*
 * moe_grouped_gemm_bwd_e4m3 -- moe_grouped_gemm_bwd with e4m3 operands.
 * dO (bf16 [P][d]) is quantised 1 x 128 along d; dab = [da|db] is stored
 * bf16 and quantised 1 x 128 along 2f for dXp = da W1^T + db W3^T; the
 * weight gradients take token blocks of h, dO, dab and of the permuted x
 * (row r is x[token_of[r]], x bf16 [T][d]).  All outputs bf16.
 * ws_bytes >= moe_workspace_bytes(sh, MOE_WS_GEMM_BWD).
 */
int moe_grouped_gemm_bwd_e4m3(const moe_shape* sh, const int32_t* offsets,
                              const int32_t* token_of, const void* x, const void* ab,
                              const void* h, const void* dO, const moe_e4m3_weights* w, void* dab,
                              void* dXp, void* dW1, void* dW3, void* dW2, void* ws,
                              size_t ws_bytes, void* stream);

/*
 * Router gradient and load-balancing loss
 * ----------------------------------------
 * The pages fuse routing, permutation and auxiliary-loss computations into
 * few kernels (German technical summary, section 2 D "Kernel Fusion";
 * Spanish summary, section 2.3 C) without stating a formula.  Readings:
 *  - y[t] = sum_j p[t][j] o[row_of[t][j]] with p the softmax over the k
 *    selected logits, so dp[t][j] = <dY[t], o[row_of[t][j]]> and
 *    dlogits[t][topk_idx[t][j]] = p_j (dp_j - sum_i p_i dp_i), 0 for the
 *    experts not selected;
 *  - L = alpha E sum_e f_e P_e, f_e = counts[e] / (T k), P_e = mean over
 *    tokens of the softmax over all E logits; counts are held constant:
 *    dL/dlogits[t] = s[t] (g - <g, s[t]>), g_e = alpha E f_e / T.
 */

/*
 * moe_aux_loss -- *loss (device fp32 scalar) = L above, from the router
 * logits [T][E] and counts [E] (from moe_permute).  ws_bytes >=
 * moe_workspace_bytes(sh with this T and E, MOE_WS_AUX_LOSS).  Deterministic.
 */
int moe_aux_loss(const float* logits, int64_t T, int64_t E, int64_t k, const int32_t* counts,
                 float alpha, float* loss, void* ws, size_t ws_bytes, void* stream);

/*
 * moe_route_aux / moe_aux_loss_final -- moe_route fused with the first half
 * of moe_aux_loss (the pages fuse routing with the auxiliary-loss
 * computation: German technical summary, section 2 D).  moe_route_aux writes
 * topk_idx and topk_prob bit-identical to moe_route and, into ws (ws_bytes >=
 * moe_workspace_bytes(sh with this T and E, MOE_WS_AUX_LOSS)), the softmax
 * column sums of each 32-token block; once the permutation has produced the
 * counts, moe_aux_loss_final (the same ws, T, E, k) writes *loss, bit-
 * identical to moe_aux_loss on the same logits and counts.  One kernel fewer
 * than moe_route followed by moe_aux_loss.  Errors as moe_aux_loss.
 */
int moe_route_aux(const float* logits, int64_t T, int64_t E, int64_t k, int32_t* topk_idx,
                  float* topk_prob, void* ws, size_t ws_bytes, void* stream);
int moe_aux_loss_final(const void* ws, int64_t T, int64_t E, int64_t k, const int32_t* counts,
                       float alpha, float* loss, void* stream);

/*
 * moe_combine_bwd -- the backward of the weighted combine with the
 * probability gradient: dO[row_of[t][j]] = round(p[t][j] dY[t]) (exactly
 * moe_permute's scaled form) and dprob [T][k] fp32 = <dY[t], o[row_of[t][j]]>
 * with o [P][d] the expert outputs of the forward (sh->dtype; bf16 for
 * e4m3 layers).  d * element bytes must be at most 32768.
 */
int moe_combine_bwd(const moe_shape* sh, const void* dY, const void* o, const int32_t* row_of,
                    const float* topk_prob, void* dO, float* dprob, void* stream);

/*
 * moe_route_bwd -- dlogits [T][E] fp32: the top-k softmax Jacobian applied to
 * dprob, plus aux_scale * dL/dlogits of the load-balancing loss (skipped when
 * counts is NULL or alpha or aux_scale is 0).  logits, topk_idx, topk_prob
 * as in moe_route.  The Jacobian term is evaluated as
 * p_j sum_i p_i (dp_j - dp_i), which keeps its relative accuracy when one
 * probability is close to 1.
 */
int moe_route_bwd(const float* logits, int64_t T, int64_t E, int64_t k, const int32_t* topk_idx,
                  const float* topk_prob, const float* dprob, const int32_t* counts, float alpha,
                  float aux_scale, float* dlogits, void* stream);

/*
 * Memory-efficient permutation
 * -----------------------------
 * The pages reorder the routing weights algebraically so that the
 * permutation keeps no redundant intermediates ("Scalable Training of
 * Mixture-of-Experts Models with Megatron Core", German technical summary,
 * section 2 B, memory; Spanish summary, section 2.3 A).  Reading: W2 is
 * linear, so p (h W2) = (p h) W2; the probability is applied to h in the fc1
 * epilogue, the combine is an unweighted sum, and the backward needs neither
 * the expert outputs o nor a scaled dO: with dh' = dY[t] W2^T (unscaled
 * rows), dh = p dh' and dp = <h, dh'>, taken in the fc2 dgrad epilogue.
 * Results equal the plain layer's up to rounding.  The stand-alone row-scaled
 * GEMM calls below are bf16; e4m3 and MXFP8 layers take the same form through
 * moe_layer_fwd / moe_layer_bwd (io->memory_efficient).
 */

/*
 * moe_row_probs -- row_prob[row_of[t][j]] = topk_prob[t][j]: each permuted
 * row's routing probability ([P] fp32).
 */
int moe_row_probs(const moe_shape* sh, const int32_t* row_of, const float* topk_prob,
                  float* row_prob, void* stream);

/*
 * moe_grouped_gemm_fwd_rowscaled -- as moe_grouped_gemm_fwd, but h =
 * row_prob[r] * silu(a) * b, so o = h W2 is already weighted (combine with
 * moe_unpermute and topk_prob = NULL).  bf16 only (MOE_ERR_UNSUPPORTED else).
 */
int moe_grouped_gemm_fwd_rowscaled(const moe_shape* sh, const int32_t* offsets, const void* xp,
                                   const void* W1, const void* W3, const void* W2,
                                   const float* row_prob, void* ab, void* h, void* o,
                                   void* stream);

/*
 * moe_grouped_gemm_bwd_rowscaled -- backward of the row-scaled forward: dO
 * [P][d] is the UNSCALED permuted upstream gradient (moe_permute without
 * row_scale), h the p-scaled h of the forward, or, when recompute_h != 0, a
 * [P][f] buffer that the call first fills with p * silu(a) * b recomputed
 * from ab (so the forward's h need not be kept).  Writes dab, dXp, dW1, dW3,
 * dW2 as moe_grouped_gemm_bwd, and, when dprob is not NULL, the probability
 * gradient <silu(a_r) b_r, dO_r W2^T> of each permuted row r: dprob [P] in
 * row order when row_of is NULL, else dprob [T][k] with
 * dprob[t][j] = that of row row_of[t][j].  ws_bytes >= moe_workspace_bytes(sh,
 * MOE_WS_GEMM_BWD_ROWSCALED) (per-row partials of the dot product).
 */
int moe_grouped_gemm_bwd_rowscaled(const moe_shape* sh, const int32_t* offsets, const void* xp,
                                   const void* ab, void* h, int32_t recompute_h, const void* dO,
                                   const void* W1, const void* W3, const void* W2,
                                   const float* row_prob, void* dab, void* dXp, void* dW1,
                                   void* dW3, void* dW2, const int32_t* row_of, float* dprob,
                                   void* ws, size_t ws_bytes, void* stream);

/*
 * 8-bit activation checkpoints
 * ----------------------------
 * The pages hold activations in 8 bits to save training memory (German summary,
 * section 2 B and results; French summary, section 2 E) without a recipe.  What
 * the experts' backward keeps from the forward besides its inputs is [a|b]
 * (h is recomputed).  Here it is kept as E4M3 codes with one E8M0 scale byte per
 * 32 columns of a row (the block rule of "MXFP8 expert GEMMs" with s at least
 * -126; a block with a NaN or an infinity has scale byte 255 and reads back as
 * NaN): 33/32 bytes a value in place of 2.  The forward's own results are those
 * of moe_grouped_gemm_fwd_rowscaled: h comes from the unrounded fp32 a and b.
 * The backward is that of moe_grouped_gemm_bwd_rowscaled with recompute_h at
 * the a and b that read back.  (Both up to the order of the fp32 sums: small
 * calls take kernels that split the contraction.)
 *
 * moe_grouped_gemm_fwd_ckpt8 -- row-scaled expert forward (probabilities before
 * W2) that writes abq uint8 [P][2f] and abs uint8 [P][2f/32] in place of ab.
 * x: row r is row token_of[r] of x [T][d] (an entry outside [0, T) counts as a
 * row of zeros), or, token_of NULL, row r of the permuted x [P][d].  h [P][f] is scratch (it need not be kept).
 */
int moe_grouped_gemm_fwd_ckpt8(const moe_shape* sh, const int32_t* offsets,
                               const int32_t* token_of, const void* x, const void* W1,
                               const void* W3, const void* W2, const float* row_prob,
                               uint8_t* abq, uint8_t* abs, void* h, void* o, void* stream);

/*
 * moe_grouped_gemm_bwd_ckpt8 -- its backward from abq, abs and the unscaled
 * permuted upstream gradient dO [P][d]: h [P][f] is filled with p silu(a) b,
 * outputs dab [P][2f], dXp, dW1, dW3, dW2 and (not NULL) dprob as
 * moe_grouped_gemm_bwd_rowscaled (row_of NULL: [P] in row order, entries from
 * offsets[E] on unspecified, else [T][k]).  dW2 may hold partial sums of dprob
 * until it is written.
 * ws_bytes >= moe_workspace_bytes(sh, MOE_WS_GEMM_BWD_ROWSCALED).  Both calls:
 * bf16 only (MOE_ERR_UNSUPPORTED else), limits as moe_grouped_gemm_fwd / _bwd
 * and, with token_of, moe_grouped_gemm_fwd_gather.
 */
int moe_grouped_gemm_bwd_ckpt8(const moe_shape* sh, const int32_t* offsets,
                               const int32_t* token_of, const void* x, const uint8_t* abq,
                               const uint8_t* abs, const void* dO, const void* W1, const void* W3,
                               const void* W2, const float* row_prob, void* h, void* dab, void* dXp,
                               void* dW1, void* dW3, void* dW2, const int32_t* row_of,
                               float* dprob, void* ws, size_t ws_bytes, void* stream);

/*
 * MXFP8 expert GEMMs
 * ------------------
 * The pages run the Blackwell results in MXFP8 (French summary, section 2 E;
 * Spanish summary, section 2.4) and name it without a definition; the
 * storage is the OCP Microscaling one.  Every block of 32 consecutive values
 * along a product's contraction axis has one scale 2^s, stored as the E8M0
 * byte s + 127, with s the smallest integer such that max|v| <= 448 * 2^s
 * (the scale rounded up, so nothing saturates; s clamped to [-127, 127]; an
 * all-zero block has s = 0 and +0 codes); codes are E4M3FN(v * 2^-s), round
 * to nearest even.  A block that holds a NaN or an infinity has scale byte 255,
 * E8M0's NaN: every product it enters is NaN.  This scale rule departs from the
 * OCP MX v1.0 reference conversion (s = floor(log2 max|v|) - 8 with elements
 * above 448 clamped), which can clip a block's largest element by up to 12.5 %.
 * gfx950's v_mfma_scale_f32_16x16x128_f8f6f4 takes one E8M0 scale per lane,
 * which is one 32-value block of one row, so the scales go straight into the
 * matrix instruction.  Scale bytes are stored row-major next to the codes they
 * scale:
 *  - activation rows [rows][K] -> bytes [rows][K/32];
 *  - each weight matrix in both orientations (the blocks of the two differ):
 *    codes [E][R][C] with row-block bytes [E][R][C/32] (read by the
 *    data-gradient products), and transposed codes [E][C][R] with
 *    column-block bytes [E][C][R/32] (read by the forward products);
 *  - weight-gradient operands as moe_quantize_token_blocks lays them out
 *    (codes [P][C]), with bytes [cap][C][4] (byte g of word (b, c): rows
 *    32 g.. of 128-row block b; 32-row blocks restart at each expert).
 * Shapes: d, f multiples of 128, no shared expert.
 */

/* Quantised expert weights as written by moe_quantize_weights_mx. */
typedef struct moe_mx_weights {
  const uint8_t *W1, *W3, *W2;       /* codes [E][d][f], [E][d][f], [E][f][d] */
  const uint8_t *W1t, *W3t, *W2t;    /* transposed codes [E][f][d], [E][f][d], [E][d][f] */
  const uint8_t *W1s, *W3s, *W2s;    /* row-block bytes [E][d][f/32], .., [E][f][d/32] */
  const uint8_t *W1ts, *W3ts, *W2ts; /* column-block bytes [E][f][d/32], .., [E][d][f/32] */
} moe_mx_weights;

/* moe_quantize_rows_mx -- 1 x 32 blocks along each row of src [rows][cols]
 * (MOE_BF16 or MOE_F32, cols a multiple of 32): codes [rows][cols], scale
 * bytes [rows][cols/32]. */
int moe_quantize_rows_mx(const void* src, int32_t src_dtype, int64_t rows, int64_t cols,
                         uint8_t* codes, uint8_t* scales, void* stream);

/* moe_quantize_weights_mx -- both orientations of E fp32 matrices W [E][R][C]
 * (R, C multiples of 128): codes [E][R][C] + bytes [E][R][C/32], codes_t
 * [E][C][R] + bytes [E][C][R/32]; one pass over W. */
int moe_quantize_weights_mx(const float* W, int64_t E, int64_t R, int64_t C, uint8_t* codes,
                            uint8_t* scales, uint8_t* codes_t, uint8_t* scales_t, void* stream);

/* moe_quantize_token_blocks_mx -- as moe_quantize_token_blocks, with 32-row
 * scale blocks: codes [P][C], scale bytes [capacity][C][4] (the four 32-row
 * blocks of each 128-row block and column in one word); 32-row blocks with
 * no rows have s = 0. */
int moe_quantize_token_blocks_mx(const int32_t* offsets, int64_t E, int64_t P, const void* src,
                                 const int32_t* src_row, int64_t C, int32_t* blk,
                                 uint8_t* codes, uint8_t* scales, void* stream);

/* moe_quantize_token_blocks_with_rows_mx -- moe_quantize_token_blocks_mx and,
 * in the same pass, moe_quantize_rows_mx of its rows: row_codes uint8 [P][C],
 * row_scales E8M0 bytes [P][C/32], bit-identical to moe_quantize_rows_mx. */
int moe_quantize_token_blocks_with_rows_mx(const int32_t* offsets, int64_t E, int64_t P,
                                           const void* src, const int32_t* src_row, int64_t C,
                                           int32_t* blk, uint8_t* codes, uint8_t* scales,
                                           uint8_t* row_codes, uint8_t* row_scales, void* stream);

/* moe_permute_mx -- moe_permute_e4m3 for MXFP8 rows: codes [T][d] and scale
 * bytes [T][d/32] moved to the permuted order (bit copies). */
int moe_permute_mx(const moe_shape* sh, const uint8_t* codes, const uint8_t* scales,
                   const int32_t* topk_idx, int build_map, int32_t* counts, int32_t* offsets,
                   int32_t* row_of, int32_t* token_of, uint8_t* dst_codes, uint8_t* dst_scales,
                   void* ws, size_t ws_bytes, void* stream);

/* moe_grouped_gemm_fwd_mx / moe_grouped_gemm_bwd_mx -- the e4m3 calls' MXFP8
 * counterparts (sh->dtype == MOE_MXFP8; xps are scale bytes [P][d/32]); the
 * same workspace sizes (MOE_WS_GEMM_FWD / MOE_WS_GEMM_BWD). */
int moe_grouped_gemm_fwd_mx(const moe_shape* sh, const int32_t* offsets, const uint8_t* xpq,
                            const uint8_t* xps, const moe_mx_weights* w, void* ab, void* h,
                            void* o, void* ws, size_t ws_bytes, void* stream);
int moe_grouped_gemm_bwd_mx(const moe_shape* sh, const int32_t* offsets, const int32_t* token_of,
                            const void* x, const void* ab, const void* h, const void* dO,
                            const moe_mx_weights* w, void* dab, void* dXp, void* dW1, void* dW3,
                            void* dW2, void* ws, size_t ws_bytes, void* stream);

/*
 * MXFP4 experts
 * -------------
 * The pages credit FP4 beside MXFP8 for the Blackwell results (German summary,
 * results table) without a definition; the storage is the OCP Microscaling one:
 * E2M1 codes (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives), two to a byte
 * with the lower index in the low nibble, and one E8M0 scale byte s + 127 per
 * 32 consecutive values along a product's contraction axis.  s is the smallest
 * integer with max|v| <= 6 * 2^s (nothing saturates; at least -126; 0 for an
 * all-zero block, whose codes are zeros), codes are E2M1(v * 2^-s), round to
 * nearest even, sign kept.  (As for MXFP8 the scale is rounded up where the OCP
 * MX v1.0 reference conversion takes s = floor(log2 max|v|) - 2 and clamps what
 * lies above 6 * 2^s, up to 25 % of a block's largest value.)  A block that holds a NaN or an infinity has scale
 * byte 255, E8M0's NaN: every product it enters is NaN.  Forward only: there
 * are no weight gradients in this format (moe_layer_bwd returns
 * MOE_ERR_UNSUPPORTED).  moe_dequantize_weights_mx4 gives the bf16 weights that
 * the codes stand for, for a bf16 backward on the weights the forward used.
 *
 * Weight layout.  A matrix with R rows (the contraction) and N columns is
 * stored in tiles of 128 rows x 16 columns, 1 KB each:
 *   codes  [E][N/16][R/128][4][16][16]: byte b of (group g, column c) of tile
 *          (nt, kt) holds rows 128 kt + 32 g + 2 b (low nibble) and + 1 of
 *          column 16 nt + c;
 *   scales [E][N/64][R/128][4][16][4]: byte j of (g, c) of (nb, kt) is the scale
 *          of rows 128 kt + 32 g .. + 31 of column 64 nb + 16 j + c.
 * W1 and W3 form one matrix W13 of N = 2f columns whose 16-column groups
 * alternate (group 2 i: columns 16 i .. of W1, group 2 i + 1: of W3).
 * d and f must be multiples of 128.  A layer call takes no shared expert
 * (MOE_ERR_UNSUPPORTED); with one, make the layer's calls one by one: the shared
 * expert is moe_grouped_gemm_fwd_mx4 of a shape {T, d, 1, 1, f_shared} on the same
 * quantised rows, offsets {0, T} and token_of NULL, and its o is moe_unpermute's
 * `add`.
 */

/* Quantised expert weights as written by moe_quantize_weights_mx4. */
typedef struct moe_mx4_weights {
  const uint8_t *W13, *W2;   /* codes of [E][d][2f] (W1 with W_pair = W3) and [E][f][d] */
  const uint8_t *W13s, *W2s; /* their scale bytes */
} moe_mx4_weights;

/* moe_quantize_rows_mx4 -- 1 x 32 blocks along each row of src [rows][cols]
 * (MOE_BF16 or MOE_F32, cols a multiple of 32): codes [rows][cols/2], scale
 * bytes [rows][cols/32]. */
int moe_quantize_rows_mx4(const void* src, int32_t src_dtype, int64_t rows, int64_t cols,
                          uint8_t* codes, uint8_t* scales, void* stream);

/* moe_quantize_weights_mx4 -- E matrices W [E][R][C] (MOE_F32 masters or
 * MOE_BF16; R, C multiples of 128) into the layout above, N = C; with W_pair
 * (a second [E][R][C], same type) N = 2C and the 16-column groups of W and
 * W_pair alternate.  One pass over the source. */
int moe_quantize_weights_mx4(const void* W, const void* W_pair, int32_t src_dtype, int64_t E,
                             int64_t R, int64_t C, uint8_t* codes, uint8_t* scales, void* stream);

/* moe_dequantize_weights_mx4 -- the values that the codes and scales stand for,
 * bf16 [E][R][C] (exact unless below bf16's range), W_pair NULL for a single
 * matrix. */
int moe_dequantize_weights_mx4(const uint8_t* codes, const uint8_t* scales, int64_t E, int64_t R,
                               int64_t C, void* W, void* W_pair, void* stream);

/*
 * moe_grouped_gemm_fwd_mx4 -- the experts' forward on quantised rows: for
 * expert e and its rows r in [offsets[e], offsets[e+1])
 *   [a|b] = xq_r W13_e, h = silu(a) b, o = Q(h) W2_e
 * with fp32 accumulation; Q rounds h once, from fp32, to MXFP4 (MOE_MXFP4) or
 * MXFP8 (MOE_MXFP4_A8, the rule of "MXFP8 expert GEMMs" with s at least -126
 * and NaN blocks as above) and o [P][d] is bf16.  xq, xs are rows as
 * moe_quantize_rows_mx4 (MOE_MXFP4) or moe_quantize_rows_mx (MOE_MXFP4_A8)
 * writes them: row r is row token_of[r] of [T] rows, or, token_of NULL, row r
 * of [P] permuted rows; an entry outside [0, T) reads a row of zeros.  Rows of o
 * from offsets[E] on are not written.
 * ws_bytes >= moe_workspace_bytes(sh, MOE_WS_GEMM_FWD).  Errors: MOE_ERR_INVALID
 * for another dtype; MOE_ERR_UNSUPPORTED for d or f not a multiple of 128,
 * P * max(d, f) >= 2^31 - 4096 or d * f >= 2^31.
 * (With E4M3 rows the matrix instruction itself cuts the products of each 8
 * consecutive k to multiples of 2^-13 of the largest before it adds them in
 * fp32; E2M1 products are added exactly.)
 */
int moe_grouped_gemm_fwd_mx4(const moe_shape* sh, const int32_t* offsets, const int32_t* token_of,
                             const uint8_t* xq, const uint8_t* xs, const moe_mx4_weights* w,
                             void* o, void* ws, size_t ws_bytes, void* stream);

/*
 * Integer expert weights
 * ----------------------
 * The 4-bit checkpoints that are common beside FP4: codes q in 0 .. 15, with a
 * scale s and a zero point z for each group of 32, 64 or 128 consecutive rows
 * (the contraction) of a column.  The weight that a code stands for is
 * bf16(s (q - z)): the difference's product is exact in fp32 and rounded once, so
 * products on the codes use the numbers that moe_dequantize_weights_i4 writes,
 * and its bf16 weights serve a backward (as for MXFP4 there are no weight
 * gradients in this format).  Activations are bf16.
 *
 * Layout.  As for MXFP4 a matrix of R rows and N columns is stored in tiles of
 * 128 rows x 16 columns, 1 KB each:
 *   codes  [E][N/16][R/128][4][16][16]: byte 4 j + b of (group g, column c) of
 *          tile (nt, kt) holds rows 128 kt + 32 j + 8 g + b (low nibble) and + 4
 *          (high nibble) of column 16 nt + c;
 *   scales [E][N/64][R/128][128/group][16][4] 32-bit words: word i of (u, c) of
 *          (nb, kt) is the scale of rows 128 kt + group u .. of column 64 nb +
 *          16 i + c: the fp32 number s, whose low four bits hold z (s has 20
 *          significant bits: fp16 and bf16 scales are kept exactly).
 * W1 and W3 form one matrix W13 of N = 2f columns whose 16-column groups alternate
 * (group 2 i: columns 16 i .. of W1, group 2 i + 1: of W3).  d and f must be
 * multiples of 128.  A layer takes a shared expert with bf16 weights.
 */

/* Packed expert weights as written by moe_quantize_weights_i4 or
 * moe_pack_weights_i4. */
typedef struct moe_i4_weights {
  const uint8_t *W13, *W2;    /* codes of [E][d][2f] (W1 with W_pair = W3) and [E][f][d] */
  const uint32_t *W13s, *W2s; /* their scale words */
  int64_t group;              /* rows of a group: 32, 64 or 128 */
} moe_i4_weights;

/* moe_quantize_weights_i4 -- E matrices W [E][R][C] (MOE_F32 masters or MOE_BF16;
 * R, C multiples of 128) into the layout above, N = C; with W_pair (a second
 * [E][R][C], same type) N = 2C and the 16-column groups of W and W_pair alternate.
 * For a group's weights w, with s the smallest number of 20 significant bits, at
 * least 2^-126, that
 *   asymmetric == 0:  max|w| <= 7 s, z = 8;
 *   asymmetric != 0:  hi - lo <= 15 s, lo = min(w, 0), hi = max(w, 0), z = the
 *                     nearest integer to -lo / s;
 * q = the nearest integer to w / s, plus z, held to 0 .. 15; all ties to even and
 * of the exact quotients.  A group of zeros has s = 1 and codes equal to z.  A
 * group with a NaN or an infinity, or whose s would be 2^124 or more, has s = NaN:
 * its weights and every product they enter are NaN. */
int moe_quantize_weights_i4(const void* W, const void* W_pair, int32_t src_dtype, int32_t asymmetric, int64_t group,
                            int64_t E, int64_t R, int64_t C, uint8_t* codes, uint32_t* scales, void* stream);

/* moe_pack_weights_i4 -- the same layout from a checkpoint's codes q uint8
 * [E][R][C] (one to a byte, the low four bits count), scales s fp32 [E][R/group][C]
 * (rounded to 20 significant bits, below 2^-126 to multiples of 2^-145; not finite, or
 * 2^124 and more after that: NaN) and zero points z uint8 [E][R/group][C] (the low
 * four bits count; NULL: 8); q_pair, s_pair, z_pair: a second matrix whose groups
 * alternate, or NULL. */
int moe_pack_weights_i4(const uint8_t* q, const float* s, const uint8_t* z, const uint8_t* q_pair, const float* s_pair,
                        const uint8_t* z_pair, int64_t group, int64_t E, int64_t R, int64_t C, uint8_t* codes,
                        uint32_t* scales, void* stream);

/* moe_dequantize_weights_i4 -- the weights bf16 [E][R][C] that codes and scales
 * stand for, W_pair NULL for a single matrix. */
int moe_dequantize_weights_i4(const uint8_t* codes, const uint32_t* scales, int64_t group, int64_t E, int64_t R,
                              int64_t C, void* W, void* W_pair, void* stream);

/*
 * moe_grouped_gemm_fwd_i4 -- the experts' forward on bf16 rows: for expert e and
 * its rows r in [offsets[e], offsets[e+1])
 *   [a|b] = x_r W13_e, h = silu(a) b rounded to bf16, o = h W2_e
 * with fp32 accumulation; o [P][d] is bf16.  Row r is row token_of[r] of x [T][d]
 * (an entry outside [0, T) reads a row of zeros), or, token_of NULL, row r of the
 * permuted x [P][d].  Rows of o from offsets[E] on are not written.
 *
 * Workspace: h, P * f * 2 bytes, is the least (MOE_ERR_WORKSPACE below).
 * moe_workspace_bytes(sh, MOE_WS_GEMM_FWD) adds the fp32 sums over up to four parts of
 * the contraction (d and f) where the rows are too few to fill the chip with whole
 * products; calls with more rows may need none, so that number does not always grow
 * with T.  With less room the call takes as many parts as fit, one at least, and is
 * slower for it.  So a workspace for the largest T serves every smaller one, and one of
 * the largest number over the T that are served serves each at its best.  A layer's
 * workspace likewise: MOE_WS_LAYER_FWD counts the sums, MOE_WS_PERMUTE + 256 + P * f * 2
 * (with io->aux_loss: + MOE_WS_AUX_LOSS) is the least.
 *
 * The order of an element's fp32 sum, and with it the last bits of a result, goes by
 * the kernel (moe_few_rows) and, in the kernel for many rows, by the parts of the
 * contraction: by P, E, d, f and by ws_bytes where that holds fewer parts.
 *
 * Errors: MOE_ERR_INVALID for another dtype; MOE_ERR_UNSUPPORTED for d or f not a
 * multiple of 128, another group than 32, 64 or 128, P * max(d, f) >= 2^30 - 2048 or
 * d * f >= 2^31.
 */
int moe_grouped_gemm_fwd_i4(const moe_shape* sh, const int32_t* offsets, const int32_t* token_of, const void* x,
                            const moe_i4_weights* w, void* o, void* ws, size_t ws_bytes, void* stream);

/*
 * The norm in front of a layer
 * ----------------------------
 * A transformer block hands the layer x = norm(residual stream).  The pages
 * keep activations in 8 bits and fuse the elementwise steps into few kernels
 * (German summary, section 2 D and 2 E) without a recipe; the norm is the root-
 * mean-square one, and the rows that a layer's products read are quantised from
 * it in the same pass.
 *
 * moe_add_rms_norm -- for each of T rows of d values (dtype MOE_BF16 or MOE_F32:
 * the type of x, residual, gamma, sum and y)
 *   s = x + residual, rounded to dtype (residual NULL: s = x)
 *   rstd = 1 / sqrt(mean(s^2) + eps),  v = s rstd gamma   (fp32)
 *   sum  out [T][d]: s (may be NULL; with a residual it is the new residual
 *        stream and what the backward reads)
 *   y    out [T][d]: v rounded to dtype (may be NULL)
 *   rstd out fp32 [T] (may be NULL)
 *   codes, scales out (both or neither): v quantised row by row, straight from
 *        fp32, q_dtype (ignored without them) MOE_E4M3 (moe_quantize_rows'
 *        rule: codes [T][d], fp32 scales [T][d/128]), MOE_MXFP8
 *        (moe_quantize_rows_mx's with s at least -126: codes [T][d], bytes
 *        [T][d/32]) or MOE_MXFP4 (moe_quantize_rows_mx4's: codes [T][d/2], bytes
 *        [T][d/32]).  A block with a NaN or an infinity reads back as NaN (scale
 *        byte 255; MOE_E4M3: the scale is NaN).
 * A layer takes them as io->xq and io->xs with io->x_quantized set.  sum may be
 * x or residual, and y may be x, residual or sum.  The squares are added in
 * fp32, scaled where they would leave its range: any finite s is in range as long
 * as rstd is.  T = 0 does nothing.  Errors:
 * MOE_ERR_INVALID for null x or gamma, no output, codes without scales, T < 0, d
 * < 1, eps negative or not finite; MOE_ERR_UNSUPPORTED for d not a multiple of 8
 * (128 for E4M3 rows, 32 for MX rows) or above 32768, T >= 2^31 (2^26, 2^24 and 2^22 for
 * d up to 1024, up to 8192 and above: 2^32 threads), other types, misaligned pointers.
 */
int moe_add_rms_norm(const void* x, const void* residual, const void* gamma, int32_t dtype, int64_t T, int64_t d,
                     float eps, void* sum, void* y, float* rstd, int32_t q_dtype, uint8_t* codes, void* scales,
                     void* stream);

/*
 * moe_add_rms_norm_bwd -- its gradients for the upstream gradient dy [T][d] of y
 * and, dsum not NULL, dsum [T][d] of sum: with g = dy gamma
 *   dx     out [T][d] = dsum + rstd (g - s rstd^2 mean(g s))  (of x and of the
 *          residual alike), rounded once
 *   dgamma out [d] = sum over the rows of dy s rstd, in fp32, rounded once (T = 0:
 *          zeros)
 * from the forward's sum and rstd (without a residual: x).  Deterministic.
 * dx may be dy, sum or dsum.  ws_bytes >= moe_workspace_bytes of a shape with this T
 * and d (E = k = 1 and any f do), MOE_WS_NORM_BWD.  That number falls where T passes
 * what the chip takes at once, since the rows are then dealt out evenly; a program that
 * keeps one workspace asks for MOE_WS_NORM_BWD_MAX with its largest T.  Types, limits
 * and errors as moe_add_rms_norm (T < 2^31 for every d).
 */
int moe_add_rms_norm_bwd(const void* dy, const void* sum, const float* rstd, const void* gamma, const void* dsum,
                         int32_t dtype, int64_t T, int64_t d, void* dx, void* dgamma, void* ws, size_t ws_bytes,
                         void* stream);

/*
 * moe_dequantize_rows -- the values that quantised rows [rows][cols] stand for
 * (q_dtype MOE_E4M3, MOE_MXFP8 or MOE_MXFP4, as moe_quantize_rows, _rows_mx,
 * _rows_mx4 and moe_add_rms_norm write them), dst [rows][cols] MOE_BF16 or
 * MOE_F32: code times scale in fp32, rounded once.
 */
int moe_dequantize_rows(const uint8_t* codes, const void* scales, int32_t q_dtype, int64_t rows, int64_t cols,
                        void* dst, int32_t dst_dtype, void* stream);

/* moe_probe_mfma -- measurement helper, not a step of the layer: the dense
 * matrix-core rate and the shader clock this GPU sustains under MFMAs alone,
 * the ceiling against which the grouped GEMMs' rates can be read (published
 * peaks assume the peak clock; the chip clocks lower under a sustained
 * matrix-core load).  Launches, on `stream`, 8 blocks of 256 threads per
 * compute unit; every wavefront runs `iters` (1 .. 2^24) rounds of 8
 * independent MFMAs on register operands, v_mfma_f32_16x16x32_bf16 for
 * dtype = MOE_BF16 or v_mfma_scale_f32_16x16x128_f8f6f4 on e4m3 codes for
 * MOE_E4M3 (other dtypes: MOE_ERR_UNSUPPORTED).
 *   ticks    device, 2 x uint64, written by the kernel: the shader-clock
 *            cycles and the wall-clock ticks one wavefront's loop took;
 *   sink     device, 1 float, written only in the unlikely case that the
 *            folded results equal a sentinel (keeps the MFMAs alive);
 *   flops    host: the launch's MFMA flop count (2 per multiply-add);
 *   wall_khz host: the wall-clock tick rate, so clock = ticks[0] /
 *            (ticks[1] / (wall_khz * 1e3)).
 * The rate is flops / the launch's duration measured by the caller on
 * `stream`.  Returns MOE_ERR_INVALID for null pointers or iters outside the
 * range, MOE_ERR_HIP if the device cannot be queried or the launch fails. */
int moe_probe_mfma(int dtype, int64_t iters, unsigned long long* ticks, float* sink,
                   int64_t* flops, int64_t* wall_khz, void* stream);

/* Bytes of workspace the call `kind` needs for shape sh (0 if none). */
size_t moe_workspace_bytes(const moe_shape* sh, int kind);

/* 1 where the expert products of shape sh run on the kernels for few rows, else
 * 0: moe_grouped_gemm_fwd_mx4 (MOE_MXFP4, MOE_MXFP4_A8), moe_grouped_gemm_fwd_i4
 * (MOE_INT4) and the 8-bit checkpoint calls (MOE_BF16).  Those kernels split the
 * contraction, so results of calls on the two sides differ in the order of their fp32
 * sums.  (With MOE_INT4 so may those of two calls that both give 0: see
 * moe_grouped_gemm_fwd_i4.)  0 for other types and for shapes that are refused. */
int moe_few_rows(const moe_shape* sh);

/* Static, NUL-terminated name of a moe_status value. */
const char* moe_status_str(int status);

#ifdef __cplusplus
}
#endif

#endif /* TRE_MOE_H */
