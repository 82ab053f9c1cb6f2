/*
 * lpq — block-scaled low-precision quantize-then-GEMM for transformer linear
 * layers on GB300 (sm_103a).  C ABI of liblpq.so.
 *
 * What the library computes is defined by these pages:
 *   [FP8]   "Optimizing Transformer models for low-precision training"
 *           (setupai.cc summary), "technical deep dive": E4M3 (1/4/3 bits,
 *           forward activations and weights) and E5M2 (1/5/2, gradients);
 *           per-tensor dynamic scaling from the amax; amax history.
 *   [NVFP4] "Accelerate LLM training with NVFP4 on Blackwell" (setupai.cc
 *           summary), "technical deep dive": E2M1 values (range about +-6), an
 *           E4M3 scale per 16-value micro-block plus an FP32 tensor scale;
 *           MXFP4, the format it refines, shares one scale per 32 values.
 *   [TE]    "How to optimize Transformer-based models for low-precision
 *           training" (developer.nvidia.cn): config -> 12 GEMM shapes
 *           ("model configuration and training input", "autocast vs
 *           pre-quantize"), Fprop/Dgrad/Wgrad benchmarked separately,
 *           pre-quantize mode, the NVFP4 extra costs (random Hadamard
 *           transform on Wgrad inputs, stochastic rounding of gradients, 2D
 *           weight blocks, extra amax pass) and silent fallbacks to avoid
 *           ("interpreting real-model results").
 *   [NeMo]  "Faster training throughput in FP8 with NVIDIA NeMo", "advantages
 *           and trade-offs": delayed, current, sub-channel (1x128 / 128x128)
 *           and MXFP8 (32-value blocks, E8M0 power-of-two scales).
 *
 * Conventions for every entry point:
 *   - Device pointers are owned by the caller; the library allocates no device
 *     memory (TMEM inside kernels is allocated and released per launch).
 *   - Work is enqueued on `stream` (a cudaStream_t; NULL = legacy default
 *     stream) and the call returns without synchronising.
 *   - Every call returns an lpq_status; nothing throws across the ABI.  A
 *     non-OK status leaves a message readable with lpq_last_error() on the
 *     calling thread.  A call that returns non-OK has enqueued nothing unless
 *     the status is LPQ_ERR_CUDA.
 *   - No call ever falls back to another format, precision or a CPU path
 *     ([TE] warns of silent fallbacks): an unsupported combination is an error.
 *   - Matrices are row-major and contiguous along their last dimension.
 */
#ifndef LPQ_H_
#define LPQ_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st *lpq_stream_t; /* same type as cudaStream_t */

typedef enum {
  LPQ_OK = 0,
  LPQ_ERR_INVALID_ARG = 1, /* NULL pointer, bad enum or flag */
  LPQ_ERR_SHAPE = 2,       /* a dimension is not a multiple of the block / tile rule */
  LPQ_ERR_ALIGN = 3,       /* a pointer is not 16-byte aligned */
  LPQ_ERR_UNSUPPORTED = 4, /* format / layout / operand pairing not provided */
  LPQ_ERR_ARCH = 5,        /* current device is not compute capability 10.3 */
  LPQ_ERR_CUDA = 6,        /* a CUDA runtime call failed */
  LPQ_ERR_TIMEOUT = 7      /* a device-side wait gave up (see lpq_device_status) */
} lpq_status;

typedef enum {
  LPQ_BF16 = 0,               /* unquantized bf16 (the speed-up baseline) */
  LPQ_FP8_E4M3 = 1,           /* per-tensor scaled E4M3 [FP8] */
  LPQ_FP8_E5M2 = 2,           /* per-tensor scaled E5M2 [FP8] */
  LPQ_MXFP8 = 3,              /* E4M3 codes, one E8M0 scale per 32 values [NeMo] */
  LPQ_NVFP4 = 4,              /* E2M1 codes, E4M3 scale per 16 + FP32 tensor scale [NVFP4] */
  LPQ_NVFP4_2D = 5,           /* NVFP4 with one scale per 16x16 tile (weights) [TE] */
  LPQ_FP8_BLOCK_1x128 = 6,    /* E4M3, FP32 scale per 1x128 block (activations) [NeMo] */
  LPQ_FP8_BLOCK_128x128 = 7,  /* E4M3, FP32 scale per 128x128 block (weights) [NeMo] */
  LPQ_MXFP8_E5M2 = 8,         /* E5M2 codes, one E8M0 scale per 32 values (gradients) [NeMo], [FP8] */
  LPQ_MXFP4 = 9               /* packed E2M1 codes, one E8M0 scale per 32 values [NVFP4] */
} lpq_format;

/* Per-tensor FP8 scaling.  Every scale that is a quotient of a format maximum
 * by an amax (fmax / amax, NVFP4's 2688 / amax and s_enc / dec(S), the
 * sub-channel 448 / block max) is clamped to the largest finite float when it
 * overflows (an amax below about fmax / 3.4e38), so zeros stay +0 and every
 * dequantization factor stays positive. */
typedef enum { LPQ_SCALING_CURRENT = 0, LPQ_SCALING_DELAYED = 1 } lpq_scaling;

/* lpq_quantize flags */
enum {
  LPQ_ROWWISE = 1,     /* emit the row-wise copy [rows, cols] */
  LPQ_COLWISE = 2,     /* emit the column-wise copy [cols, rows] (re-blocked along rows) */
  LPQ_RHT_COLWISE = 4, /* NVFP4: 16-point random-sign Hadamard on the column-wise copy */
  LPQ_STOCHASTIC = 8,  /* NVFP4: stochastic rounding of the E2M1 codes (both copies) */
  LPQ_GIVEN_AMAX = 16  /* per-tensor FP8 (current scaling) and NVFP4: the views' amax fields
                          already hold the amax to scale with (e.g. the MAX over all shards of a
                          token-sharded tensor); no amax pass is run and they are left as given */
};

/* Scale-factor layouts of a copy. */
enum {
  LPQ_SF_PLAIN = 0, /* [rows, cols / block] row-major (FP8 block: FP32 [rows / br, cols / 128]) */
  LPQ_SF_GEMM = 1   /* tensor-core layout read by lpq_gemm (see lpq_copy_bytes) */
};

/* One quantized copy of a matrix.  All pointers are device pointers.
 *   codes        [rows, cols] bytes (FP8 formats), [rows, cols / 2] packed
 *                E2M1 (NVFP4, MXFP4: low nibble = even column), or bf16
 *                [rows, cols].
 *   scales       block scales: u8 E8M0 (MXFP8, MXFP8_E5M2, MXFP4), u8 E4M3
 *                (NVFP4), FP32 scale_inv (FP8 block); NULL for per-tensor FP8
 *                and bf16.  An E8M0 scale s stands for 2^(s - 127), where the
 *                block exponent is the smallest e with fmax * 2^e >= the
 *                block's max |value| (fmax 448 E4M3, 57344 E5M2, 6 E2M1), so
 *                that no code saturates.
 *   tensor_scale one FP32 dequantization factor: scale_inv for per-tensor
 *                FP8, the FP32 tensor scale for NVFP4; NULL otherwise.
 *   amax         one FP32: max |value| of this copy's input values (after the
 *                Hadamard transform for an RHT copy).  Required for per-tensor
 *                FP8 and NVFP4 (lpq_quantize writes it), optional for the MX
 *                formats (written when non-NULL), unused by the others.
 *   rows, cols   dimensions of this copy (the column-wise copy of an
 *                [R, C] tensor is [C, R]).
 *   colwise      1 for a column-wise copy, 0 for a row-wise copy.        */
typedef struct {
  void *codes;
  void *scales;
  float *tensor_scale;
  float *amax;
  int64_t rows, cols;
  int32_t fmt;       /* lpq_format */
  int32_t sf_layout; /* LPQ_SF_PLAIN or LPQ_SF_GEMM */
  int32_t colwise;
  int32_t reserved;
} lpq_qview;

typedef struct {
  lpq_qview row, col;
} lpq_qtensor;

/* Delayed-scaling state of one tensor role ([FP8] amax history; [NeMo]
 * per-tensor delayed scaling).  Device pointers.  Initial state: history all
 * 0, pos 0, scale 1, scale_inv 1.  The state is raw FP32/INT32 arrays, so a
 * checkpoint is a copy of them. */
typedef struct {
  float *amax_history; /* [len] */
  int32_t *pos;        /* next slot of the ring */
  float *scale;        /* scale used by the next quantize */
  float *scale_inv;
  int32_t len;         /* 1..1024; the workloads use 16 */
} lpq_delayed_state;

/* Bytes of one copy's codes and scales for format `fmt`, a copy of `rows` x
 * `cols` and scale layout `sf_layout`.  Host-only, needs no GPU.
 * LPQ_SF_GEMM layout for the MX formats and NVFP4: 128-row groups x KT atoms of 512
 * bytes; atom (g, t) starts at (g * KT + t) * 512 and holds, for row
 * r = 128 g + 32 j + i (i < 32, j < 4), its 4 scales of column-blocks
 * 4t .. 4t+3 at bytes 16 i + 4 j + 0..3.  KT = ceil(cols / 128) for MXFP8
 * and MXFP8_E5M2, 2 * ceil(cols / 256) for MXFP4 and 4 * ceil(cols / 256) for
 * NVFP4; entries beyond the matrix read as 0.
 * LPQ_SF_GEMM for FP8_BLOCK_1x128 is FP32 [cols / 128, rows] (rows fastest);
 * for FP8_BLOCK_128x128 it equals the plain layout. */
lpq_status lpq_copy_bytes(int32_t fmt, int64_t rows, int64_t cols, int32_t sf_layout,
                          size_t *codes_bytes, size_t *scale_bytes);

/* Quantizes x [rows, cols] bf16 (device) into the copies `flags` selects.
 *   fmt            LPQ_FP8_E4M3/E5M2 (with `scaling`), LPQ_MXFP8,
 *                  LPQ_MXFP8_E5M2, LPQ_MXFP4, LPQ_NVFP4, LPQ_NVFP4_2D,
 *                  LPQ_FP8_BLOCK_*, or LPQ_BF16 (row-wise = copy,
 *                  column-wise = transpose).
 *   scaling        per-tensor FP8 only.  CURRENT: scale = fmax / amax(x)
 *                  from an extra amax pass.  DELAYED: scale = *state->scale
 *                  from earlier steps; amax(x) is measured in the same pass
 *                  and written to out->row.amax (or col.amax); the state is
 *                  NOT advanced — call lpq_scale_update with that amax.
 *   seed, counter_offset   stochastic rounding: Philox-4x32-10 key = seed,
 *                  element j of a copy (row-major index + counter_offset)
 *                  uses word j mod 4 of counter (j / 4, copy id, 0).
 *                  counter_offset must be a multiple of 4.
 *   rht_seed       the 16 Hadamard signs: bits of word 0 of
 *                  Philox(key = (rht_seed, 0), counter = (0, 0, 2, 0)).
 *   out            views to fill; out->row used if LPQ_ROWWISE, out->col if
 *                  LPQ_COLWISE.  Each view's rows/cols/fmt must match.
 *                  With LPQ_GIVEN_AMAX the amax of each requested view is an
 *                  input (NVFP4: the row view's the raw amax, the column
 *                  view's the amax of its own values, after the RHT when
 *                  LPQ_RHT_COLWISE is set; FP8: the row view's, else the
 *                  column view's, for both copies).  Quantizing the shards of
 *                  a tensor with the MAX of their amaxes gives exactly the
 *                  codes and scales of the whole tensor (for the row-wise
 *                  copy with stochastic rounding, pass counter_offset =
 *                  first row * cols).
 * Shape rules: cols a multiple of the row-wise block (16 NVFP4, 32 MX formats, 128
 * FP8 block, 16 NVFP4_2D), rows a multiple of the column-wise block when
 * LPQ_COLWISE is set (same numbers; 128x128 needs neither rows nor cols beyond
 * cols % 128 == 0 and rows % 128 == 0 for its column copy), and every row of
 * every output 16-byte aligned.  A 0 x n or n x 0 input is valid and enqueues
 * nothing but the scalar outputs. */
lpq_status lpq_quantize(const void *x, int64_t rows, int64_t cols, int32_t fmt, int32_t scaling,
                        uint32_t flags, uint64_t seed, uint64_t counter_offset, uint32_t rht_seed,
                        const lpq_delayed_state *state, lpq_qtensor *out, lpq_stream_t stream);

/* The global amax pass ([TE] "interpreting real-model results": the extra
 * memory pass for the per-tensor amax; [FP8] per-tensor scaling from the
 * tensor's amax): *amax = max |x| over x [rows, cols] bf16 (NaN ignored,
 * infinities counted), overwritten (not accumulated).  With LPQ_RHT_COLWISE
 * in flags, *rht_amax gets max |RHT16(v)| over the column-wise copy (each
 * column's 16-runs of rows transformed with the signs of rht_seed, as in
 * lpq_quantize), the amax an NVFP4 RHT column copy is scaled with; rows must
 * then be a multiple of 16.  amax and rht_amax are device FP32 pointers;
 * either may be NULL, not both (rht_amax is ignored without the flag).  cols
 * must be a multiple of 16 and x 16-byte aligned; an empty x gives 0.  This is
 * the pass lpq_quantize runs before current-scaled FP8 and NVFP4 copies: a
 * token-sharded caller runs it on its own shard, combines the shards' values
 * with a MAX all-reduce and quantizes with LPQ_GIVEN_AMAX.  flags other than
 * LPQ_RHT_COLWISE give LPQ_ERR_INVALID_ARG. */
lpq_status lpq_amax(const void *x, int64_t rows, int64_t cols, uint32_t flags, uint32_t rht_seed, float *amax,
                    float *rht_amax, lpq_stream_t stream);

/* Delayed-scaling update (one CTA): history[pos] = *amax; pos = (pos+1) % len;
 * m = max(history); scale = fmax / m if m > 0 and finite (else unchanged),
 * clamped to the largest finite float if the quotient overflows;
 * scale_inv = 1 / scale.  fmax is 448 (E4M3) or 57344 (E5M2).  pos should be
 * in [0, len); a value outside is taken modulo len (no write leaves the
 * history). */
lpq_status lpq_scale_update(const lpq_delayed_state *state, const float *amax, float fmax,
                            lpq_stream_t stream);

/* Which copies a GEMM of a linear layer reads ([TE]: Fprop, Dgrad and Wgrad
 * are separate GEMMs).  X [M, K] activations, W [N, K] weights, dY [M, N]:
 *   LPQ_FPROP  Y  = X W^T   : a = X row-wise,   b = W row-wise   -> C [M, N]
 *   LPQ_DGRAD  dX = dY W    : a = dY row-wise,  b = W col-wise   -> C [M, K]
 *   LPQ_WGRAD  dW = dY^T X  : a = dY col-wise,  b = X col-wise   -> C [N, K]
 * The layout only states which copies are expected (checked against the
 * views' `colwise` flags); the arithmetic is the same. */
typedef enum { LPQ_FPROP = 0, LPQ_DGRAD = 1, LPQ_WGRAD = 2 } lpq_layout;

/* C[m, n] = sum_k deq(a)[m, k] * deq(b)[n, k], FP32 accumulation on the
 * tensor cores (tcgen05), output bf16 (c_is_fp32 = 0) or FP32, row-major with
 * leading dimension n.  a is [m, k], b is [n, k], both contiguous along k.
 * Legal pairings: BF16 x BF16; {E4M3, E5M2} x {E4M3, E5M2} (per-tensor,
 * scale_inv product applied in the epilogue); {MXFP8, MXFP8_E5M2} x {MXFP8,
 * MXFP8_E5M2} (E5M2 gradients against E4M3 activations or weights);
 * MXFP4 x MXFP4; {NVFP4,
 * NVFP4_2D} x {NVFP4, NVFP4_2D} (tensor scales in the epilogue); FP8 block
 * (1x128 or 128x128) x FP8 block (FP32 block scales applied per 128-deep
 * slice).  Block-scaled operands must use LPQ_SF_GEMM.  k must be a multiple
 * of 32 (128 for FP8 block); m and n are arbitrary (>= 0).  Anything else
 * returns LPQ_ERR_UNSUPPORTED or LPQ_ERR_SHAPE; nothing falls back. */
lpq_status lpq_gemm(int32_t layout, const lpq_qview *a, const lpq_qview *b, void *c, int32_t c_is_fp32,
                    int64_t m, int64_t n, int64_t k, lpq_stream_t stream);

/* Kernel-path options of lpq_gemm_ex.  They choose between kernels that
 * compute the same result (every path passes the same parity tests); they
 * never change the format, the precision or the arithmetic, and nothing else
 * (no environment variable, no global setting) selects a path.  All-zero is
 * the default path that lpq_gemm takes.
 *   single_cta    0: CTA pairs (cta_group::2, 256 x 256 output tiles) when
 *                 m >= 256, one CTA per 128 x 256 tile otherwise; 1: always
 *                 one CTA per tile.
 *   tile_n        single-CTA block-scaled kinds: 0 or 256 (128 x 256 tiles,
 *                 one TMEM accumulator) or 128 (128 x 128 tiles, two
 *                 accumulators).  Ignored elsewhere.
 *   scale_copies  block-scaled kinds: 0 = the scale factors are written into
 *                 TMEM by four scale warps (tcgen05.st); 1 = copied by the
 *                 MMA-issuing thread (tcgen05.cp).
 *   direct_store  CTA-pair kernel, bf16 output: 0 = TMA tile stores through
 *                 shared memory (when n % 8 == 0); 1 = stores from registers.
 *   whole_tiles   CTA-pair kernel: 0 = when the tiles left for the last round
 *                 of the persistent schedule fill at most half of the CTA
 *                 pairs, each of them runs as two 256 x 128 halves (N = 128
 *                 MMAs) on two pairs, so that the last round takes half as
 *                 long; 1 = whole 256 x 256 tiles only.
 *   reserved      must be 0.
 * Values outside these sets give LPQ_ERR_INVALID_ARG. */
typedef struct {
  int32_t single_cta;
  int32_t tile_n;
  int32_t scale_copies;
  int32_t direct_store;
  int32_t whole_tiles;
  int32_t reserved[3];
} lpq_gemm_opts;

/* lpq_gemm with explicit kernel-path options (NULL = all defaults). */
lpq_status lpq_gemm_ex(int32_t layout, const lpq_qview *a, const lpq_qview *b, void *c, int32_t c_is_fp32,
                       int64_t m, int64_t n, int64_t k, const lpq_gemm_opts *opts, lpq_stream_t stream);

/* ------------------------------------------------------------------------
 * The operators around the linear layers: the norm in front of them, the loss
 * behind the last one, and their product for the few tokens of decoding.
 * Sums, row statistics and softmax statistics are held in FP32. */

/* Element types of the norm's tensors. */
typedef enum { LPQ_TYPE_BF16 = 0, LPQ_TYPE_FP32 = 1 } lpq_type;

/* Layer norm of every row of x [rows, cols] (rows ldx elements apart):
 *   mean = sum(x) / cols,  rstd = 1 / sqrt(sum((x - mean)^2) / cols + eps),
 *   y = (x - mean) * rstd * weight + bias.
 *   x_type       type of x and y; w_type that of weight and bias.
 *   weight, bias [cols]; NULL weight = 1, NULL bias = 0.
 *   y            [rows, cols], rows ldy elements apart; rounded once.
 *   mean, rstd   [rows] FP32, what lpq_layer_norm_backward reads; either may
 *                be NULL.
 *   amax         one FP32, max |y| over the rounded outputs (NaN ignored,
 *                infinities counted, 0 without rows): the value lpq_amax gives
 *                for y, so that lpq_quantize with LPQ_GIVEN_AMAX needs no amax
 *                pass.  NULL: not computed.
 * Any rows >= 0, cols >= 1, ldx and ldy >= cols and eps >= 0.  Pointers need
 * their element's alignment; 16-byte aligned rows (of x and y) of a multiple
 * of 16 bytes, with 16-byte aligned weight and bias, take 16-byte accesses.  x
 * and y must not overlap. */
lpq_status lpq_layer_norm(const void *x, int64_t ldx, int32_t x_type, const void *weight, const void *bias,
                          int32_t w_type, int64_t rows, int64_t cols, float eps, void *y, int64_t ldy, float *mean,
                          float *rstd, float *amax, lpq_stream_t stream);

/* Bytes of lpq_layer_norm_backward's workspace (16-byte aligned device
 * memory).  Host-only. */
lpq_status lpq_layer_norm_workspace(int64_t rows, int64_t cols, size_t *bytes);

/* Backward pass of lpq_layer_norm from dy [rows, cols] and the forward's x,
 * mean and rstd.  With xhat = (x - mean) * rstd and g = dy * weight:
 *   dx      = rstd * (g - sum(g) / cols - xhat * sum(g * xhat) / cols)
 *   dweight = sum over the rows of dy * xhat,  dbias = that of dy   (FP32)
 * dx has x's type and rows lddx elements apart.  dweight and dbias may be
 * NULL.  The sums over the rows are split into a fixed number of parts joined
 * in a fixed order: the same inputs give the same bits.  Alignment as for
 * lpq_layer_norm; dy, x and dx must not overlap.  0 rows give zero gradients. */
lpq_status lpq_layer_norm_backward(const void *dy, int64_t lddy, const void *x, int64_t ldx, int32_t x_type,
                                   const float *mean, const float *rstd, const void *weight, int32_t w_type,
                                   int64_t rows, int64_t cols, void *dx, int64_t lddx, float *dweight, float *dbias,
                                   void *workspace, size_t workspace_bytes, lpq_stream_t stream);

/* Softmax cross entropy of a vocabulary projection, logits not kept.  For
 * hidden states h [t, d] and weights w [v, d] (bf16, rows ldh / ldw elements
 * apart) and the logits l = h w^T (FP32):
 *   lse[i]  = log(sum_j exp(l[i, j])),   loss[i] = lse[i] - l[i, labels[i]].
 * labels [t] are int64; a label outside 0 .. v - 1 (-100, say) marks a row
 * without target: its loss is 0 and its gradients vanish, its lse is computed.
 * Any t >= 0, v >= 1; d >= 8 a multiple of 8; ldh and ldw >= d multiples of 8;
 * h, w and the workspace 16-byte aligned.  A row whose logits hold a NaN has
 * lse NaN; one with a +infinity has lse +infinity.  The exponentials are taken of
 * differences from the row's largest logit, the loss too: it is as near for a
 * confident token (2^-21 of 1 + loss, beside the logits' own error) as for others,
 * and never negative. */
lpq_status lpq_linear_ce(const void *h, int64_t ldh, const void *w, int64_t ldw, const int64_t *labels, int64_t t,
                         int64_t v, int64_t d, float *loss, float *lse, void *workspace, size_t workspace_bytes,
                         lpq_stream_t stream);

/* Gradients of sum_i dloss[i] * loss[i]: with the forward's lse and
 *   dl[i, j] = dloss[i] * (exp(l[i, j] - lse[i]) - (j == labels[i]))
 * (0 in rows without target, whatever their h, dloss and lse hold; such rows are
 * left out of the work)
 *   dh [t, d] = dl w,   dw [v, d] = dl^T h,
 * contiguous, bf16 (grads_fp32 = 0) or FP32.  The logits are computed again,
 * vocab_piece words at a time (0: the library's choice; else a positive
 * multiple of 64), so that only t * vocab_piece values of dl exist at once.
 * They are divided by max |dloss| and rounded to bf16, which the tensor cores
 * read (where up to 128 rows have a target: held as the sum of two bf16 terms;
 * beyond, FP32 gradients too carry that rounding, 2^-9 of each value, unless two
 * terms are asked for by lpq_linear_ce_backward_ex); all sums are FP32 and the
 * factor is put back before the final rounding.  The same inputs give the same
 * bits.  0 rows give dw = 0.  dh and dw must be 16-byte aligned. */
lpq_status lpq_linear_ce_backward(const void *h, int64_t ldh, const void *w, int64_t ldw, const int64_t *labels,
                                  const float *lse, const float *dloss, int64_t t, int64_t v, int64_t d, void *dh,
                                  void *dw, int32_t grads_fp32, int64_t vocab_piece, void *workspace,
                                  size_t workspace_bytes, lpq_stream_t stream);

/* Options of lpq_linear_ce_backward_ex (all zero: lpq_linear_ce_backward).
 *   two_terms   1: each value of dl as the sum of two bf16 terms (16 bits) for
 *               any number of rows, at 10 t v d operations instead of 6 beyond
 *               128 rows; 0: up to 128 rows with a target alone.
 *   reserved    must be 0. */
typedef struct {
  int32_t two_terms;
  int32_t reserved[3];
} lpq_ce_opts;

/* lpq_linear_ce_backward with explicit options (NULL = all defaults). */
lpq_status lpq_linear_ce_backward_ex(const void *h, int64_t ldh, const void *w, int64_t ldw, const int64_t *labels,
                                     const float *lse, const float *dloss, int64_t t, int64_t v, int64_t d, void *dh,
                                     void *dw, int32_t grads_fp32, int64_t vocab_piece, void *workspace,
                                     size_t workspace_bytes, const lpq_ce_opts *opts, lpq_stream_t stream);

/* Workspace bytes of lpq_linear_ce (backward = 0) and lpq_linear_ce_backward
 * (backward = 1, or 2 with the option two_terms; with the same vocab_piece).
 * Host-only. */
lpq_status lpq_linear_ce_workspace(int64_t t, int64_t v, int64_t d, int32_t backward, int64_t vocab_piece,
                                   size_t *bytes);

/* y[i, n] = sum_k x[i, k] * deq(w)[n, k] for a few tokens i on 4-bit weights:
 * w is a row-wise copy [n, k] of NVFP4, NVFP4_2D or MXFP4 as lpq_quantize
 * writes it (either scale layout; codes 16-byte aligned, scales 4-byte
 * aligned), x [m, k] is bf16 and not quantized (rows ldx elements apart, ldx
 * a multiple of 8, 16-byte aligned), y [m, n] contiguous bf16 or FP32, 16-byte
 * aligned.  Codes times scales are exact (a code of zero is 0 beside any finite
 * scale), products are summed in FP32 and the tensor scale is applied to the sum.  k must be a multiple of 32, at most 2^19 (2^16 with
 * LPQ_SF_PLAIN scales); m and n are arbitrary
 * (>= 0), but m is meant to be small: the weights are read once per 8 tokens. */
lpq_status lpq_matvec(const lpq_qview *w, const void *x, int64_t ldx, int64_t m, void *y, int32_t y_is_fp32,
                      lpq_stream_t stream);

/* Low-rank adapters of one linear layer: pair e is a[e] [rank, k] and b[e] [n, rank]
 * (bf16, contiguous, 16-byte aligned), rank a multiple of 8 up to 256 (smaller ones
 * are padded with zeros); scale [count] FP32, NULL = 1. */
typedef struct {
  const void *a, *b;
  const float *scale;
  int64_t count, rank;
} lpq_adapters;

/* lpq_matvec with an adapter for every token:
 *   y[i, n] = sum_k x[i, k] * deq(w)[n, k] + scale[e] * sum_r b[e][n, r] * (sum_k
 *             a[e][r, k] * x[i, k]),   e = index[i]
 * index [m] int64, device; outside 0 .. count - 1: no adapter.  The inner vector and
 * all sums are FP32, y is rounded once.  The workspace (16-byte aligned device
 * memory) is written before it is read. */
lpq_status lpq_matvec_adapted(const lpq_qview *w, const void *x, int64_t ldx, int64_t m, void *y, int32_t y_is_fp32,
                              const lpq_adapters *adapters, const int64_t *index, void *workspace, size_t workspace_bytes,
                              lpq_stream_t stream);

/* Bytes of lpq_matvec_adapted's workspace.  Host-only. */
lpq_status lpq_matvec_adapted_workspace(int64_t m, int64_t rank, size_t *bytes);

/* A mixture-of-experts layer for a few tokens.  The router: with the logits l = x w^T
 * (FP32) of x [m, d] and w [experts, d] (bf16, rows ldx and ldw elements apart),
 *   ids [m, k] int64: the k largest in descending order (equal ones: the lower index
 *   first; NaN below everything),
 *   probs [m, k] FP32: the softmax over the chosen (renormalize = 1) or over all
 *   (renormalize = 0) at those places.
 * d is a multiple of 8 up to 65536, ldx and ldw multiples of 8, x and w 16-byte
 * aligned; 1 <= k <= 32, k <= experts <= 1024; 0 <= m <= 2^30 - 4 (made for few). */
lpq_status lpq_moe_route(const void *x, int64_t ldx, const void *w, int64_t ldw, int64_t m, int64_t d, int64_t experts,
                         int64_t k, int32_t renormalize, int64_t *ids, float *probs, lpq_stream_t stream);

/* The experts' products: for token i
 *   y[i] = sum_j probs[i, j] * W2_e (silu(W1g_e x[i]) * (W1u_e x[i])),   e = ids[i, j]
 * on 4-bit weights (NVFP4, NVFP4_2D or MXFP4, row-wise copies with LPQ_SF_GEMM scales):
 *   up    [experts * 2 f, d]: each expert's f gate rows, then its f up rows;
 *   down  [experts * d, f].
 * x [m, d] bf16 (rows ldx elements apart, a multiple of 8; 16-byte aligned), not
 * quantized; ids [m, k] int64 (outside 0 .. experts - 1: the place counts for nothing;
 * one expert may stand twice), probs [m, k] FP32; y [m, d] bf16, contiguous.  Sums are
 * FP32; hidden values enter the second product off by at most 2^-22 of themselves or
 * 2^-39 of their vector's largest; y is rounded once, its sum taken in the order of j.
 * d and f are multiples of 32 up to 65536; 0 <= k <= 32, experts <= 1024; any m >= 0, but m is meant
 * to be small: an expert's weights are read once for up to 8 of its tokens. */
lpq_status lpq_moe(const lpq_qview *up, const lpq_qview *down, int64_t experts, const void *x, int64_t ldx, int64_t m,
                   const int64_t *ids, const float *probs, int64_t k, void *y, void *workspace, size_t workspace_bytes,
                   lpq_stream_t stream);

/* Bytes of lpq_moe's workspace (16-byte aligned device memory; written before it is
 * read).  Host-only. */
lpq_status lpq_moe_workspace(int64_t m, int64_t k, int64_t d, int64_t f, size_t *bytes);

/* RMS norm of every query and key head with the position rotation, behind the
 * QKV projection.  x [rows, >= (q_heads + k_heads) * head_dim] holds a token's
 * query heads, then its key heads (rows ldx elements apart; what lies behind the
 * key heads is not touched).  Of every head, with w the query or key weight:
 *   n = x * rstd * w,  rstd = 1 / sqrt(sum(x^2) / head_dim + eps),
 *   pair i < rotary_dim / 2 turned by a = positions[row] * freqs[i]:
 *     (y1, y2) = (n1 cos a - n2 sin a, n2 cos a + n1 sin a).
 *   type         of x and y; w_type that of the weights.
 *   q_weight, k_weight  [head_dim], one for all heads; NULL = 1.
 *   positions    [rows] int64, device.
 *   freqs        [rotary_dim / 2] radians per position, HOST memory, read before
 *                the call returns (base^(-2 i / rotary_dim) by custom); finite.
 *   interleaved  0: the pairs are values i and i + rotary_dim / 2 of the head;
 *                1: values 2 i and 2 i + 1.  Values from rotary_dim on are not
 *                turned.
 *   y            rows ldy elements apart, same heads; y may be x itself (then
 *                ldy = ldx), else they must not overlap.
 * Angles are reduced modulo a turn in integers: off by at most 1e-7 radians (they are
 * rounded to 2^-26 turns) and 2^-52 |position freqs[i]|; any int64 position is valid.
 * Statistics are FP32 and y is rounded once: squares beyond that range (values from 2^60
 * on; with eps = 0 below 2^-60, too) are not those of the formula.  head_dim is even, 2 ..
 * 512; rotary_dim even, 0 .. head_dim; any rows, heads >= 0; eps >= 0.  Rows
 * that begin at 16 bytes, with head_dim and rotary_dim multiples of 16 values (FP32:
 * 8; interleaved: rotary_dim of 4), take 16-byte accesses; bf16 with 8 in place of 16
 * takes 8-byte ones; others go value by value. */
lpq_status lpq_qk_norm_rope(const void *x, int64_t ldx, int32_t type, int64_t rows, int64_t q_heads, int64_t k_heads,
                            int64_t head_dim, const void *q_weight, const void *k_weight, int32_t w_type,
                            const int64_t *positions, const double *freqs, int64_t rotary_dim, int32_t interleaved,
                            float eps, void *y, int64_t ldy, lpq_stream_t stream);

/* Bytes of lpq_qk_norm_rope_backward's workspace (16-byte aligned device memory).
 * Host-only. */
lpq_status lpq_qk_norm_rope_workspace(int64_t rows, int64_t head_dim, size_t *bytes);

/* Backward pass of lpq_qk_norm_rope from dy and the forward's x.  With g = dy
 * turned by -a:
 *   dx = rstd * (g * w - x * rstd^2 * sum(g * w * x) / head_dim),
 *   dq_weight = sum over rows and query heads of g * x * rstd, dk_weight over the
 *   key heads (FP32; either may be NULL, no workspace is needed without both).
 * dx may be dy or x itself (with its leading dimension), else they must not
 * overlap.  The sums are split into parts by sizes and joined in a fixed order:
 * the same inputs give the same bits.  0 rows or heads give zero gradients. */
lpq_status lpq_qk_norm_rope_backward(const void *dy, int64_t lddy, const void *x, int64_t ldx, int32_t type, int64_t rows,
                                     int64_t q_heads, int64_t k_heads, int64_t head_dim, const void *q_weight,
                                     const void *k_weight, int32_t w_type, const int64_t *positions, const double *freqs,
                                     int64_t rotary_dim, int32_t interleaved, float eps, void *dx, int64_t lddx,
                                     float *dq_weight, float *dk_weight, void *workspace, size_t workspace_bytes,
                                     lpq_stream_t stream);

/* What changes the logits of the next words.  Device pointers; any group may be
 * NULL, which leaves its step out.
 *   history      [rows, max_len <= 2^30] int64 words of every request's context, rows
 *                ld_history elements apart: lengths[row] of them (taken within 0 ..
 *                max_len), of which the first prompt[row] (NULL: 0) are the prompt
 *                and the others the answer so far.  Words outside 0 .. v - 1 count
 *                for nothing.  lengths goes with it.
 *   repetition   [rows]: a word of the context has its logit divided by r where it
 *                is positive and multiplied by r elsewhere.
 *   frequency, presence  [rows]: a word that stands c > 0 times in the answer loses
 *                frequency * c + presence.
 *   bias_offsets [rows + 1], bias_words [bias_count] int64, bias_values
 *                [bias_count]: entries bias_offsets[row] .. bias_offsets[row + 1] - 1
 *                (taken within 0 .. bias_count) are added to their words' logits,
 *                those of one word in the list's order.
 *   allowed      [rows, ceil(v / 32)] int32, rows ld_allowed elements apart: bit j %
 *                32 of element j / 32 says whether word j may follow; the others get
 *                -infinity, whatever they held (a row without a bit: all of them).
 * The penalties need a history; the history has no effect without them. */
typedef struct {
  const int64_t *history;
  int64_t ld_history, max_len;
  const int64_t *lengths, *prompt;
  const float *repetition, *frequency, *presence;
  const int64_t *bias_offsets, *bias_words;
  const float *bias_values;
  int64_t bias_count;
  const int32_t *allowed;
  int64_t ld_allowed;
} lpq_logit_controls;

/* out = the logits [rows, v] (type lpq_type, rows ld elements apart) under the
 * controls, in the order repetition, frequency and presence, bias, mask; FP32
 * arithmetic, rounded once.  out has the logits' type, rows ldo elements apart, and
 * may be the logits themselves (then ldo = ld), else they must not overlap.  Any
 * rows and v >= 0, v at most 2^30; rows that begin equally far from a 16-byte
 * boundary on both sides take 16-byte accesses. */
lpq_status lpq_adjust_logits(const void *logits, int64_t ld, int32_t type, int64_t rows, int64_t v,
                             const lpq_logit_controls *controls, void *out, int64_t ldo, lpq_stream_t stream);

/* Transformer configuration ([TE] "model configuration and training input"). */
typedef struct {
  int64_t hidden, intermediate, heads, layers, micro_batch, seq;
} lpq_transformer_cfg;

typedef struct {
  char name[24];   /* e.g. "qkv_fprop" */
  int32_t layout;  /* lpq_layout */
  int64_t m, k, n; /* C [m, n] = sum over k */
} lpq_gemm_shape;

/* The 12 GEMMs of one layer: M = micro_batch * seq; QKV (K = hidden,
 * N = 3 hidden), attention out (hidden, hidden), MLP up (hidden,
 * intermediate), MLP down (intermediate, hidden), each as Fprop (M, K, N),
 * Dgrad (M, N, K) and Wgrad (N, M, K).  `heads` and `layers` do not change
 * the linear shapes.  Host-only. */
lpq_status lpq_layer_shapes(const lpq_transformer_cfg *cfg, lpq_gemm_shape out[12], int32_t *count);

/* Text of the last non-OK status on this thread ("" if none). */
const char *lpq_last_error(void);

/* Synchronises `stream`, then reads and clears the device error word that
 * kernels set when a bounded wait gives up (0 = none, else an lpq_status). */
lpq_status lpq_device_status(lpq_stream_t stream, int32_t *code);

/* Failure-detection check: launches one CTA whose bounded wait (the same
 * helper the GEMM pipeline uses) waits on a barrier that nothing completes.
 * After limit_ns (0 < limit_ns <= 1 s) the wait gives up and records
 * LPQ_ERR_TIMEOUT in the device error word, which lpq_device_status then
 * returns; the CUDA context stays usable.  No fault, trap or hang is involved. */
lpq_status lpq_selftest_wait(uint64_t limit_ns, lpq_stream_t stream);

/* Arithmetic self-check of the quantizers' device helpers against their
 * definitions, for the test suite.  Counts mismatches over indices i in
 * [begin, begin + count):
 *   which 0: x = the float with bits i (i <= 0x7F800000: every non-negative
 *            float and +inf): the block-max division by 6 (a product with
 *            RN(1/6) corrected by one fused multiply-add of the exact
 *            residual) against the IEEE quotient x / 6;
 *   which 1: |y| = the float with bits i >> 3 and the (i & 7)-th of eight
 *            probe words r (r >> 8 = 0, 1, 2^23 - 2, 2^23, 2^24 - 3,
 *            2^24 - 2, 2^24 - 1, 2^24 - 1, low bytes 0x00 or 0xFF): the
 *            stochastic E2M1 rounding of y and -y against the definition
 *            (round up to the next grid magnitude iff float(r >> 8) <
 *            frac * 2^24; 6 at and beyond 6 and for NaN);
 *   which 2: y = the float with bits `param` and r = i << 8 | (i * 37 mod
 *            256), i < 2^24 (every threshold value for one y), y and -y.
 * result (device, two int64, 8-byte aligned) receives the mismatch count and
 * the smallest mismatching index (-1 if none); the call returns at once, read
 * result after synchronising `stream`.  Ranges beyond the mode's index limit
 * give LPQ_ERR_INVALID_ARG. */
lpq_status lpq_selftest_arith(int32_t which, uint64_t begin, uint64_t count, uint32_t param, int64_t *result,
                              lpq_stream_t stream);

/* Tensor-core rate measurement (the dense peaks the roofline divides by):
 * one CTA per SM issues `iters` k-steps of four 128 x 256 tcgen05.mma on
 * zero operands resident in shared memory; kind 0 = kind::f16 (bf16, K 16),
 * 1 = kind::f8f6f4 (E4M3, K 32), 2 = MXFP8 block-scaled (K 32), 3 = NVFP4
 * block-scaled (K 64).  with_scale_copies adds the per-step tcgen05.cp of the
 * scale factors (kinds 2, 3): 1 = all of a step's copies before its MMAs,
 * 2 = the same into two alternating TMEM regions, 3 = each MMA's copies
 * right before it, 4 = the scale columns rewritten by four other warps with
 * tcgen05.st while the MMAs run, 5 = the step's copies issued by a thread of
 * another warp while the MMAs run (4 and 5: NVFP4 only, unsynchronised with
 * the MMAs, throughput only), 6 = CTA pairs (cta_group::2: clusters of two
 * CTAs, each pair issuing four 256 x 256 MMAs per k-step, each SM holding
 * 128 rows of A and of B, the shape of the product GEMM; any kind), 7 = CTA
 * pairs with the scale columns rewritten by four warps per CTA with
 * tcgen05.st while the MMAs run (kinds 2, 3), 8 = CTA pairs issuing each
 * k-step as eight 256 x 128 MMAs (two column halves into two TMEM regions;
 * any kind).  Other values give LPQ_ERR_INVALID_ARG.  Modes 6 to 8 launch SMs
 * rounded down to even CTAs.
 * FLOPs = CTAs * iters * 4 * 2 * 128 * 256 * K;
 * the caller times the launch with events on `stream`. */
lpq_status lpq_mma_peak(int32_t kind, int32_t iters, int32_t with_scale_copies, lpq_stream_t stream);

/* Library version (major * 10000 + minor * 100 + patch). */
int32_t lpq_version(void);

#ifdef __cplusplus
}
#endif
#endif /* LPQ_H_ */
