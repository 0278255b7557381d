/*
 * opt_layer.h -- C ABI of the training-layer operators of the GB300 (sm_103a)
 * optimizer-step library: what makes the gradients that opt.h's calls consume,
 * in the same low-precision form.
 *
 *   opt_dropout            dropout from the counter-based generator, with the
 *                          residual's addition; the mask is never stored
 *   opt_rms_norm           branch dropout, residual sum, root-mean-square norm
 *                          and 8-bit output with block scales, in one pass
 *   opt_rms_norm_backward  its gradients
 *   opt_quantize           a matrix to E4M3 codes with a scale for each block
 *                          of 128, in one or both orientations
 *   opt_matmul             the product of two matrices held in that form
 *
 * Conventions (as in opt.h): pointers named d_* are device pointers on the
 * current device; `stream` is a cudaStream_t as void*.  Calls are
 * stream-ordered, never synchronise, allocate nothing, keep nothing between
 * calls and may be captured into a CUDA graph.  Arguments are validated on the
 * host before any launch; failures return a negative status and launch
 * nothing.  There is no CPU fallback.  Results are bit-identical run to run.
 *
 * Matrices are row-major with a pitch: element (r, c) of a matrix at d_t with
 * pitch t_pitch is d_t[r * t_pitch + c], t_pitch >= cols (not looked at for
 * fewer than two rows).  Plain matrices need only the alignment of their
 * element; 16-byte aligned rows are faster.  Rows, columns and depths may each
 * be 0 (an empty output is a no-op; a product over a depth of 0 is the addend
 * or zero) and are at most 2^31 - 1 (OPT_ELIMIT).
 *
 * Codes: an 8-bit operand of rows x cols is a matrix of E4M3 bytes, 16-byte
 * aligned with a pitch that is a multiple of 16 (OPT_EALIGN), and its scales.
 * Rows that start on 128 bytes are faster in products.
 *
 * Scales: each block of 1 x 128 elements along a row (the row's last block
 * may be shorter), or of 128 x 128 (block_rows 128), has the scale 2^e with e
 * the smallest integer, not below -127, for which the block's largest finite
 * magnitude is at most 448 * 2^e.  The block's codes are the elements over 2^e
 * rounded to nearest (ties to even); an infinity or NaN is stored as NaN, so
 * that it reaches the gradient norm's count.  A scale is held as the byte
 * e + 127 for every one of its block's rows, in tiles of 128 rows by 4 blocks
 * (512 bytes, the tiles of 128 rows one after another): with B =
 * ceil(cols / 128), the byte of row r, block b is at
 *   512 * ((r / 128) * ceil(B / 4) + b / 4)
 *       + 16 * (r mod 32) + 4 * ((r / 32) mod 4) + b mod 4,
 * opt_scales_bytes(rows, cols) bytes in all, 16-byte aligned.  This is the
 * order in which the tensor core's scale memory takes them, so a product
 * copies a tile as it is.  Bytes of rows and blocks beyond the matrix are
 * neither written nor used.
 *
 * Dropout: element i of a rows x cols matrix (i = r * cols + c, whatever the
 * pitch) is kept iff its 16-bit draw is at least T = 65536 p rounded to the
 * nearest integer, and a kept element is multiplied by 65536 / (65536 - T), so
 * that the expectation is exact for the rounded probability.  Draws come from
 * opt.h's generator, eight elements per Philox4x32-10 call as in opt_encode:
 * key = seed, counter = (g low 32, g high 32 | 2^31, tensor index, step low
 * 32) for g = i / 8; element 8g + j takes word j / 2, its low half for even j
 * and its high half for odd j.  The set top bit keeps these draws apart from
 * those that round optimizer states under the same seed.
 */
#ifndef PS_OPT_LAYER_H
#define PS_OPT_LAYER_H

#include "opt.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Bytes of the scale tiles of a rows x cols operand; a negative status for a
 * negative size. */
int64_t opt_scales_bytes(int64_t rows, int64_t cols);

/* y = residual + dropout(x) (residual NULL: no addition).  x, residual and y
 * are of `dtype` (OPT_F32 or OPT_BF16), formed in fp32 and rounded once.  y may
 * be x or residual themselves (same pointer and pitch).  The backward pass is
 * the same call on the gradient, without a residual.  0 <= p <= 1. */
typedef struct opt_dropout_args {
  const void* d_x;
  const void* d_residual;
  void* d_y;
  int64_t x_pitch, residual_pitch, y_pitch;
  int64_t rows, cols;
  double p;
  uint64_t seed;
  int64_t step;              /* >= 0 */
  uint32_t tensor_index;
  int32_t dtype;
} opt_dropout_args;
int opt_dropout(const opt_dropout_args* a, void* stream);

/* Per row, in fp32 with one rounding of each output:
 *   h = residual + dropout(x)       (residual NULL: h = dropout(x); p 0: no dropout)
 *   rstd = 1 / sqrt(mean(h^2) + eps)
 *   y = h rstd weight
 * written to any of d_h, d_y (of `dtype`), d_rstd (fp32 per row) and d_codes with
 * d_scales (y as E4M3 with a scale for each 1 x 128); at least one of them is
 * given.  y and the codes come from h and y before they are rounded to `dtype`.
 * d_h may be d_x or d_residual (same pointer and pitch); the other outputs
 * overlap no input.  eps >= 0.  The sum of h^2 is held in fp32: a NaN in h makes
 * its whole row NaN; an infinity, or values whose squares add up beyond fp32
 * (about 1.8e19 / sqrt(cols) each), make rstd 0; a row of zeros with eps 0 gives
 * NaN. */
typedef struct opt_rms_norm_args {
  const void* d_x;
  const void* d_residual;
  const void* d_weight;      /* cols elements of weight_dtype */
  void* d_h;
  void* d_y;
  float* d_rstd;
  void* d_codes;
  void* d_scales;
  int64_t x_pitch, residual_pitch, h_pitch, y_pitch, codes_pitch;
  int64_t rows, cols;
  double p;
  uint64_t seed;
  int64_t step;
  uint32_t tensor_index;
  int32_t dtype;             /* OPT_F32 or OPT_BF16 */
  int32_t weight_dtype;      /* OPT_F32 or OPT_BF16 */
  float eps;
} opt_rms_norm_args;
int opt_rms_norm(const opt_rms_norm_args* a, void* stream);

/* Gradients of opt_rms_norm from dy (the gradient of y), the stored h and rstd:
 *   g = dy weight
 *   dh = rstd (g - h rstd^2 mean(g h)) + dh_in     (dh_in NULL: 0), the residual's gradient
 *   dx = dropout(dh), same draws                   (d_dx NULL: not wanted)
 *   dweight = sum over rows of dy h rstd           (d_dweight NULL: not wanted), fp32
 * in fp32, each rounded once (dx from dh before its rounding).  d_dh may be d_dy
 * or d_dh_in (same pointer and pitch).  The sum over rows runs in a fixed order;
 * it needs d_workspace of opt_rms_norm_backward_workspace(rows, cols) bytes,
 * 16-byte aligned, when d_dweight is given (none for few rows: 0 bytes). */
typedef struct opt_rms_norm_backward_args {
  const void* d_dy;
  const void* d_h;
  const void* d_weight;
  const float* d_rstd;
  const void* d_dh_in;
  void* d_dh;
  void* d_dx;
  float* d_dweight;
  void* d_workspace;
  int64_t dy_pitch, h_pitch, dh_in_pitch, dh_pitch, dx_pitch;
  int64_t workspace_bytes;
  int64_t rows, cols;
  double p;
  uint64_t seed;
  int64_t step;
  uint32_t tensor_index;
  int32_t dtype;
  int32_t weight_dtype;
  int32_t reserved;          /* 0 */
} opt_rms_norm_backward_args;
int opt_rms_norm_backward(const opt_rms_norm_backward_args* a, void* stream);
int64_t opt_rms_norm_backward_workspace(int64_t rows, int64_t cols);

/* x (rows x cols, OPT_F32 or OPT_BF16) to E4M3 codes and scales, blocks of
 * block_rows x 128 (block_rows 1 or 128): as it is (d_codes, d_scales) and/or
 * transposed (d_codes_t of cols x rows and d_scales_t, blocks along the rows of
 * x, as the products of a backward pass contract them).  Each pair is given
 * whole or left NULL; at least one is given. */
typedef struct opt_quantize_args {
  const void* d_x;
  void* d_codes;
  void* d_scales;
  void* d_codes_t;
  void* d_scales_t;
  int64_t x_pitch, codes_pitch, codes_t_pitch;
  int64_t rows, cols;
  int32_t dtype;
  int32_t block_rows;
} opt_quantize_args;
int opt_quantize(const opt_quantize_args* a, void* stream);

/* out[m][n] = sum over k of a[m][k] b[n][k] (+ addend[m][n]): both operands
 * with k along their rows, as codes with scales.  Products are exact, and sums are
 * held in fp32.  The tensor core truncates where an fp32 addition rounds, once per
 * 32 of the depth, so the error grows with it: about 6e-7 of the output's norm at a
 * depth of 8191, 1.3e-7 for sums that round.  out and addend are of out_dtype
 * (OPT_F32 or OPT_BF16), rounded once.  d_addend may be d_out (same pitch).  A linear layer's three products
 * are y = x W^T (a = x, b = W), dx = dy W (a = dy, b = W transposed) and
 * dW = dy^T x (a = dy transposed, b = x transposed). */
typedef struct opt_matmul_args {
  const void* d_a;           /* m x k codes */
  const void* d_a_scales;
  const void* d_b;           /* n x k codes */
  const void* d_b_scales;
  const void* d_addend;
  void* d_out;
  int64_t a_pitch, b_pitch, addend_pitch, out_pitch;
  int64_t m, n, k;
  int32_t out_dtype;
  int32_t flags;             /* OPT_MATMUL_* bits; others must be 0 */
} opt_matmul_args;
int opt_matmul(const opt_matmul_args* a, void* stream);

/* Wait drill: make the product's bounded waits run out on purpose (after 1 ms,
 * with no fault), so that a caller can test its handling of
 * OPT_FLAG_WAIT_TIMEOUT.  No operand is loaded and nothing is written.
 * OPT_EUNSUPPORTED where a product waits on nothing (an operand of at most eight
 * rows, a depth of 0). */
#define OPT_MATMUL_WAIT_DRILL 1

/* The form in which opt_matmul computes these sizes on the current device, for
 * tests and reports: h_form[0] CTAs that share a tile (1, or 2 for a pair; 0 where
 * no tiles are formed: an operand of at most eight rows, a depth of 0, no output),
 * [1] the tile's columns (its rows are 128 for each CTA), [2] the parts in which a
 * cluster of CTAs takes the depth, [3] 1 if the tile's rows are those of b, [4] the
 * most tiles that a CTA or pair goes through.  Reads a's sizes, and of d_a, d_b and
 * their pitches only whether rows start on 128 bytes; launches nothing. */
int opt_matmul_form(const opt_matmul_args* a, int32_t h_form[5]);

/* Error flags raised by the current device's layer kernels since the last call,
 * on any stream, then cleared; 0 means that every kernel that ended before ran to
 * completion.  A flag raised during the call is in its answer or in the next
 * one's.  Copies to host and synchronises the stream.  OPT_FLAG_WAIT_TIMEOUT: a product gave up a wait on
 * its own copies or tensor-core work (each is bounded at 2 s, so the kernel never
 * hangs) and left part of its output unwritten: discard that output. */
int opt_layer_status(int32_t* h_flags, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* PS_OPT_LAYER_H */
