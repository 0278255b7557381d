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
 *   opt_gated              the gated activation between two products, with 8-bit
 *                          output and its inputs kept in 8 bits
 *   opt_gated_backward     its gradients, from the kept inputs or plain ones
 *   opt_dequantize         kept codes as plain values, or turned into the
 *                          operand of a weight's gradient
 *   opt_head_norm          the norm of each query and key head with the position
 *                          rotation, and the heads kept in 8 bits
 *   opt_head_norm_backward its gradients, from the kept heads or plain ones
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
 * Kept activations: what a forward pass leaves for the backward pass may be held
 * as such an operand with blocks of 1 x 128 (a byte and 1/128 for an element of two
 * or four); the backward calls take it in place of the plain matrix, and their
 * gradients are those of the values that the codes stand for (code times 2^e; a scale
 * byte of 255 stands for NaN).
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

/* What a kept rows x cols matrix (codes, scales) becomes in the backward pass:
 *   d_x                   its values, of `dtype` (OPT_F32: exact)
 *   d_codes_t, d_scales_t its transposed operand (cols x rows), with blocks of 128
 *                         along the matrix's rows.  The values are powers of two
 *                         apart from their codes, so a code changes only where it
 *                         falls among the subnormal ones of a column's scale.
 * At least one is given; a pair is given whole.  A value beyond fp32 is an infinity. */
typedef struct opt_dequantize_args {
  const void* d_codes;
  const void* d_scales;
  void* d_x;
  void* d_codes_t;
  void* d_scales_t;
  int64_t codes_pitch, x_pitch, codes_t_pitch;
  int64_t rows, cols;
  int32_t dtype;             /* of x: OPT_F32 or OPT_BF16 */
  int32_t reserved;          /* 0 */
} opt_dequantize_args;
int opt_dequantize(const opt_dequantize_args* a, void* stream);

/* Activations f(g) = g s(g) of opt_gated, formed in fp32 (a NaN stays one; minus
 * infinity gives NaN, except OPT_ACT_RELU, which gives 0):
 *   OPT_ACT_SILU       s(g) = 1 / (1 + exp(-g))
 *   OPT_ACT_GELU_TANH  s(g) = (1 + tanh(sqrt(2 / pi) (g + 0.044715 g^3))) / 2
 *   OPT_ACT_GELU       s(g) = the normal distribution function
 *   OPT_ACT_RELU       f(g) = max(g, 0)
 * For BF16 matrices s and exp(-g^2 / 2) are 0 where they are below 2^-126 (SiLU is 0 below
 * -87.3), and errors are a few 2^-24 of the value, up to 150 of them where s is near 2^-126;
 * for OPT_F32 subnormal numbers are kept, and errors are at most 8 (SiLU) and 17 (GELU) 2^-24
 * of f, and 6 |z| more for its tanh form, z being what its s is the logistic function of (20
 * at g = -4, 200 at -10: fp32 rounds z). */
#define OPT_ACT_SILU      0
#define OPT_ACT_GELU_TANH 1
#define OPT_ACT_GELU      2
#define OPT_ACT_RELU      3

/* y = f(gate) up (up NULL: y = f(gate)), formed in fp32 and written to d_y (of
 * `dtype`, as gate and up are) and/or d_codes with d_scales (y as E4M3 with a scale
 * for each 1 x 128, from y before it is rounded).  d_gate_codes with d_gate_scales and
 * d_up_codes with d_up_scales keep the inputs for the backward pass.  At least one
 * output is given; a pair is given whole.  d_y may be d_gate or d_up (same pointer
 * and pitch); the other outputs overlap no input.  Fastest: cols a multiple of 8, plain
 * matrices whose rows start on 16 bytes, and gate and up both kept or neither (one of
 * them takes half as long again as both). */
typedef struct opt_gated_args {
  const void* d_gate;
  const void* d_up;
  void* d_y;
  void* d_codes;
  void* d_scales;
  void* d_gate_codes;
  void* d_gate_scales;
  void* d_up_codes;
  void* d_up_scales;
  int64_t gate_pitch, up_pitch, y_pitch, codes_pitch, gate_codes_pitch, up_codes_pitch;
  int64_t rows, cols;
  int32_t dtype;             /* OPT_F32 or OPT_BF16 */
  int32_t activation;        /* OPT_ACT_* */
} opt_gated_args;
int opt_gated(const opt_gated_args* a, void* stream);

/* Gradients of opt_gated from dy (the gradient of y), gate and up:
 *   dgate = dy up f'(gate)      dup = dy f(gate)      (up NULL: dgate = dy f'(gate))
 * in fp32, each to any of: a plain matrix of `dtype`; codes with scales, the operand of
 * the product that gives the input's gradient; and transposed codes with scales, the
 * operand of the weight's gradient (rows x cols and cols x rows, blocks of 128 along
 * the operand's rows).  d_y_codes_t with d_y_scales_t is y again, transposed: the
 * operand of the gradient of the weight that y is multiplied by.  gate and up are of
 * `dtype`, as dy is, or both kept (d_gate_scales and d_up_scales given: d_gate and d_up
 * are codes).  Every output may be left NULL, but not all of them; a pair is given
 * whole.  d_dgate and d_dup may be d_dy or a plain d_gate or d_up (same pointer and
 * pitch); the other outputs overlap no input. */
typedef struct opt_gated_backward_args {
  const void* d_dy;
  const void* d_gate;
  const void* d_gate_scales;
  const void* d_up;
  const void* d_up_scales;
  void* d_dgate;
  void* d_dup;
  void* d_dgate_codes;
  void* d_dgate_scales;
  void* d_dgate_codes_t;
  void* d_dgate_scales_t;
  void* d_dup_codes;
  void* d_dup_scales;
  void* d_dup_codes_t;
  void* d_dup_scales_t;
  void* d_y_codes_t;
  void* d_y_scales_t;
  int64_t dy_pitch, gate_pitch, up_pitch, dgate_pitch, dup_pitch;
  int64_t dgate_codes_pitch, dgate_codes_t_pitch, dup_codes_pitch, dup_codes_t_pitch, y_codes_t_pitch;
  int64_t rows, cols;
  int32_t dtype;
  int32_t activation;
} opt_gated_backward_args;
int opt_gated_backward(const opt_gated_backward_args* a, void* stream);

/* Norm and rotation of heads.  q is rows x (q_heads dim), k is rows x (k_heads dim)
 * (matrices of their own, or columns of one projection's output); k_heads may be 0.
 * Per row and head, in fp32 with one rounding of each output:
 *   n = x weight / sqrt(mean(x^2) + eps)        (the mean over the head's dim elements)
 *   out = n with its first `rot` elements turned in pairs: with c and s the cosine and
 *   sine of pair i at the row's position,
 *     (a, b) -> (a c - b s, b c + a s)
 * where pair i is (i, i + rot / 2), or (2 i, 2 i + 1) with OPT_HEADS_INTERLEAVED.
 * d_cos and d_sin are fp32 tables of `positions` x rot / 2 (contiguous); row r stands
 * at d_positions[r] (int64), or at r if d_positions is NULL (rows <= positions then).
 * A position outside the tables makes the rotated elements NaN; nothing is read there.
 * rot is even, 0 <= rot <= dim (0: no rotation, and no tables); 1 <= dim <= 1024.
 * d_q_codes with d_q_scales (and k's) keep the inputs x for the backward pass: the
 * whole matrix's 1 x 128 blocks, across heads.  d_q_out may be d_q and d_k_out may be
 * d_k (same pointer and pitch); the other outputs overlap no input.  The sum of x^2 is
 * held in fp32, as in opt_rms_norm: a NaN makes its head NaN, squares that add up beyond
 * fp32 make it 0 (an infinity NaN), a head of zeros with eps 0 gives NaN.  No head and no
 * row reaches another's output.  Fastest: dim a multiple of 8 up to 256, and plain
 * matrices whose rows start on 16 bytes; then rot a multiple of 16, or of 8 with
 * OPT_HEADS_INTERLEAVED; and for keeping, dim a power of two. */
#define OPT_HEADS_INTERLEAVED 1
typedef struct opt_head_norm_args {
  const void* d_q;
  const void* d_q_weight;    /* dim elements of weight_dtype */
  void* d_q_out;
  void* d_q_codes;
  void* d_q_scales;
  const void* d_k;
  const void* d_k_weight;
  void* d_k_out;
  void* d_k_codes;
  void* d_k_scales;
  const float* d_cos;
  const float* d_sin;
  const int64_t* d_positions;
  int64_t q_pitch, q_out_pitch, q_codes_pitch, k_pitch, k_out_pitch, k_codes_pitch;
  int64_t rows, q_heads, k_heads, dim, rot, positions;
  int32_t dtype;             /* OPT_F32 or OPT_BF16 */
  int32_t weight_dtype;      /* OPT_F32 or OPT_BF16 */
  int32_t flags;             /* OPT_HEADS_* bits; others must be 0 */
  float eps;
} opt_head_norm_args;
int opt_head_norm(const opt_head_norm_args* a, void* stream);

/* Gradients of opt_head_norm from dout (the gradients of q_out and k_out) and the
 * inputs, plain or kept (d_q_scales, and d_k_scales if there are key heads, given: d_q
 * and d_k are codes):
 *   g = dout turned back, t = g weight, rstd = 1 / sqrt(mean(x^2) + eps)
 *   dx = rstd (t - x rstd^2 mean(t x))
 *   dweight = sum over rows and heads of g x rstd          (NULL: not wanted), fp32
 * in fp32, each rounded once; over no rows or no heads the sum is 0.  d_dq may be
 * d_dq_out and d_dk may be d_dk_out (same pointer and pitch).  The sums
 * run in a fixed order; they need d_workspace of
 * opt_head_norm_backward_workspace(rows, q_heads, k_heads, dim) bytes, 16-byte aligned,
 * when d_dq_weight or d_dk_weight is given (0 bytes: none). */
typedef struct opt_head_norm_backward_args {
  const void* d_dq_out;
  const void* d_q;
  const void* d_q_scales;
  const void* d_q_weight;
  void* d_dq;
  float* d_dq_weight;
  const void* d_dk_out;
  const void* d_k;
  const void* d_k_scales;
  const void* d_k_weight;
  void* d_dk;
  float* d_dk_weight;
  const float* d_cos;
  const float* d_sin;
  const int64_t* d_positions;
  void* d_workspace;
  int64_t dq_out_pitch, q_pitch, dq_pitch, dk_out_pitch, k_pitch, dk_pitch;
  int64_t workspace_bytes;
  int64_t rows, q_heads, k_heads, dim, rot, positions;
  int32_t dtype;             /* of dout, dx and plain inputs */
  int32_t weight_dtype;
  int32_t flags;
  float eps;
} opt_head_norm_backward_args;
int opt_head_norm_backward(const opt_head_norm_backward_args* a, void* stream);
int64_t opt_head_norm_backward_workspace(int64_t rows, int64_t q_heads, int64_t k_heads, int64_t dim);

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
