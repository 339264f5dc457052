/*
 * moe_dense.h — C ABI of the dense half of a serving step around the routed
 * layer of moe_mxfp4.h, exported by the same libmoe_mxfp4.so:
 *
 *   moe_rms_norm        a residual sum and its root-mean-square norm, the result
 *                       in fp32, bf16 or as an MX matrix
 *   moe_mx_quantize     fp32 or bf16 rows to an MX matrix (MXFP4 or MXFP8)
 *   moe_mx_dequantize   an MX matrix to fp32 or bf16 rows
 *   moe_mx_linear       the product of MX activations with MXFP4 weights, with
 *                       an addend (a residual)
 *   moe_token_logprobs  log probabilities of given tokens under rows of logits,
 *                       their ranks, entropies, and the best alternatives
 *
 * A step: moe_rms_norm -> moe_mx_linear (queries, keys, values) ->
 * moe_kv_append -> moe_prefix_attention -> moe_mx_quantize -> moe_mx_linear (into
 * the residual) -> moe_rms_norm -> moe_forward -> ... -> moe_sample or
 * moe_token_logprobs.
 *
 * Conventions are those of moe_mxfp4.h and moe_serve.h: plain device pointers,
 * work enqueued on `stream`, nothing allocated, argument problems reported
 * before anything is launched.  Structs are read during the call only.
 */
#ifndef MOE_DENSE_H
#define MOE_DENSE_H

#include "moe_mxfp4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of an MX matrix. */
typedef enum {
  MOE_MX_E2M1 = 0, /* MXFP4: 4-bit codes, two to a byte, element 2i in the low nibble */
  MOE_MX_E4M3 = 1  /* MXFP8: one byte each, largest value 448, 0x7F and 0xFF NaN */
} moe_mx_type;

/* An MX matrix [rows][cols] (cols a multiple of 32): element (r, c) is
 * code(r, c) * 2^(s[r][c / 32] - 127), scale 255 meaning NaN.  Blocks of 32 run
 * along a row; with type MOE_MX_E2M1 and contiguous rows it is the moe_mx_mat of
 * moe_mxfp4.h.
 *   q         codes, 16-byte aligned, q_stride bytes between rows (a multiple of
 *             16, at least cols / 2 or cols)
 *   s         scales, s_stride bytes between rows (at least cols / 32) */
typedef struct {
  uint8_t* q;
  uint8_t* s;
  int32_t type, rows, cols;
  int64_t q_stride, s_stride;
} moe_mx;

/* What is beyond these is refused with MOE_ERR_UNSUPPORTED. */
#define MOE_DENSE_MAX_COLS 16384     /* of moe_rms_norm, moe_mx_quantize, moe_mx_dequantize, moe_mx_linear's inner size */
#define MOE_DENSE_MAX_STRIDE (1LL << 38) /* strides in elements stay below it to either side, of codes and scales below 4 times it in bytes */
#define MOE_MX_MAX_VALUES 34359730144LL /* rows x cols of one conversion: 2^35 less 8,224 */
#define MOE_LINEAR_MAX_ROWS 65536    /* rows of activations */
#define MOE_LINEAR_MAX_OUTS 262144   /* rows of weights */
#define MOE_LOGPROBS_MAX_ROWS 16777216
#define MOE_LOGPROBS_MAX_VOCAB 262144
#define MOE_LOGPROBS_MAX_TOP 32

/* Quantise: out = x, block by block.  With M the largest magnitude of a block and
 * emax = 2 (E2M1) or 8 (E4M3), the scale is 2^max(floor(log2 M) - emax, -127) and
 * codes are x / scale rounded to nearest, ties to even, saturating.  A block of
 * zeros has scale code 0.  A block that holds an infinity or a NaN has scale code
 * 255 and codes 0: all of it reads as NaN.
 *   x         [out->rows][out->cols] of type x_dtype (MOE_DT_F32 / MOE_DT_BF16),
 *             16-byte aligned, x_stride elements between rows (a multiple of 16
 *             bytes); at most MOE_MX_MAX_VALUES.  x and out must not overlap. */
int moe_mx_quantize(const void* x, int x_dtype, int64_t x_stride, const moe_mx* out, void* stream);

/* Dequantise: out = x, each value rounded once (fp32: exact where it is in
 * range; bf16: exact down to its subnormals).  `out` as x above; its rows must not
 * overlap, nor x. */
int moe_mx_dequantize(const moe_mx* x, void* out, int out_dtype, int64_t out_stride, void* stream);

/* Residual sum and root-mean-square norm, row by row:
 *   h = x + residual (fp32),   residual_out = h (rounded once to its type),
 *   y = h * weight / sqrt(mean(h^2) + eps)
 * in fp32, rounded once to the output's type (an MX output as moe_mx_quantize
 * does it).  The norm takes h before the rounding of residual_out.
 *   x          [rows][cols], f32 or bf16, x_stride elements between rows
 *   residual   NULL, or [rows][cols] of type res_dtype
 *   residual_out NULL (only without a residual), or as residual, with the same
 *              stride; may be residual itself; rows must not overlap
 *   weight     [cols] fp32 or NULL (ones)
 *   eps        > 0
 *   out, out_dtype, out_stride  MOE_DT_F32 or MOE_DT_BF16 rows, or
 *   mx         an MX matrix of [rows][cols]; one of out and mx is NULL
 * cols: a multiple of 8 (of 32 with mx), at most MOE_DENSE_MAX_COLS.  Pointers are
 * 16-byte aligned, strides a multiple of 16 bytes.  out (or residual_out) may be
 * x or residual itself with the same type and stride; other overlaps of outputs
 * are the caller's to avoid. */
int moe_rms_norm(int rows, int cols, const void* x, int x_dtype, int64_t x_stride, const void* residual,
                 void* residual_out, int res_dtype, int64_t res_stride, const float* weight, float eps, void* out,
                 int out_dtype, int64_t out_stride, const moe_mx* mx, void* stream);

/* Product: out[t][n] = (add ? add[t][n] : 0) + sum_k x[t][k] w[n][k], products
 * exact, sums in fp32, one rounding to the output's type.  The sums are the tensor
 * core's, which aligns and cuts addends: 32 products (64 with MOE_MX_E2M1
 * activations) and the sum so far are off by at most 18 units of 2^-23 of their
 * magnitudes.  A scale 255 or a NaN code gives NaN where the definition has it.
 *   x         [T][K], MOE_MX_E4M3 or MOE_MX_E2M1
 *   w         [N][K], MOE_MX_E2M1
 *   add       NULL, or [T][N] of out's type; may be out itself
 *   out       [T][N], MOE_DT_F32 or MOE_DT_BF16, *_stride elements between rows
 *             (rows of out must not overlap); any alignment of its type.  Other
 *             overlaps of out with the operands are the caller's to avoid.
 *   status    a DEVICE int32 or NULL, as in moe_serve.h (MOE_ERR_TIMEOUT: a
 *             bounded wait gave up; results without their whole sum are NaN)
 * K: a multiple of 128.  Codes are 32-byte aligned with row strides a multiple
 * of 32 bytes, scales 4-byte aligned with row strides a multiple of 4.  A row's
 * sum is taken in a fixed order for given sizes: results are the same from run
 * to run. */
int moe_mx_linear(const moe_mx* x, const moe_mx* w, const void* add, int64_t add_stride, void* out, int out_dtype,
                  int64_t out_stride, int32_t* status, void* stream);

/* Scores of given tokens, row by row.  With m the largest logit, S = sum
 * exp(z_i - m):
 *   logprob = z_t - m - log S          t = tokens[r]
 *   rank    = tokens before t in the order by (logit descending, index)
 *   entropy = log S - sum exp(z_i - m) (z_i - m) / S
 *   top     = the first `top` tokens of that order and their log probabilities
 * Statistics are fp32, and logprob <= 0 <= entropy.  NaN counts as -inf; if some
 * logits are +inf, those share the probability evenly and all others have none.  A
 * token outside [0, vocab) gives logprob -inf and rank -1 (padding).  Tokens of
 * probability 0 by a logit of -inf are not listed: where fewer than `top` are left,
 * ids are -1 with log probability -inf.  A row with nothing but -inf or NaN gives
 * logprob -inf, entropy 0 and no alternatives.
 *   logits       [rows][vocab], f32 or bf16 (aligned to the element), `stride`
 *                elements between rows, which do not overlap; rows <=
 *                MOE_LOGPROBS_MAX_ROWS, vocab <= MOE_LOGPROBS_MAX_VOCAB
 *   tokens       [rows] int32, or NULL: entropy and alternatives only (logprob
 *                and rank are then NULL too)
 *   logprob, entropy [rows] fp32 or NULL;  rank [rows] int32 or NULL
 *   top          0 .. MOE_LOGPROBS_MAX_TOP;  top_ids [rows][top] int32,
 *                top_logprobs [rows][top] fp32 (both, where top > 0) */
int moe_token_logprobs(int rows, int vocab, const void* logits, int dtype, int64_t stride, const int32_t* tokens,
                       float* logprob, int32_t* rank, float* entropy, int top, int32_t* top_ids, float* top_logprobs,
                       void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_DENSE_H */
