/*
 * qemb_serving.h -- C ABI of libqemb_serving: what stands around the
 * attention of qemb_attention.h in a serving loop on AMD Instinct MI355X
 * (gfx950).
 *
 *  - qemb_add_norm        a residual's addition and the root-mean-square norm
 *                         of the sum in one pass, as 16-bit values, as 8-bit
 *                         codes with scales, or as packed INT8 rows of qemb.h
 *  - qemb_token_logprobs  log probabilities of given tokens, entropies and the
 *                         most likely tokens, from one pass over the logits
 *
 * Conventions (those of qemb.h): every array is a device pointer owned by
 * the caller; nothing is allocated, kept or synchronized; work goes onto
 * `stream`; errors that the host can see return before anything is enqueued.
 * Bad device data never faults: it is skipped as stated and, where an
 * err_count (nullable, device, caller-zeroed) is taken, counted.  Calls are
 * deterministic: equal calls give equal bits.  Sums, norms and softmax
 * statistics are held in binary32.
 */
#ifndef QEMB_SERVING_H
#define QEMB_SERVING_H

#include "qemb_attention.h"

#ifdef __cplusplus
extern "C" {
#endif

#define QEMB_DTYPE_FP32 2 /* qemb_token_logprobs only */

#define QEMB_FORM_VALUES 0 /* 16-bit values of dtype */
#define QEMB_FORM_INT8 1   /* signed codes -127 .. 127, fp32 scales */
#define QEMB_FORM_E4M3 2   /* 8-bit floats (4 exponent bits, bias 7, no infinities), fp32 scales */
#define QEMB_FORM_ROWS8 3  /* packed INT8 rows of qemb.h */

#define QEMB_MAX_NORM_DIM 32768
#define QEMB_MAX_TOP 64

/*
 * Residual addition and norm.  For every row, in binary32:
 *     h = x + residual,   y = (h * rsqrt(mean(h^2) + eps)) * weight
 * sum_out takes h rounded once to dtype; y comes from the unrounded h:
 *   QEMB_FORM_VALUES  y rounded once to dtype
 *   QEMB_FORM_INT8    codes rint(y * (127 / a)), value code * scale, and
 *   QEMB_FORM_E4M3    codes round(y * (448 / a)), value code * scale, where a is
 *                     the largest |y| of the row (group = 0) or of each `group`
 *                     elements, and scale = a / 127 or a / 448.  Scales below
 *                     2^-126 (a = 0 among them) are 0 with codes 0.  An infinity
 *                     or a NaN among the elements: the scale is NaN, codes are 0.
 *   QEMB_FORM_ROWS8   the row as qemb_quantize_rowwise would pack it (the range
 *                     rule; dim at most QEMB_MAX_DIM, |y| at most 65504)
 *   x, residual  [rows][dim] of dtype, strides in elements between rows
 *                (multiples of 8; the stride of a single row is not read), dim a
 *                multiple of 8 up to QEMB_MAX_NORM_DIM, 16-byte aligned; residual
 *                nullable: h = x
 *   weight       [dim] of dtype, or NULL for ones
 *   group        0, or 32, 64, 128, 256 or 512, dividing dim; 0 unless the form
 *                has scales
 *   out          [rows][dim] of dtype or of bytes, or packed rows; contiguous
 *   scales       [rows][dim / group] or [rows] fp32, with such a form only
 *   sum_out      [rows][dim] of dtype, with a stride as x; nullable.  It may be
 *                x or residual itself (the same address and stride); nothing
 *                else may overlap
 */
int qemb_add_norm(const void* x, const void* residual, const void* weight, int64_t rows, int32_t dim,
                  int32_t dtype, int64_t x_stride, int64_t residual_stride, int64_t sum_stride,
                  float eps, int32_t form, int32_t group, void* out, float* scales, void* sum_out,
                  qemb_stream_t stream);

/*
 * Log probabilities.  For every row x of logits,
 *     lse = log sum_j exp(x_j),   logprob = x_target - lse,
 *     entropy = lse - sum_j exp(x_j - lse) x_j   (a logit of -inf adds nothing)
 * and the `top` largest logits' ids, largest first (ties: the lowest id first;
 * -0 equals 0; a NaN counts as -inf), with x_id - lse.
 * A row of -inf alone: lse and log probabilities -inf, entropy 0.  A NaN or a
 * +inf in a row makes its lse, entropy and log probabilities NaN (ids stand).
 *   logits      [rows][vocab] of dtype (QEMB_DTYPE_FP32 too), row_stride >= 0
 *               elements between rows (not read of a single row), aligned to its elements
 *   targets     [rows] of index_type, nullable with logprobs.  One that leaves
 *               [0, vocab) gives 0; it is counted if it is not negative
 *   top         0 .. QEMB_MAX_TOP.  Ids past vocab are -1, their logprobs -inf
 *   logprobs, entropy, lse  [rows] fp32, each nullable
 *   top_ids     [rows][top] int32, top_logprobs [rows][top] fp32 (with top > 0)
 *   workspace   qemb_logprobs_workspace_bytes(...) bytes, 16-byte aligned
 *               (NULL where that is 0); contents need not be kept
 * vocab 1 .. 2^30.
 */
size_t qemb_logprobs_workspace_bytes(int64_t rows, int64_t vocab, int32_t dtype, int32_t top);

int qemb_token_logprobs(const void* logits, int64_t rows, int64_t vocab, int32_t dtype,
                        int64_t row_stride, const void* targets, int32_t index_type, int32_t top,
                        float* logprobs, float* entropy, float* lse, int32_t* top_ids,
                        float* top_logprobs, void* workspace, int32_t* err_count,
                        qemb_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif
