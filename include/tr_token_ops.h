/*
 * tr_token_ops.h — token-row operators of libtrfn.so: what turns a normalised
 * batch's patches into a network's hidden rows.
 *
 *   tr_rms_norm            residual addition and root-mean-square norm, output in
 *                          the input's type or in 8 bits with a scale per row
 *   tr_rms_norm_backward   its gradients
 *   tr_quantize_rows       8-bit rows with a scale per row (patches, weights)
 *   tr_dequantize_rows     reads them back
 *   tr_int8_matmul         product of two 8-bit matrices with a scale for each
 *                          token and each channel
 *
 * Conventions: those of tr_fused_norm.h (tr_status codes, host checks before
 * anything is launched, caller-owned buffers, no allocation, asynchronous on
 * `stream`, the current device).  In addition:
 *   - Matrices are row-major with unit column stride; *_stride is the distance
 *     of two rows in elements.  Output strides are at least the row's length
 *     (a single row's stride is not looked at); input strides are 0 or more (0
 *     repeats one row).  A matrix ends within the address space.
 *   - Pointers are aligned to their element.  Rows whose start and stride are
 *     multiples of 16 bytes are read in 16-byte pieces; any other alignment
 *     gives the same results more slowly.
 *   - An output may be the very same matrix (pointer, stride, element size) as
 *     an input where an entry says so; any other overlap of an output with
 *     another buffer is TR_ERR_INVALID_ARGUMENT.  Matrices interleaved in one
 *     buffer (column blocks with the same row distance in bytes) do not
 *     overlap; with different row distances, ranges that cross are refused.
 *   - rows = 0 is no work (a dweight is still written: zeros); cols is at least 1.
 *   - Calls that may run at the same time need workspaces of their own.
 *   - A product whose pipeline waits for more than about a second sets bit 0 of
 *     tr_device_status()'s word; parts of its output are then not written, the
 *     rest is right.
 */
#ifndef TR_TOKEN_OPS_H
#define TR_TOKEN_OPS_H

#include "tr_fused_norm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types; F32 and F16 have tr_out_dtype's values. */
typedef enum tr_elem {
    TR_ELEM_F32 = 0,          /* binary32 */
    TR_ELEM_F16 = 1,          /* binary16 */
    TR_ELEM_BF16 = 2,         /* bfloat16 */
    TR_ELEM_I8 = 3            /* int8 with a binary32 scale per row */
} tr_elem;

/* Longest row of the norm and quantisation entries (TR_ERR_NOT_SUPPORTED
 * above), and longest sum of tr_int8_matmul: 2^14 * 131071 < 2^31.           */
#define TR_MAX_ROW 32768
#define TR_MAX_INT8_K 131071
/* Most tokens or channels of tr_int8_matmul.                                */
#define TR_MAX_INT8_ROWS 2147479552

/* 8-bit rows.  With a = max_c |v_c| of a row v:
 *     scale = a / 127,   q_c = v_c * (127 / a) rounded to nearest (ties to even),
 * so q lies in [-127, 127] and q_c * scale stands for v_c.  A row with
 * a < 2^-119 holds zeros with scale 0 (127/a would not be finite much below);
 * a row that holds an infinity or a NaN holds zeros with scale NaN, so that
 * whatever is computed from it is NaN.                                      */

/* tr_rms_norm — with h = x + residual (h = x without one), for each row
 *     y_c = h_c * w_c / sqrt(mean_c(h_c^2) + eps)
 *   x            rows x cols of dtype (F32, F16 or BF16).
 *   residual     as x, or NULL.
 *   weight       cols binary32, or NULL for ones.
 *   out          rows x cols of out_dtype: dtype, or TR_ELEM_I8.
 *   residual_out receives h, rounded to dtype; or NULL.  Only with residual.
 *   scale        rows binary32, written for TR_ELEM_I8 (else ignored).
 * h is formed, squared, summed and scaled in binary32 and rounded once per
 * output: y is made from the unrounded h.  (A row whose squares sum beyond
 * binary32, |h| from 2^59 or so, gives y = 0, as the formula does in binary32.)  out
 * and residual_out may be x or residual (not both the same matrix).
 * Errors: TR_ERR_INVALID_ARGUMENT for bad pointers, strides, types, overlaps,
 * an eps that is negative or not finite; TR_ERR_NOT_SUPPORTED for
 * cols > TR_MAX_ROW or rows > 2^31 - 1.                                     */
int tr_rms_norm(const void* x, const void* residual, const float* weight, void* out, void* residual_out,
                float* scale, long long rows, long long cols, long long x_stride, long long residual_stride,
                long long out_stride, long long residual_out_stride, int dtype, int out_dtype, float eps,
                void* stream);

/* Bytes of tr_rms_norm_backward's workspace for a dweight of up to `rows` rows
 * of this length (host only).  It never shrinks as rows grows; it may as cols
 * does.                                                                      */
size_t tr_rms_norm_backward_workspace_bytes(long long rows, long long cols);

/* tr_rms_norm_backward — gradients of tr_rms_norm's y in the input's type.
 * With s = 1 / sqrt(mean_c(h_c^2) + eps) and g_c = dy_c * w_c:
 *     dx_c = s * (g_c - h_c * s^2 * mean_c(g_c * h_c)) + dresidual_c
 *     dweight_c = sum over rows of dy_c * h_c * s
 *   dy, h        rows x cols of dtype; h is the forward's residual_out (or its
 *                x where there was no residual).
 *   dresidual    gradient that reaches h along the residual stream, or NULL.
 *   dx           gradient of h, hence of x and of residual alike; may be dy, h
 *                or dresidual.
 *   dweight      cols binary32, overwritten; or NULL.
 *   workspace    device, tr_rms_norm_backward_workspace_bytes() bytes for these
 *                rows or more of this length, 16-byte aligned, not initialised;
 *                needed for a dweight only.
 * Sums are binary32 in a fixed order: the same call gives the same bits.    */
int tr_rms_norm_backward(const void* dy, const void* h, const float* weight, const void* dresidual, void* dx,
                         float* dweight, long long rows, long long cols, long long dy_stride, long long h_stride,
                         long long dresidual_stride, long long dx_stride, int dtype, float eps, void* workspace,
                         void* stream);

/* tr_quantize_rows — 8-bit rows (above) of x: q rows x cols int8, scale rows
 * binary32.                                                                 */
int tr_quantize_rows(const void* x, int8_t* q, float* scale, long long rows, long long cols, long long x_stride,
                     long long q_stride, int dtype, void* stream);

/* tr_dequantize_rows — out_c = q_c * scale, rounded to dtype.               */
int tr_dequantize_rows(const int8_t* q, const float* scale, void* out, long long rows, long long cols,
                       long long q_stride, long long out_stride, int dtype, void* stream);

/* Bytes of a workspace for tr_int8_matmul of up to M tokens with this N and K
 * (host only; 0 where none of them needs one).  It never shrinks as M grows, so
 * the largest M's workspace serves all.                                      */
size_t tr_int8_matmul_workspace_bytes(long long M, long long N, long long K);

/* tr_int8_matmul — for token m and channel n
 *     y[m][n] = (sum_k x[m][k] * w[n][k]) * x_scale[m] * w_scale[n] + bias[n]
 *   x        M x K int8, any value in [-128, 127];  x_scale  M binary32
 *   w        N x K int8;                            w_scale  N binary32
 *   bias     N binary32, or NULL.
 *   y        M x N of out_dtype (F32, F16 or BF16).
 *   workspace device, tr_int8_matmul_workspace_bytes() bytes for this M or a
 *            larger one, 16-byte aligned, not initialised; NULL where that is 0.
 * The sum is exact in integers; it is rounded to binary32 once, scaled, and
 * rounded to out_dtype.  K = 0 gives the bias (a sum of 0, which scales that
 * are not finite make NaN).
 * TR_ERR_NOT_SUPPORTED for K > TR_MAX_INT8_K or M, N > TR_MAX_INT8_ROWS.    */
int tr_int8_matmul(const int8_t* x, const float* x_scale, const int8_t* w, const float* w_scale,
                   const float* bias, void* y, long long M, long long N, long long K, long long x_stride,
                   long long w_stride, long long y_stride, int out_dtype, void* workspace, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* TR_TOKEN_OPS_H */
