/*
 * tr_token_ops.h — token-row operators of libtrfn.so: what turns a normalised
 * batch's patches into a network's hidden rows.
 *
 *   tr_rms_norm            residual addition and root-mean-square norm, output in
 *                          the input's type or in 8 bits with a scale per row
 *   tr_rms_norm_backward   its gradients
 *   tr_layer_norm          the same with layer norm, which takes the mean away and
 *                          adds a bias
 *   tr_layer_norm_backward its gradients
 *   tr_quantize_rows       8-bit rows with a scale per row (patches, weights)
 *   tr_dequantize_rows     reads them back
 *   tr_int8_matmul         product of two 8-bit matrices with a scale for each
 *                          token and each channel
 *   tr_rotary              rotary positions of heads, and back (the gradient);
 *                          tr_rotary_frequencies makes their frequencies
 *   tr_attention           attention over packed sequences, grouped heads
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
 *   - A product or an attention whose pipeline waits for more than about a
 *     second sets bit 0 of tr_device_status()'s word; parts of its output are then
 *     not written, the rest is right.
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

/* tr_layer_norm — with h = x + residual (h = x without one), for each row
 *     y_c = (h_c - m) * w_c / sqrt(mean_c((h_c - m)^2) + eps) + b_c,   m = mean_c(h_c)
 *   bias         cols binary32, or NULL for zeros; the others as tr_rms_norm's.
 * h, its mean, the squares (of values less the mean) and y are formed in
 * binary32 and rounded once per output; y is made from the unrounded h.
 * Errors: those of tr_rms_norm.                                             */
int tr_layer_norm(const void* x, const void* residual, const float* weight, const float* bias, void* out,
                  void* residual_out, float* scale, long long rows, long long cols, long long x_stride,
                  long long residual_stride, long long out_stride, long long residual_out_stride, int dtype,
                  int out_dtype, float eps, void* stream);

/* Bytes of tr_layer_norm_backward's workspace for the dweight and dbias of up to
 * `rows` rows of this length (host only).  It never shrinks as rows grows.     */
size_t tr_layer_norm_backward_workspace_bytes(long long rows, long long cols);

/* tr_layer_norm_backward — gradients of tr_layer_norm's y in the input's type.
 * With s = 1 / sqrt(mean_c((h_c - m)^2) + eps), u_c = (h_c - m) * s, g_c = dy_c * w_c:
 *     dx_c = s * (g_c - mean_c(g_c) - u_c * mean_c(g_c * u_c)) + dresidual_c
 *     dweight_c = sum over rows of dy_c * u_c,   dbias_c = sum over rows of dy_c
 *   dweight, dbias  cols binary32 each, overwritten; or NULL, either of them.
 *   workspace    device, tr_layer_norm_backward_workspace_bytes() bytes for these
 *                rows or more of this length, 16-byte aligned, not initialised;
 *                needed for a dweight or a dbias only.
 * The rest as tr_rms_norm_backward.                                         */
int tr_layer_norm_backward(const void* dy, const void* h, const float* weight, const void* dresidual, void* dx,
                           float* dweight, float* dbias, long long rows, long long cols, long long dy_stride,
                           long long h_stride, long long dresidual_stride, long long dx_stride, int dtype, float eps,
                           void* workspace, void* stream);

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

/* Rotary positions.  The pairs of a head: value k with value k + rot/2, or
 * value 2k with value 2k + 1.                                               */
typedef enum tr_rotary_layout { TR_ROTARY_HALVES = 0, TR_ROTARY_PAIRS = 1 } tr_rotary_layout;

/* How frequencies are scaled for contexts `factor` times as long.           */
typedef enum tr_rotary_scaling {
    TR_ROTARY_UNSCALED = 0,   /* f_k = base^(-2k / rot) */
    TR_ROTARY_LINEAR = 1,     /* f_k / factor: positions interpolated */
    TR_ROTARY_BASE = 2,       /* base * factor^(rot / (rot - 2)): the last pair interpolated, the first kept */
    TR_ROTARY_PARTS = 3       /* by the turns r_k = trained * f_k / 2 pi that a pair makes over the positions it was
                               * trained on (the YaRN paper): with g_k = (r_k - 1) / (32 - 1) cut to [0, 1],
                               * f_k * (g_k + (1 - g_k) / factor), and magnitude 0.1 ln(factor) + 1 */
} tr_rotary_scaling;

/* Most turned values of a head, heads of a matrix; longest head of attention. */
#define TR_MAX_ROTARY 512
#define TR_MAX_HEADS 65535
#define TR_MAX_HEAD_DIM 256

/* Frequencies of rot/2 pairs, radians for each position, and the magnitude that
 * goes with them (host only).  trained: for TR_ROTARY_PARTS.
 * Errors: TR_ERR_INVALID_ARGUMENT for an odd rot or one below 2 (4 for
 * TR_ROTARY_BASE), base <= 1, factor < 1, trained < 1 where it counts;
 * TR_ERR_NOT_SUPPORTED for rot > TR_MAX_ROTARY.                             */
int tr_rotary_frequencies(long long rot, double base, int scaling, double factor, long long trained, double* freqs,
                          float* magnitude);

/* tr_rotary — for token i, every head and pair k, with t = positions[i]:
 *     (a, b) -> magnitude * (a cos(t f_k) - b sin(t f_k), b cos(t f_k) + a sin(t f_k))
 *   x, out       tokens x (heads * dim) of dtype (F32, F16 or BF16): head h is
 *                columns h * dim ... ; out may be x.
 *   positions    tokens int32 on the device, any value; or NULL: token i is at i.
 *   freqs        rot / 2 finite frequencies on the HOST, read before the call
 *                returns (a captured call keeps them).
 *   rot          turned values of a head, its first; even, up to dim.  The rest
 *                are copied.
 *   inverse      not 0: turns by -t f_k, which is the gradient: dx of dout.
 * Angles are exact to 2^-24 of a half turn at any position; the products are
 * binary32, rounded once.
 * TR_ERR_NOT_SUPPORTED for rot > TR_MAX_ROTARY, heads > TR_MAX_HEADS, dim >
 * TR_MAX_ROW or tokens > 2^31 - 1.                                          */
int tr_rotary(const void* x, void* out, const int32_t* positions, const double* freqs, long long tokens, long long heads,
              long long dim, long long rot, long long x_stride, long long out_stride, int dtype, int layout,
              float magnitude, int inverse, void* stream);

/* Most rows of q or k, and most sequences, of tr_attention.                 */
#define TR_MAX_ATTENTION_ROWS 2147483647
#define TR_MAX_SEQUENCES 1048576

/* Bytes of tr_attention's workspace for up to this many rows of q and sequences
 * (host only; 0 where none of them needs one).  It never shrinks as either grows. */
size_t tr_attention_workspace_bytes(long long q_rows, long long sequences, long long heads, long long kv_heads,
                                    long long dim);

/* tr_attention — for query i and head h of a sequence,
 *     o = sum_j p_j v_j / sum_j p_j,   p_j = exp(scale * (q . k_j)),
 * over the keys j of the sequence that the query sees: all of its Lk keys, or,
 * causal, the first i + 1 + Lk - Lq of them (the last query sees all: a step's new
 * tokens come after what is cached).  A query that sees no key gets zeros.
 *   q, out       q_rows x (heads * dim) of dtype (F32, F16 or BF16): head h is
 *                columns h * dim ... ;  k, v  k_rows x (kv_heads * dim).  Heads
 *                h with the same h / (heads / kv_heads) share a key head.
 *   q_starts     sequences + 1 int32 on the device: sequence s's queries are rows
 *                q_starts[s] .. q_starts[s + 1]; with q_lengths (sequences int32,
 *                or NULL) q_starts[s] .. q_starts[s] + q_lengths[s], and what lies
 *                between is left as it is.  k_starts, k_lengths: keys and values,
 *                likewise (slots of a cache, filled in part).
 * Sequences may be empty, keys shared by several.  The arrays are read by the
 * GPU: nothing outside q, k and v is read whatever they hold (rows beyond a
 * matrix, or ends before starts, are cut off).  Sequences' queries do not overlap
 * (rows of q that two of them claim get the output of either, or none).  Rows that
 * belong to none are not written.
 *   workspace    device, tr_attention_workspace_bytes() bytes for these rows and
 *                sequences or more, 16-byte aligned, not initialised.
 * Scores, maxima, sums and outputs are binary32; in F16 and BF16 a weight p is
 * rounded to dtype for the product with v and for the sum.  What a query does not see does not
 * reach its output, whatever it holds (infinities and NaN included).  The same
 * call gives the same bits.
 * Fast for F16 and BF16 with dim a multiple of 8 up to 128, up to 64 heads to a
 * key head, a scale above 0, and matrices and strides on 16 bytes (rows that do
 * not overlap); a plain kernel takes the rest.
 * TR_ERR_INVALID_ARGUMENT where heads is no multiple of kv_heads or out overlaps
 * another buffer; TR_ERR_NOT_SUPPORTED for dim > TR_MAX_HEAD_DIM, heads >
 * TR_MAX_HEADS, sequences > TR_MAX_SEQUENCES or rows > TR_MAX_ATTENTION_ROWS. */
int tr_attention(const void* q, const void* k, const void* v, void* out, const int32_t* q_starts,
                 const int32_t* k_starts, const int32_t* q_lengths, const int32_t* k_lengths, long long q_rows,
                 long long k_rows, long long sequences, long long heads, long long kv_heads, long long dim,
                 long long q_stride, long long k_stride, long long v_stride, long long out_stride, int dtype,
                 float scale, int causal, void* workspace, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* TR_TOKEN_OPS_H */
