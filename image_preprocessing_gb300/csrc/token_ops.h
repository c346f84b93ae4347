// Internal declarations of the token-row operators (the C ABI is
// include/tr_token_ops.h): arguments after the host checks, and launchers.
#pragma once

#include <cstddef>
#include <cstdint>

#include "internal.h"
#include "tr_token_ops.h"

namespace trfn {

constexpr int kMaxDevices = 64;

// Norm or quantisation of rows; what == kQuantize has no residual, weight or eps.
enum RowWhat { kNorm, kNormQ8, kQuantize };
struct RowArgs {
    const void* x;
    const void* residual;      // or null
    const float* weight;       // or null
    const float* bias;         // layer norm's, or null
    void* out;
    void* residual_out;        // or null
    float* scale;
    long long rows, x_stride, residual_stride, out_stride, residual_out_stride;
    int cols;
    float eps;
    int dtype;
    RowWhat what;
    void* stream;
};
int launch_rows(const RowArgs& a);
int launch_layer_norm(const RowArgs& a);   // what: kNorm or kNormQ8

struct RowGradArgs {
    const void* dy;
    const void* h;
    const float* weight;       // or null
    const void* dresidual;     // or null
    void* dx;
    float* dweight;            // or null
    float* dbias;              // layer norm's, or null
    float* partial;            // workspace for these
    long long rows, dy_stride, h_stride, dresidual_stride, dx_stride;
    int cols;
    float eps;
    int dtype;
    void* stream;
};
int launch_row_grad(const RowGradArgs& a);
// CTAs of the gradient kernel, each with one partial dweight row.
int row_grad_parts(long long rows, long long cols);
int launch_layer_norm_grad(const RowGradArgs& a);
// At most this many CTAs, each with a partial row of 2 cols.
int layer_norm_grad_parts(long long rows, long long cols);

struct DequantArgs {
    const int8_t* q;
    const float* scale;
    void* out;
    long long rows, q_stride, out_stride;
    int cols;
    int dtype;
    void* stream;
};
int launch_dequant(const DequantArgs& a);

struct RotaryArgs {
    const void* x;
    void* out;
    const int32_t* positions;  // or null: the row's number
    const double* freqs;       // host
    long long tokens, x_stride, out_stride;
    int heads, dim, rot;
    int dtype;
    bool halves, inverse;
    float magnitude;
    void* stream;
};
int launch_rotary(const RotaryArgs& a);

// Attention; the arrays are on the device.
struct AttentionArgs {
    const void* q;
    const void* k;
    const void* v;
    void* out;
    const int32_t* q_starts;
    const int32_t* k_starts;
    const int32_t* q_lengths;  // or null
    const int32_t* k_lengths;  // or null
    int q_rows, k_rows, sequences;
    int heads, kv_heads, dim;
    long long q_stride, k_stride, v_stride, out_stride;
    int dtype;
    float scale;
    bool causal;
    void* workspace;
    void* stream;
};
int launch_attention(const AttentionArgs& a);
size_t attention_workspace(long long q_rows, long long sequences, long long heads, long long kv_heads, long long dim);

struct MatmulArgs {
    const int8_t* x;
    const float* x_scale;
    const int8_t* w;
    const float* w_scale;
    const float* bias;         // or null
    void* y;
    int M, N, K;
    long long x_stride, w_stride, y_stride;
    int out_dtype;
    void* workspace;
    void* stream;
};
int launch_int8_matmul(const MatmulArgs& a);
// What a product of these sizes needs, and what all of up to M tokens need at most.
size_t int8_matmul_workspace(long long M, long long N, long long K);
size_t int8_matmul_workspace_up_to(long long M, long long N, long long K);
// many tokens (int8_gemm.cu): binary16 copies in the workspace, tcgen05
int launch_int8_gemm(const MatmulArgs& a);
size_t int8_gemm_workspace(long long M, long long N, long long K);
// tokens in between (int8_mid.cu): tcgen05 on tiles converted on the way
int launch_int8_mid(const MatmulArgs& a);
// Estimates of the two, in SM cycles.
double int8_gemm_cycles(long long M, long long N, long long K);
double int8_mid_cycles(long long M, long long N, long long K);

// The int8 product's and the attention's status word (int8_status.cu) on device `dev`, the current
// one; reading it (as read_device_status, on the current device) copies nothing
// before the word has been asked for there.
int product_status_word(int dev, unsigned** word);
int read_product_status(int* flags, bool clear);

// tr_tune_tiled's test hook for bounded waits (flags bit 6), for the product's.
void set_test_waits(bool on);
bool test_waits();

// A failed runtime call as a tr_status: keeps its text for tr_last_error_message, and takes it from the runtime's
// last error, where another call would find it.
int cuda_failed(const char* what, int cuda_error);
// What a launch returned as a tr_status; counts the launch.  (Not cudaGetLastError(): an error that an earlier
// call left would be reported for a kernel that runs, and a caller who repeats an in-place call does it twice.)
int launched(const char* what, int cuda_error);

}  // namespace trfn
