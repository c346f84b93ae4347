// C ABI entry points of the token-row operators: argument checks on the host,
// before anything touches the GPU.

#include <cuda_runtime.h>

#include <atomic>
#include <cmath>

#include "token_ops.h"

namespace trfn {

namespace {
std::atomic<bool> g_test_waits{false};
}
void set_test_waits(bool on) { g_test_waits.store(on, std::memory_order_relaxed); }
bool test_waits() { return g_test_waits.load(std::memory_order_relaxed); }

int cuda_failed(const char* what, int cuda_error) {
    set_last_error(what, cuda_error);
    (void)cudaGetLastError();
    return TR_ERR_CUDA;
}

int launched(const char* what, int cuda_error) {
    if (cuda_error != (int)cudaSuccess) return cuda_failed(what, cuda_error);
    count_launch();
    return TR_OK;
}

namespace {

constexpr long long kMaxRows = 2147483647LL;
constexpr long long kMaxProductRows = TR_MAX_INT8_ROWS;   // row numbers of whole tiles stay below 2^31
constexpr long long kMaxStride = 1LL << 40;

int elem_bytes(int dtype) {
    switch (dtype) {
        case TR_ELEM_F32: return 4;
        case TR_ELEM_F16:
        case TR_ELEM_BF16: return 2;
        case TR_ELEM_I8: return 1;
        default: return 0;
    }
}

bool is_float(int dtype) { return dtype == TR_ELEM_F32 || dtype == TR_ELEM_F16 || dtype == TR_ELEM_BF16; }

// A row-major matrix as the kernels read or write it.
struct Mat {
    const void* p;
    long long rows, cols, stride;
    int es;

    // first byte and one past the last, for a stride of 0 or more
    uintptr_t lo() const { return (uintptr_t)p; }
    unsigned __int128 hi() const {
        return lo() + ((unsigned __int128)(rows - 1) * (unsigned long long)stride + cols) * (unsigned)es;
    }
    bool empty() const { return p == nullptr || rows == 0 || cols == 0; }
    bool aligned() const { return lo() % (unsigned)es == 0; }
};

bool same(const Mat& a, const Mat& b) {
    return a.p == b.p && a.es == b.es && (a.rows <= 1 || a.stride == b.stride);
}

// Whether two matrices share a byte.  Exact for equal row distances (column
// blocks of one buffer) and for byte ranges that do not cross; else assumed.
bool overlaps(const Mat& a, const Mat& b) {
    if (a.empty() || b.empty()) return false;
    if (a.lo() >= b.hi() || b.lo() >= a.hi()) return false;
    const unsigned long long sa = (unsigned long long)a.stride * a.es, sb = (unsigned long long)b.stride * b.es;
    const unsigned long long wa = (unsigned long long)a.cols * a.es, wb = (unsigned long long)b.cols * b.es;
    if (a.rows > 1 && b.rows > 1 && sa == sb && sa >= wa && sb >= wb) {
        const unsigned long long d = b.lo() >= a.lo() ? (b.lo() - a.lo()) % sa : (sa - (a.lo() - b.lo()) % sa) % sa;
        return !(d >= wa && d + wb <= sa);
    }
    return true;
}

bool bad_input(const Mat& m) {
    return m.p == nullptr || !m.aligned() || m.stride < 0 || m.stride > kMaxStride || m.hi() >> 64 != 0;
}
bool bad_output(const Mat& m) { return bad_input(m) || (m.rows > 1 && m.stride < m.cols); }

// A single row's stride is not looked at (and may be anything): make it plain.
long long row_stride(long long rows, long long cols, long long stride) { return rows <= 1 ? cols : stride; }

int check_rows(long long rows, long long cols) {
    if (rows < 0 || cols < 1) return TR_ERR_INVALID_ARGUMENT;
    if (rows > kMaxRows || cols > TR_MAX_ROW) return TR_ERR_NOT_SUPPORTED;
    return TR_OK;
}

int grad_workspace_ok(const Mat& ws) { return ws.p != nullptr && ws.lo() % 16 == 0; }

}  // namespace
}  // namespace trfn

using namespace trfn;

extern "C" {

int tr_rms_norm(const void* x, const void* residual, const float* weight, void* out, void* residual_out,
                float* scale, long long rows, long long cols, long long x_stride, long long residual_stride,
                long long out_stride, long long residual_out_stride, int dtype, int out_dtype, float eps,
                void* stream) {
    if (!is_float(dtype) || (out_dtype != dtype && out_dtype != TR_ELEM_I8)) return TR_ERR_INVALID_ARGUMENT;
    if (!std::isfinite(eps) || eps < 0.0f) return TR_ERR_INVALID_ARGUMENT;
    const int rc = check_rows(rows, cols);
    if (rc != TR_OK) return rc;
    if (rows == 0) return TR_OK;
    const int es = elem_bytes(dtype);
    const Mat mx{x, rows, cols, row_stride(rows, cols, x_stride), es};
    const Mat mr{residual, rows, cols, row_stride(rows, cols, residual_stride), es};
    const Mat mo{out, rows, cols, row_stride(rows, cols, out_stride), elem_bytes(out_dtype)};
    const Mat mh{residual_out, rows, cols, row_stride(rows, cols, residual_out_stride), es};
    const Mat mw{weight, 1, cols, cols, 4};
    const Mat ms{out_dtype == TR_ELEM_I8 ? scale : nullptr, 1, rows, rows, 4};
    if (bad_input(mx) || bad_output(mo) || !mw.aligned()) return TR_ERR_INVALID_ARGUMENT;
    if (residual != nullptr && bad_input(mr)) return TR_ERR_INVALID_ARGUMENT;
    if (residual_out != nullptr && (residual == nullptr || bad_output(mh))) return TR_ERR_INVALID_ARGUMENT;
    if (out_dtype == TR_ELEM_I8 && bad_input(ms)) return TR_ERR_INVALID_ARGUMENT;
    for (const Mat* w : {&mo, &mh}) {
        for (const Mat* r : {&mx, &mr})
            if (overlaps(*w, *r) && !same(*w, *r)) return TR_ERR_INVALID_ARGUMENT;
        if (overlaps(*w, mw) || overlaps(*w, ms)) return TR_ERR_INVALID_ARGUMENT;
    }
    if (overlaps(mo, mh) || overlaps(ms, mx) || overlaps(ms, mr) || overlaps(ms, mw)) return TR_ERR_INVALID_ARGUMENT;
    RowArgs a{};
    a.x = x; a.residual = residual; a.weight = weight; a.out = out; a.residual_out = residual_out; a.scale = scale;
    a.rows = rows; a.cols = (int)cols;
    a.x_stride = mx.stride; a.residual_stride = mr.stride; a.out_stride = mo.stride;
    a.residual_out_stride = mh.stride;
    a.eps = eps; a.dtype = dtype; a.what = out_dtype == TR_ELEM_I8 ? kNormQ8 : kNorm; a.stream = stream;
    return launch_rows(a);
}

size_t tr_rms_norm_backward_workspace_bytes(long long rows, long long cols) {
    if (check_rows(rows, cols) != TR_OK) return 0;
    return (size_t)row_grad_parts(rows, cols) * (size_t)cols * sizeof(float);
}

int tr_rms_norm_backward(const void* dy, const void* h, const float* weight, const void* dresidual, void* dx,
                         float* dweight, long long rows, long long cols, long long dy_stride, long long h_stride,
                         long long dresidual_stride, long long dx_stride, int dtype, float eps, void* workspace,
                         void* stream) {
    if (!is_float(dtype) || !std::isfinite(eps) || eps < 0.0f) return TR_ERR_INVALID_ARGUMENT;
    const int rc = check_rows(rows, cols);
    if (rc != TR_OK) return rc;
    const int es = elem_bytes(dtype);
    const Mat my{dy, rows, cols, row_stride(rows, cols, dy_stride), es};
    const Mat mh{h, rows, cols, row_stride(rows, cols, h_stride), es};
    const Mat mr{dresidual, rows, cols, row_stride(rows, cols, dresidual_stride), es};
    const Mat mx{dx, rows, cols, row_stride(rows, cols, dx_stride), es};
    const Mat mw{weight, 1, cols, cols, 4};
    const Mat md{dweight, 1, cols, cols, 4};
    if (!mw.aligned() || !md.aligned()) return TR_ERR_INVALID_ARGUMENT;
    if (rows == 0) {
        if (dweight == nullptr) return TR_OK;
        const cudaError_t e = cudaMemsetAsync(dweight, 0, (size_t)cols * 4, static_cast<cudaStream_t>(stream));
        return e == cudaSuccess ? TR_OK : cuda_failed("cudaMemsetAsync(dweight)", (int)e);
    }
    if (bad_input(my) || bad_input(mh) || bad_output(mx)) return TR_ERR_INVALID_ARGUMENT;
    if (dresidual != nullptr && bad_input(mr)) return TR_ERR_INVALID_ARGUMENT;
    for (const Mat* r : {&my, &mh, &mr})
        if (overlaps(mx, *r) && !same(mx, *r)) return TR_ERR_INVALID_ARGUMENT;
    if (overlaps(mx, mw)) return TR_ERR_INVALID_ARGUMENT;
    if (dweight != nullptr) {
        const long long n = row_grad_parts(rows, cols) * cols;
        const Mat ws{workspace, 1, n, n, 4};
        if (!grad_workspace_ok(ws)) return TR_ERR_INVALID_ARGUMENT;
        for (const Mat* r : {&my, &mh, &mr, &mx, &mw})
            if (overlaps(md, *r) || overlaps(ws, *r)) return TR_ERR_INVALID_ARGUMENT;
        if (overlaps(md, ws)) return TR_ERR_INVALID_ARGUMENT;
    }
    RowGradArgs a{};
    a.dy = dy; a.h = h; a.weight = weight; a.dresidual = dresidual; a.dx = dx; a.dweight = dweight;
    a.partial = static_cast<float*>(workspace);
    a.rows = rows; a.cols = (int)cols;
    a.dy_stride = my.stride; a.h_stride = mh.stride; a.dresidual_stride = mr.stride; a.dx_stride = mx.stride;
    a.eps = eps; a.dtype = dtype; a.stream = stream;
    return launch_row_grad(a);
}

int tr_quantize_rows(const void* x, int8_t* q, float* scale, long long rows, long long cols, long long x_stride,
                     long long q_stride, int dtype, void* stream) {
    if (!is_float(dtype)) return TR_ERR_INVALID_ARGUMENT;
    const int rc = check_rows(rows, cols);
    if (rc != TR_OK) return rc;
    if (rows == 0) return TR_OK;
    const Mat mx{x, rows, cols, row_stride(rows, cols, x_stride), elem_bytes(dtype)};
    const Mat mq{q, rows, cols, row_stride(rows, cols, q_stride), 1};
    const Mat ms{scale, 1, rows, rows, 4};
    if (bad_input(mx) || bad_output(mq) || bad_input(ms)) return TR_ERR_INVALID_ARGUMENT;
    if (overlaps(mx, mq) || overlaps(mx, ms) || overlaps(mq, ms)) return TR_ERR_INVALID_ARGUMENT;
    RowArgs a{};
    a.x = x; a.out = q; a.scale = scale;
    a.rows = rows; a.cols = (int)cols; a.x_stride = mx.stride; a.out_stride = mq.stride;
    a.dtype = dtype; a.what = kQuantize; a.stream = stream;
    return launch_rows(a);
}

int tr_dequantize_rows(const int8_t* q, const float* scale, void* out, long long rows, long long cols,
                       long long q_stride, long long out_stride, int dtype, void* stream) {
    if (!is_float(dtype)) return TR_ERR_INVALID_ARGUMENT;
    const int rc = check_rows(rows, cols);
    if (rc != TR_OK) return rc;
    if (rows == 0) return TR_OK;
    const Mat mq{q, rows, cols, row_stride(rows, cols, q_stride), 1};
    const Mat mo{out, rows, cols, row_stride(rows, cols, out_stride), elem_bytes(dtype)};
    const Mat ms{scale, 1, rows, rows, 4};
    if (bad_input(mq) || bad_output(mo) || bad_input(ms)) return TR_ERR_INVALID_ARGUMENT;
    if (overlaps(mo, mq) || overlaps(mo, ms)) return TR_ERR_INVALID_ARGUMENT;
    DequantArgs a{};
    a.q = q; a.scale = scale; a.out = out; a.rows = rows; a.cols = (int)cols;
    a.q_stride = mq.stride; a.out_stride = mo.stride; a.dtype = dtype; a.stream = stream;
    return launch_dequant(a);
}

size_t tr_int8_matmul_workspace_bytes(long long M, long long N, long long K) {
    if (M < 1 || N < 1 || K < 1 || M > kMaxProductRows || N > kMaxProductRows || K > TR_MAX_INT8_K) return 0;
    return int8_matmul_workspace_up_to(M, N, K);
}

int tr_int8_matmul(const int8_t* x, const float* x_scale, const int8_t* w, const float* w_scale,
                   const float* bias, void* y, long long M, long long N, long long K, long long x_stride,
                   long long w_stride, long long y_stride, int out_dtype, void* workspace, void* stream) {
    if (!is_float(out_dtype) || M < 0 || N < 0 || K < 0) return TR_ERR_INVALID_ARGUMENT;
    if (M > kMaxProductRows || N > kMaxProductRows || K > TR_MAX_INT8_K) return TR_ERR_NOT_SUPPORTED;
    if (M == 0 || N == 0) return TR_OK;
    const Mat mx{x, M, K, row_stride(M, K, x_stride), 1};
    const Mat mw{w, N, K, row_stride(N, K, w_stride), 1};
    const Mat my{y, M, N, row_stride(M, N, y_stride), elem_bytes(out_dtype)};
    const Mat mxs{x_scale, 1, M, M, 4}, mws{w_scale, 1, N, N, 4}, mb{bias, 1, N, N, 4};
    if (bad_output(my) || bad_input(mxs) || bad_input(mws) || !mb.aligned()) return TR_ERR_INVALID_ARGUMENT;
    if (K > 0 && (bad_input(mx) || bad_input(mw))) return TR_ERR_INVALID_ARGUMENT;
    const long long need = K > 0 ? (long long)int8_matmul_workspace(M, N, K) : 0;
    const Mat ws{need > 0 ? workspace : nullptr, 1, need, need, 1};
    if (need > 0 && (workspace == nullptr || ws.lo() % 16 != 0)) return TR_ERR_INVALID_ARGUMENT;
    for (const Mat* r : {&mx, &mw, &mxs, &mws, &mb})
        if (overlaps(my, *r) || overlaps(ws, *r)) return TR_ERR_INVALID_ARGUMENT;
    if (overlaps(my, ws)) return TR_ERR_INVALID_ARGUMENT;
    MatmulArgs a{};
    a.x = x; a.x_scale = x_scale; a.w = w; a.w_scale = w_scale; a.bias = bias; a.y = y;
    a.M = (int)M; a.N = (int)N; a.K = (int)K;
    a.x_stride = mx.stride; a.w_stride = mw.stride; a.y_stride = my.stride;
    a.out_dtype = out_dtype; a.workspace = workspace; a.stream = stream;
    return launch_int8_matmul(a);
}

}  // extern "C"
