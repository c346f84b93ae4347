// Row operators: RMS norm with the residual's addition (output in the input's
// type or in 8 bits), its gradients, 8-bit quantisation of rows and reading
// them back.
//
// Mathematics, for a row h = x + r of n values:
//     s = 1/sqrt(sum_c h_c^2 / n + eps),  y_c = h_c s w_c
//     8 bits: a = max_c |y_c|, scale = a/127, q_c = rint(y_c 127/a)
//     gradients, with g_c = dy_c w_c:
//     dx_c = s (g_c - h_c s^2 (sum_j g_j h_j)/n) + dres_c,   dw_c = sum_rows dy_c h_c s
//
// All of them are bound by HBM: a row is read once, kept in registers, reduced
// once, and written.  max_c |y_c| = s max_c |h_c w_c| needs no s, so the 8-bit
// output takes one reduction, of the pair (sum of squares, maximum).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "token_ops.h"

namespace trfn {
namespace {

constexpr float kTiny = 0x1p-119f;   // rows below it are zeros in 8 bits (127/a stays finite above)

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T> __device__ __forceinline__ T from_f(float v);
template <> __device__ __forceinline__ float from_f<float>(float v) { return v; }
template <> __device__ __forceinline__ __half from_f<__half>(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

template <int B> struct Word;
template <> struct Word<1> { using T = uint8_t; };
template <> struct Word<2> { using T = uint16_t; };
template <> struct Word<4> { using T = uint32_t; };
template <> struct Word<8> { using T = uint2; };
template <> struct Word<16> { using T = uint4; };

// V values as one access of V * sizeof(E) bytes.
template <typename E, int V>
union Pack {
    typename Word<sizeof(E) * V>::T word;
    E e[V];
    __device__ __forceinline__ Pack() {}
};

// Values c .. c+V-1 of a row of n, zeros past its end.  V > 1 only where every
// row starts on a boundary of the access.
template <typename E, int V>
__device__ __forceinline__ Pack<E, V> load_pack(const E* row, int c, int n) {
    Pack<E, V> p;
    if (c + V <= n) {
        p.word = *reinterpret_cast<const typename Word<sizeof(E) * V>::T*>(row + c);
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) p.e[j] = (c + j < n) ? row[c + j] : from_f<E>(0.0f);
    }
    return p;
}

template <typename E, int V>
__device__ __forceinline__ void store_pack(E* row, int c, int n, const Pack<E, V>& p) {
    if (c + V <= n) {
        *reinterpret_cast<typename Word<sizeof(E) * V>::T*>(row + c) = p.word;
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (c + j < n) row[c + j] = p.e[j];
    }
}

template <int V>
__device__ __forceinline__ void load_weight(const float* w, int c, int n, float (&v)[V]) {
    if (w == nullptr) {
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] = 1.0f;
        return;
    }
    if constexpr (V >= 4) {
        if (c + V <= n) {
#pragma unroll
            for (int j = 0; j < V; j += 4) {
                const float4 f = *reinterpret_cast<const float4*>(w + c + j);
                v[j] = f.x; v[j + 1] = f.y; v[j + 2] = f.z; v[j + 3] = f.w;
            }
            return;
        }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] = (c + j < n) ? w[c + j] : 0.0f;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Sum of `a`, and sum (Q = false) or maximum of the bits (Q = true) of `b`,
// over the T threads of a row, in a fixed order.
template <int T, bool Q>
__device__ __forceinline__ void reduce_row(float& a, float& b) {
    __shared__ float sa[T / 32], sb[T / 32];
    a = warp_sum(a);
    if (Q) b = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(b)));
    else b = warp_sum(b);
    if constexpr (T > 32) {
        const int w = threadIdx.x >> 5;
        __syncthreads();   // the previous row's reads of sa, sb are over
        if ((threadIdx.x & 31) == 0) { sa[w] = a; sb[w] = b; }
        __syncthreads();
        a = sa[0];
        b = sb[0];
#pragma unroll
        for (int i = 1; i < T / 32; ++i) {
            a += sa[i];
            if (Q) b = __uint_as_float(max(__float_as_uint(b), __float_as_uint(sb[i])));
            else b += sb[i];
        }
    }
}

// v rounded to the nearest integer, ties to even, for |v| <= 2^22: the low bits of v + 1.5 * 2^23 (the
// conversion instruction takes several times as long).
__device__ __forceinline__ uint32_t round_bits(float v) { return __float_as_uint(__fadd_rn(v, 12582912.0f)); }

struct RowParams {
    const void* x;
    const void* residual;
    const float* weight;
    void* out;
    void* residual_out;
    float* scale;
    long long rows, x_stride, residual_stride, out_stride, residual_out_stride;
    int cols;
    float eps;
};

// Rows of T = 32 threads share a CTA of 256; longer rows have a CTA each.
template <int T> constexpr int kThreads = T == 32 ? 256 : T;

// T threads take a row, thread i the packs i, i + T, ... (NV of them).
template <typename E, RowWhat WHAT, int V, int T, int NV>
__global__ void __launch_bounds__(kThreads<T>) row_kernel(const RowParams p) {
    const int t = T == 32 ? (threadIdx.x & 31) : threadIdx.x;
    const long long row = T == 32 ? (long long)blockIdx.x * (kThreads<T> / 32) + (threadIdx.x >> 5) : blockIdx.x;
    if (T == 32 && row >= p.rows) return;
    const int n = p.cols;
    const E* x = static_cast<const E*>(p.x) + row * p.x_stride;
    Pack<E, V> px[NV];
    float h[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i) px[i] = load_pack<E, V>(x, (i * T + t) * V, n);
    if (WHAT != kQuantize && p.residual != nullptr) {
        const E* r = static_cast<const E*>(p.residual) + row * p.residual_stride;
        Pack<E, V> pr[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) pr[i] = load_pack<E, V>(r, (i * T + t) * V, n);
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) h[i][j] = to_f(px[i].e[j]) + to_f(pr[i].e[j]);
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) h[i][j] = to_f(px[i].e[j]);
    }
    float sum = 0.0f;
    unsigned top = 0;   // |.| as bits: orders like the values, infinities and NaN on top
    float w[V];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (WHAT == kNormQ8) load_weight<V>(p.weight, (i * T + t) * V, n, w);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            if (WHAT != kQuantize) sum = fmaf(h[i][j], h[i][j], sum);
            if (WHAT != kNorm) {
                const float v = WHAT == kNormQ8 ? h[i][j] * w[j] : h[i][j];
                top = max(top, __float_as_uint(v) & 0x7fffffffu);
            }
        }
    }
    float ftop = __uint_as_float(top);
    reduce_row<T, true>(sum, ftop);
    const float s = WHAT == kQuantize ? 1.0f : rsqrtf(sum / (float)n + p.eps);
    if (p.residual_out != nullptr) {
        E* ho = static_cast<E*>(p.residual_out) + row * p.residual_out_stride;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            Pack<E, V> o;
#pragma unroll
            for (int j = 0; j < V; ++j) o.e[j] = from_f<E>(h[i][j]);
            store_pack<E, V>(ho, (i * T + t) * V, n, o);
        }
    }
    if constexpr (WHAT == kNorm) {
        E* out = static_cast<E*>(p.out) + row * p.out_stride;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            load_weight<V>(p.weight, (i * T + t) * V, n, w);
            Pack<E, V> o;
#pragma unroll
            for (int j = 0; j < V; ++j) o.e[j] = from_f<E>(h[i][j] * s * w[j]);
            store_pack<E, V>(out, (i * T + t) * V, n, o);
        }
    } else {
        const float a = __float_as_uint(ftop) >= 0x7f800000u ? __uint_as_float(0x7fffffffu) : s * ftop;
        const bool finite = fabsf(a) < __uint_as_float(0x7f800000u);
        const float k = finite && a >= kTiny ? 127.0f / a : 0.0f;
        if (t == 0) p.scale[row] = !finite ? __uint_as_float(0x7fffffffu) : a >= kTiny ? a / 127.0f : 0.0f;
        int8_t* out = static_cast<int8_t*>(p.out) + row * p.out_stride;
        const uint32_t keep = finite ? 0xffffffffu : 0u;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (WHAT == kNormQ8) load_weight<V>(p.weight, (i * T + t) * V, n, w);
            Pack<int8_t, V> o;
            uint32_t b[V];
#pragma unroll
            for (int j = 0; j < V; ++j)
                b[j] = round_bits(__fmul_rn(WHAT == kNormQ8 ? h[i][j] * s * w[j] : h[i][j], k)) & keep;
            if constexpr (V >= 4) {
                uint32_t* words = reinterpret_cast<uint32_t*>(&o.word);
#pragma unroll
                for (int j = 0; j < V; j += 4)
                    words[j / 4] = __byte_perm(__byte_perm(b[j], b[j + 1], 0x0040), __byte_perm(b[j + 2], b[j + 3], 0x0040), 0x5410);
            } else {
                o.e[0] = (int8_t)b[0];
            }
            store_pack<int8_t, V>(out, (i * T + t) * V, n, o);
        }
    }
}

template <typename E, RowWhat WHAT, int V, int T, int EPT>
void start_rows(const RowParams& p, cudaStream_t st) {
    const long long per = kThreads<T> / T;
    row_kernel<E, WHAT, V, T, EPT / V><<<(unsigned)((p.rows + per - 1) / per), kThreads<T>, 0, st>>>(p);
}

// Threads for a row, and values for a thread, by the row's length alone.
template <typename E, RowWhat WHAT, int V>
void pick_rows(const RowParams& p, cudaStream_t st) {
    const int n = p.cols;
    if (n <= 256) start_rows<E, WHAT, V, 32, 8>(p, st);
    else if (n <= 512) start_rows<E, WHAT, V, 32, 16>(p, st);
    else if (n <= 768) start_rows<E, WHAT, V, 32, 24>(p, st);
    else if (n <= 1024) start_rows<E, WHAT, V, 32, 32>(p, st);
    else if (n <= 2048) start_rows<E, WHAT, V, 128, 16>(p, st);
    else if (n <= 4096) start_rows<E, WHAT, V, 128, 32>(p, st);
    else if (n <= 8192) start_rows<E, WHAT, V, 256, 32>(p, st);
    else if (n <= 16384) start_rows<E, WHAT, V, 512, 32>(p, st);
    else start_rows<E, WHAT, V, 1024, 32>(p, st);
}

bool on16(const void* p, long long stride_bytes, long long rows) {
    return (uintptr_t)p % 16 == 0 && (rows <= 1 || stride_bytes % 16 == 0);
}
// Whether packs of V values of es bytes can be accessed whole.
bool on_pack(const void* p, long long stride, int es, int V, long long rows) {
    return (uintptr_t)p % (unsigned)(es * V) == 0 && (rows <= 1 || (stride * es) % (es * V) == 0);
}

template <typename E, RowWhat WHAT>
void align_rows(const RowParams& p, cudaStream_t st) {
    constexpr int V = 16 / sizeof(E), es = sizeof(E);
    const bool wide = on_pack(p.x, p.x_stride, es, V, p.rows) &&
                      (p.residual == nullptr || on_pack(p.residual, p.residual_stride, es, V, p.rows)) &&
                      on_pack(p.out, p.out_stride, WHAT == kNorm ? es : 1, V, p.rows) &&
                      (p.residual_out == nullptr || on_pack(p.residual_out, p.residual_out_stride, es, V, p.rows)) &&
                      (uintptr_t)p.weight % 16 == 0;
    if (wide) pick_rows<E, WHAT, V>(p, st);
    else pick_rows<E, WHAT, 1>(p, st);
}

template <typename E>
void type_rows(const RowParams& p, RowWhat what, cudaStream_t st) {
    if (what == kNorm) align_rows<E, kNorm>(p, st);
    else if (what == kNormQ8) align_rows<E, kNormQ8>(p, st);
    else align_rows<E, kQuantize>(p, st);
}

struct GradParams {
    const void* dy;
    const void* h;
    const float* weight;
    const void* dresidual;
    void* dx;
    float* partial;   // gridDim.x rows of cols, or null
    long long rows, dy_stride, h_stride, dresidual_stride, dx_stride;
    int cols;
    float eps;
};

// T threads take a row, T = 32 eight rows to a CTA at a time, which goes
// through the matrix with the grid's stride; thread t keeps the sums of dweight
// for its columns in registers, and the CTA writes them as one partial row.
template <typename E, int V, int T, int NV>
__global__ void __launch_bounds__(kThreads<T>, T == 32 ? 2 : 1) grad_kernel(const GradParams p) {
    constexpr int R = kThreads<T> / T;
    const int t = threadIdx.x % T, n = p.cols;
    float acc[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) acc[i][j] = 0.0f;
    for (long long row = (long long)blockIdx.x * R + threadIdx.x / T; row < p.rows; row += (long long)gridDim.x * R) {
        const E* dy = static_cast<const E*>(p.dy) + row * p.dy_stride;
        const E* h = static_cast<const E*>(p.h) + row * p.h_stride;
        Pack<E, V> py[NV], ph[NV], pr[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            py[i] = load_pack<E, V>(dy, (i * T + t) * V, n);
            ph[i] = load_pack<E, V>(h, (i * T + t) * V, n);
        }
        if (p.dresidual != nullptr) {
            const E* r = static_cast<const E*>(p.dresidual) + row * p.dresidual_stride;
#pragma unroll
            for (int i = 0; i < NV; ++i) pr[i] = load_pack<E, V>(r, (i * T + t) * V, n);
        }
        float hh = 0.0f, gh = 0.0f, w[V];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            load_weight<V>(p.weight, (i * T + t) * V, n, w);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float hv = to_f(ph[i].e[j]);
                hh = fmaf(hv, hv, hh);
                gh = fmaf(to_f(py[i].e[j]) * w[j], hv, gh);
            }
        }
        reduce_row<T, false>(hh, gh);
        const float s = rsqrtf(hh / (float)n + p.eps);
        const float along = gh / (float)n * s * s;
        E* dx = static_cast<E*>(p.dx) + row * p.dx_stride;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            load_weight<V>(p.weight, (i * T + t) * V, n, w);
            Pack<E, V> o;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float hv = to_f(ph[i].e[j]), yv = to_f(py[i].e[j]);
                float d = s * (yv * w[j] - hv * along);
                if (p.dresidual != nullptr) d += to_f(pr[i].e[j]);
                o.e[j] = from_f<E>(d);
                acc[i][j] = fmaf(yv, hv * s, acc[i][j]);
            }
            store_pack<E, V>(dx, (i * T + t) * V, n, o);
        }
    }
    if (p.partial == nullptr) return;
    float* part = p.partial + (long long)blockIdx.x * n;
    if constexpr (R > 1) {
        // the CTA's rows of sums, one after the other
        __shared__ float sums[NV * V * T];
        for (int r = 0; r < R; ++r) {
            if (threadIdx.x / T == r) {
#pragma unroll
                for (int i = 0; i < NV; ++i)
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        float* at = &sums[(i * V + j) * T + t];   // a bank for each thread
                        *at = r == 0 ? acc[i][j] : *at + acc[i][j];
                    }
            }
            __syncthreads();
        }
        for (int c = threadIdx.x; c < n; c += kThreads<T>) {
            const int i = c / (T * V), j = c % V;
            part[c] = sums[(i * V + j) * T + c / V % T];
        }
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int c = (i * T + t) * V + j;
                if (c < n) part[c] = acc[i][j];
            }
    }
}

// dweight = sum of the partial rows: 32 columns to a CTA, 32 rows of threads,
// each summing every 32nd partial in order, then the 32 sums in order.
__global__ void __launch_bounds__(1024) grad_sum_kernel(const float* partial, float* dweight, int parts, int cols) {
    __shared__ float sm[32][33];
    asm volatile("griddepcontrol.wait;" ::: "memory");   // the partial rows are the kernel's before
    const int c = blockIdx.x * 32 + threadIdx.x;
    float v = 0.0f;
    if (c < cols) {
#pragma unroll 5
        for (int r = threadIdx.y; r < parts; r += 32) v += partial[(long long)r * cols + c];
    }
    sm[threadIdx.y][threadIdx.x] = v;
    __syncthreads();
    if (threadIdx.y == 0 && c < cols) {
#pragma unroll
        for (int i = 1; i < 32; ++i) v += sm[i][threadIdx.x];
        dweight[c] = v;
    }
}

template <typename E, int V, int T, int EPT>
void start_grad(const GradParams& p, int parts, cudaStream_t st) {
    grad_kernel<E, V, T, EPT / V><<<parts, kThreads<T>, 0, st>>>(p);
}

template <typename E, int V>
void pick_grad(const GradParams& p, int parts, cudaStream_t st) {
    const int n = p.cols;
    if (n <= 256) start_grad<E, V, 32, 8>(p, parts, st);
    else if (n <= 512) start_grad<E, V, 32, 16>(p, parts, st);
    else if (n <= 1024) start_grad<E, V, 32, 32>(p, parts, st);
    else if (n <= 2048) start_grad<E, V, 128, 16>(p, parts, st);
    else if (n <= 4096) start_grad<E, V, 256, 16>(p, parts, st);
    else if (n <= 8192) start_grad<E, V, 512, 16>(p, parts, st);
    else if (n <= 16384) start_grad<E, V, 1024, 16>(p, parts, st);
    else start_grad<E, V, 1024, 32>(p, parts, st);
}

template <typename E>
void type_grad(const GradParams& p, int parts, cudaStream_t st) {
    constexpr int es = sizeof(E);
    const bool wide = on16(p.dy, p.dy_stride * es, p.rows) && on16(p.h, p.h_stride * es, p.rows) &&
                      (p.dresidual == nullptr || on16(p.dresidual, p.dresidual_stride * es, p.rows)) &&
                      on16(p.dx, p.dx_stride * es, p.rows) && (uintptr_t)p.weight % 16 == 0;
    if (wide) pick_grad<E, 16 / es>(p, parts, st);
    else pick_grad<E, 1>(p, parts, st);
}

// A warp takes kSpan values of a row, V to a lane at a time, the loads first.
constexpr int kSpan = 1024;
template <typename E, int V>
__global__ void __launch_bounds__(256) dequant_kernel(const int8_t* q, const float* scale, E* out, unsigned spans,
                                                      long long q_stride, long long out_stride, int cols,
                                                      unsigned spans_a_row) {
    constexpr int NV = V == 1 ? 4 : kSpan / (32 * V), LOOPS = kSpan / (32 * V * NV);
    const unsigned span = blockIdx.x * 8u + (threadIdx.x >> 5);
    if (span >= spans) return;
    const unsigned row = span / spans_a_row;
    const int c0 = (int)(span - row * spans_a_row) * kSpan, lane = threadIdx.x & 31;
    const float s = scale[row];
    const int8_t* src = q + row * q_stride;
    E* dst = out + row * out_stride;
    for (int l = 0; l < LOOPS; ++l) {
        Pack<int8_t, V> in[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = c0 + ((l * NV + i) * 32 + lane) * V;
            if (c + V <= cols) in[i].word = *reinterpret_cast<const typename Word<V>::T*>(src + c);
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = c0 + ((l * NV + i) * 32 + lane) * V;
            if (c + V <= cols) {
                Pack<E, V> o;
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    // the byte u = q + 128 as 2^23 + u, exactly
                    const uint32_t u = (uint32_t)(uint8_t)in[i].e[j] ^ 0x80u;
                    o.e[j] = from_f<E>((__uint_as_float(0x4B000000u | u) - 8388736.0f) * s);
                }
                *reinterpret_cast<typename Word<sizeof(E) * V>::T*>(dst + c) = o.word;
            } else {
                for (int j = c; j < cols; ++j) dst[j] = from_f<E>((float)src[j] * s);
            }
        }
    }
}

template <typename E>
int type_dequant(const DequantArgs& a, cudaStream_t st) {
    constexpr int V = 16 / sizeof(E);
    const bool wide = on_pack(a.q, a.q_stride, 1, V, a.rows) && on_pack(a.out, a.out_stride, sizeof(E), V, a.rows);
    const long long spans_a_row = (a.cols + kSpan - 1) / kSpan;
    // rows beyond a grid's reach in further launches
    for (long long r0 = 0; r0 < a.rows;) {
        const long long most = (1LL << 31) / spans_a_row, rows = a.rows - r0 < most ? a.rows - r0 : most;
        const unsigned spans = (unsigned)(rows * spans_a_row), grid = (spans + 7) / 8;
        const int8_t* q = a.q + r0 * a.q_stride;
        E* out = static_cast<E*>(a.out) + r0 * a.out_stride;
        if (wide)
            dequant_kernel<E, V><<<grid, 256, 0, st>>>(q, a.scale + r0, out, spans, a.q_stride, a.out_stride, a.cols,
                                                       (unsigned)spans_a_row);
        else
            dequant_kernel<E, 1><<<grid, 256, 0, st>>>(q, a.scale + r0, out, spans, a.q_stride, a.out_stride, a.cols,
                                                       (unsigned)spans_a_row);
        const int rc = launched("dequantisation kernel");
        if (rc != TR_OK) return rc;
        r0 += rows;
    }
    return TR_OK;
}

}  // namespace

int launch_rows(const RowArgs& a) {
    RowParams p{a.x, a.residual, a.weight, a.out, a.residual_out, a.scale, a.rows, a.x_stride, a.residual_stride,
                a.out_stride, a.residual_out_stride, a.cols, a.eps};
    cudaStream_t st = static_cast<cudaStream_t>(a.stream);
    if (a.dtype == TR_ELEM_F32) type_rows<float>(p, a.what, st);
    else if (a.dtype == TR_ELEM_F16) type_rows<__half>(p, a.what, st);
    else type_rows<__nv_bfloat16>(p, a.what, st);
    return launched("row kernel");
}

int row_grad_parts(long long rows, long long cols) {
    // the CTAs that 152 SMs hold at once, a row for each thread group at least
    const long long per = cols <= 1024 ? 8 : 1;
    const long long want = 152 * (cols <= 1024 ? 2 : cols <= 2048 ? 8 : cols <= 4096 ? 4 : cols <= 8192 ? 2 : 1);
    const long long most = (rows + per - 1) / per;
    return (int)(most < want ? (most < 1 ? 1 : most) : want);
}

int launch_row_grad(const RowGradArgs& a) {
    GradParams p{a.dy, a.h, a.weight, a.dresidual, a.dx, a.dweight != nullptr ? a.partial : nullptr, a.rows,
                 a.dy_stride, a.h_stride, a.dresidual_stride, a.dx_stride, a.cols, a.eps};
    cudaStream_t st = static_cast<cudaStream_t>(a.stream);
    const int parts = row_grad_parts(a.rows, a.cols);
    if (a.dtype == TR_ELEM_F32) type_grad<float>(p, parts, st);
    else if (a.dtype == TR_ELEM_F16) type_grad<__half>(p, parts, st);
    else type_grad<__nv_bfloat16>(p, parts, st);
    int rc = launched("row gradient kernel");
    if (rc != TR_OK || a.dweight == nullptr) return rc;
    // its start overlaps the end of the kernel that it waits for
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)((a.cols + 31) / 32));
    cfg.blockDim = dim3(32, 32);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, grad_sum_kernel, (const float*)a.partial, a.dweight, parts, a.cols);
    if (e != cudaSuccess) {
        set_last_error("cudaLaunchKernelEx(weight gradient sum)", (int)e);
        return TR_ERR_CUDA;
    }
    return launched("weight gradient sum kernel");
}

int launch_dequant(const DequantArgs& a) {
    cudaStream_t st = static_cast<cudaStream_t>(a.stream);
    if (a.dtype == TR_ELEM_F32) return type_dequant<float>(a, st);
    if (a.dtype == TR_ELEM_F16) return type_dequant<__half>(a, st);
    return type_dequant<__nv_bfloat16>(a, st);
}

}  // namespace trfn
