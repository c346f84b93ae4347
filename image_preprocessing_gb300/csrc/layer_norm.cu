// Layer norm with the residual's addition (output in the input's type or in 8
// bits), and its gradients.
//
// Mathematics, for a row h = x + r of n values:
//     m = sum_c h_c / n,  s = 1/sqrt(sum_c (h_c - m)^2 / n + eps)
//     y_c = (h_c - m) s w_c + b_c
//     8 bits: a = max_c |y_c|, scale = a/127, q_c = rint(y_c 127/a)
//     gradients, with u_c = h_c - m and g_c = dy_c w_c:
//     dx_c = s (g_c - sum_j g_j / n - u_c s^2 (sum_j g_j u_j) / n) + dres_c
//     dw_c = sum_rows dy_c u_c s,  db_c = sum_rows dy_c
//
// Bound by HBM, like the RMS norm (row_ops.cu), whose layout this keeps: a row
// is read once into registers, in packs of 16 bytes at any phase.  The squares
// are of the values less their mean, a second reduction of the registers: from
// sums of h and h^2 alone a mean far from zero would cancel the variance away.
// b keeps max |y| from following from max |h w|: 8 bits take a third reduction.
// Measured (of the 6.78 TB/s copy rate): 50176 x 1024 binary16 62.5 us (0.97), 12544 x
// 4096 bfloat16 64 us (0.94) and with 8-bit output 60 us (0.86; the instructions take
// 61 % of the issue slots); 50176 x 999 91 us (0.65: shifted packs).
#include "row_parts.h"

namespace trfn {
namespace {

struct LayerParams {
    const void* x;
    const void* residual;
    const float* weight;
    const float* bias;
    void* out;
    void* residual_out;
    float* scale;
    long long rows, x_stride, residual_stride, out_stride, residual_out_stride;
    int cols;
    float eps;
};

// CTAs of one-warp rows that an SM is to hold: enough rows under way, without spills.
template <int V, int T, bool Q8>
constexpr int kLayerResident = T > 32 || V == 1 ? 1 : Q8 ? 3 : V == 8 ? 4 : 2;

// T threads take a row, thread i the packs i, i + T, ... (NV of them).
template <typename E, bool Q8, int V, int T, int NV, bool SHIFT>
__global__ void __launch_bounds__(kThreads<T>, kLayerResident<V, T, Q8>) layer_kernel(const LayerParams p) {
    extern __shared__ float shared_weight[];   // with SHIFT: weights, then biases
    wait_for_previous();
    const int t = threadIdx.x % T;
    const long long row = (long long)blockIdx.x * (kThreads<T> / T) + threadIdx.x / T;
    const bool some = T > 32 || row < p.rows;   // (threads of no row stay for the barrier, or for their warp)
    if (T == 32 && !SHIFT && !some) return;
    const int n = some ? p.cols : 0, shift = SHIFT ? (int)((row * p.x_stride) & (V - 1)) : 0, c0 = t * V - shift;
    const E* x = static_cast<const E*>(p.x) + row * p.x_stride;
    Pack<E, V> px[NV], pr[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) px[i] = load_pack<E, V>(x, i * T * V + c0, n, SHIFT && may_over(row, p.rows, p.x_stride, V));
    const bool add = p.residual != nullptr;
    if (add) {
        const E* r = static_cast<const E*>(p.residual) + row * p.residual_stride;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            pr[i] = load_pack<E, V>(r, i * T * V + c0, n, SHIFT && may_over(row, p.rows, p.residual_stride, V));
    }
    float* const shared_bias = shared_weight + (SHIFT ? V * shift_pitch<V>(p.cols) : 0);
    if constexpr (SHIFT && T <= 32) {   // while the rows are on their way
        share_weight<V>(p.weight, shared_weight, p.cols);
        share_weight<V>(p.bias, shared_bias, p.cols, 0.0f);
        __syncthreads();
    }
    if (T == 32 && !some) return;
    // values in pairs: half the instructions, which compete with HBM here
    constexpr int N = NV * V, P = N / 2;   // pair k: values 2 k and 2 k + 1, value e of pack e / V
    static_assert(N % 2 == 0, "values are taken in pairs");
    auto pair = [&](const Pack<E, V> (&v)[NV], int k) { return two(to_f(v[2 * k / V].e[2 * k % V]), to_f(v[(2 * k + 1) / V].e[(2 * k + 1) % V])); };
    auto column = [&](int e) { return e / V * (T * V) + c0 + e % V; };
    auto in_row = [&](int e) { return column(e) >= 0 && column(e) < n; };
    Two h[P];
    __shared__ float between[3][kRowWarps<T>];   // of the sum, the squares, the maximum
    Two sum2 = two(0.0f, 0.0f);
#pragma unroll
    for (int k = 0; k < P; ++k) {
        h[k] = add ? add_two(pair(px, k), pair(pr, k)) : pair(px, k);
        sum2 = add_two(sum2, h[k]);   // (zeros outside the row)
    }
    const float sum = apart(sum2).x + apart(sum2).y;
    auto value = [&](int e) { return e % 2 ? apart(h[e / 2]).y : apart(h[e / 2]).x; };
    if (p.residual_out != nullptr) {
        E* ho = static_cast<E*>(p.residual_out) + row * p.residual_out_stride;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            Pack<E, V> o;
#pragma unroll
            for (int j = 0; j < V; ++j) o.e[j] = from_f<E>(value(i * V + j));
            store_pack<E, V>(ho, i * T * V + c0, n, o);
        }
    }
    const float mean = row_sum<T>(sum, between[0]) / (float)n;
    const Two less = two(-mean, -mean);
    Two squares2 = two(0.0f, 0.0f);
#pragma unroll
    for (int k = 0; k < P; ++k) {
        h[k] = add_two(h[k], less);
        // (whole packs need no look at each value)
        const int c = 2 * k / V * (T * V) + c0;
        if (V == 1 || c < 0 || c + V > n) {
            const float2 v = apart(h[k]);
            h[k] = two(in_row(2 * k) ? v.x : 0.0f, in_row(2 * k + 1) ? v.y : 0.0f);
        }
        squares2 = fma_two(h[k], h[k], squares2);
    }
    const float squares = apart(squares2).x + apart(squares2).y;
    const float s = rsqrtf(row_sum<T>(squares, between[1]) / (float)n + p.eps);
    const Two s2 = two(s, s);
    unsigned top = 0;   // |.| as bits: orders like the values, infinities and NaN on top
    float w[V], b[V];
#pragma unroll
    for (int k = 0; k < P; ++k) {
        const int i = 2 * k / V, j = 2 * k % V;
        Two wk, bk;
        if constexpr (V > 1) {
            if (j == 0) {
                load_weight<V, SHIFT, T <= 32>(p.weight, shared_weight, i * T * V + c0, i * T + t, shift, n, w);
                load_weight<V, SHIFT, T <= 32>(p.bias, shared_bias, i * T * V + c0, i * T + t, shift, n, b, 0.0f);
            }
            wk = two(w[j], w[(j + 1) % V]);
            bk = two(b[j], b[(j + 1) % V]);
        } else {
            wk = two(p.weight == nullptr ? 1.0f : in_row(2 * k) ? p.weight[column(2 * k)] : 0.0f,
                     p.weight == nullptr ? 1.0f : in_row(2 * k + 1) ? p.weight[column(2 * k + 1)] : 0.0f);
            bk = two(p.bias != nullptr && in_row(2 * k) ? p.bias[column(2 * k)] : 0.0f,
                     p.bias != nullptr && in_row(2 * k + 1) ? p.bias[column(2 * k + 1)] : 0.0f);
        }
        h[k] = fma_two(mul_two(h[k], s2), wk, bk);
        if constexpr (Q8) {
            const float2 y = apart(h[k]);
            // (places outside the row are zeros, but in shifted packs they may hold some other value's bias)
            if (!SHIFT || in_row(2 * k)) top = max(top, __float_as_uint(y.x) & 0x7fffffffu);
            if (!SHIFT || in_row(2 * k + 1)) top = max(top, __float_as_uint(y.y) & 0x7fffffffu);
        }
    }
    if constexpr (!Q8) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            Pack<E, V> o;
#pragma unroll
            for (int j = 0; j < V; ++j) o.e[j] = from_f<E>(value(i * V + j));
            store_pack<E, V>(static_cast<E*>(p.out) + row * p.out_stride, i * T * V + c0, n, o);
        }
    } else {
        const float a = __uint_as_float(row_top<T>(top, between[2]));
        const bool finite = __float_as_uint(a) < 0x7f800000u;
        const float scale = finite && a >= kTiny ? 127.0f / a : 0.0f;
        if (t == 0 && some) p.scale[row] = !finite ? __uint_as_float(0x7fffffffu) : a >= kTiny ? a / 127.0f : 0.0f;
        int8_t* out = static_cast<int8_t*>(p.out) + row * p.out_stride;
        const uint32_t keep = finite ? 0xffffffffu : 0u;
        const Two scale2 = two(scale, scale), round2 = two(12582912.0f, 12582912.0f);   // (round_bits, of two values)
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            Pack<int8_t, V> o;
            uint32_t bits[V];
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float2 v = apart(add_two(mul_two(h[(i * V + j) / 2], scale2), round2));
                bits[j] = __float_as_uint((i * V + j) % 2 ? v.y : v.x) & keep;
            }
            if constexpr (V >= 4) {
                uint32_t* words = reinterpret_cast<uint32_t*>(&o.word);
#pragma unroll
                for (int j = 0; j < V; j += 4)
                    words[j / 4] = __byte_perm(__byte_perm(bits[j], bits[j + 1], 0x0040), __byte_perm(bits[j + 2], bits[j + 3], 0x0040), 0x5410);
            } else {
                o.e[0] = (int8_t)bits[0];
            }
            store_pack<int8_t, V>(out, i * T * V + c0, n, o);
        }
    }
}

template <typename E, bool Q8, int V, int T, int EPT, bool SHIFT>
int start_layer(const LayerParams& p, cudaStream_t st) {
    const long long per = kThreads<T> / T;
    const size_t smem = SHIFT && T <= 32 ? 2 * V * shift_pitch<V>(p.cols) * sizeof(float) : 0;
    return launch_row_kernel("layer norm kernel", layer_kernel<E, Q8, V, T, EPT / V, SHIFT>, (unsigned)((p.rows + per - 1) / per),
                             kThreads<T>, smem, st, p);
}

// Threads for a row, and values for a thread, by the row's length alone.
template <typename E, bool Q8, int V, bool SHIFT>
int pick_layer(const LayerParams& p, cudaStream_t st) {
    const int n = p.cols + (SHIFT ? V - 1 : 0);
    if (n <= 64) return start_layer<E, Q8, V, 8, 8, SHIFT>(p, st);
    if (n <= 128) return start_layer<E, Q8, V, 8, 16, SHIFT>(p, st);
    if (n <= 256) return start_layer<E, Q8, V, 32, 8, SHIFT>(p, st);
    if (n <= 512) return start_layer<E, Q8, V, 32, 16, SHIFT>(p, st);
    if (n <= 768) return start_layer<E, Q8, V, 32, 24, SHIFT>(p, st);
    if (n <= 1024) return start_layer<E, Q8, V, 32, 32, SHIFT>(p, st);
    if (n <= 2048) return start_layer<E, Q8, V, 128, 16, SHIFT>(p, st);
    if (n <= 4096) return start_layer<E, Q8, V, 128, 32, SHIFT>(p, st);
    if (SHIFT || n <= 8192) return start_layer<E, Q8, V, SHIFT ? 512 : 256, SHIFT ? 24 : 32, SHIFT>(p, st);
    if constexpr (!SHIFT) {
        if (n <= 16384) return start_layer<E, Q8, V, 512, 32, SHIFT>(p, st);
        return start_layer<E, Q8, V, 1024, 32, SHIFT>(p, st);
    }
    return TR_ERR_NOT_SUPPORTED;   // not reached
}

template <typename E, bool Q8>
int align_layer(const LayerParams& p, cudaStream_t st) {
    constexpr int es = sizeof(E), V = 16 / es;
    Phase phase;
    phase.add(p.x, p.x_stride, es, V, p.rows);
    phase.add(p.residual, p.residual_stride, es, V, p.rows);
    phase.add(p.out, p.out_stride, Q8 ? 1 : es, V, p.rows);
    phase.add(p.residual_out, p.residual_out_stride, es, V, p.rows);
    if (phase.f == 0 && (uintptr_t)p.weight % 16 == 0 && (uintptr_t)p.bias % 16 == 0) return pick_layer<E, Q8, V, false>(p, st);
    if (phase.f >= 0 && p.cols <= kShiftCols) return pick_layer<E, Q8, V, true>(p, st);
    return pick_layer<E, Q8, 1, false>(p, st);
}

template <typename E>
int type_layer(const LayerParams& p, bool q8, cudaStream_t st) {
    return q8 ? align_layer<E, true>(p, st) : align_layer<E, false>(p, st);
}

}  // namespace

int launch_layer_norm(const RowArgs& a) {
    LayerParams p{a.x, a.residual, a.weight, a.bias, a.out, a.residual_out, a.scale, a.rows, a.x_stride, a.residual_stride,
                  a.out_stride, a.residual_out_stride, a.cols, a.eps};
    cudaStream_t st = static_cast<cudaStream_t>(a.stream);
    const bool q8 = a.what == kNormQ8;
    if (a.dtype == TR_ELEM_F32) return type_layer<float>(p, q8, st);
    if (a.dtype == TR_ELEM_F16) return type_layer<__half>(p, q8, st);
    return type_layer<__nv_bfloat16>(p, q8, st);
}

}  // namespace trfn
