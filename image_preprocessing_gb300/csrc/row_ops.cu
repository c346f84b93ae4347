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
//
// Rows are accessed in packs of 16 bytes.  Where a row's length is odd, its
// rows start off the 16-byte boundaries, but all matrices of a call alike
// (the usual case: equal strides, aligned buffers): then row r starts
// s = r * stride mod V values into a pack, and lane i's pack holds columns
// i V - s ... (SHIFT).  Any other alignment goes value by value.
//
// Measured (of the 6.79 TB/s copy rate): norm with residual 50176 x 1024
// binary16 61.3 us (0.99), 12544 x 4096 bfloat16 61.8 us (0.98) and with 8-bit
// output 54.4 us (0.97); quantisation 50176 x 768 20.6 us (0.83), reading back
// 18.2 us (0.93); gradients 50176 x 1024 77.0 us (0.79), 12544 x 4096 74.2 us
// (0.82), where the instructions, 22 a value with the weights' sums, take half of
// the issue slots.  With shifted packs the ends of rows cost instructions: norm
// 50176 x 999 80.7 us (0.73).  Above 8192 values a row has a CTA of 512
// or 1024 threads, few of which fit an SM: norm 8192 x 16384 bfloat16 184 us (0.86),
// quantisation 8192 x 16384 binary16 118 us (0.50).
#include "row_parts.h"

namespace trfn {
namespace {

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

// CTAs of one-warp rows that an SM is to hold: enough rows under way, without spills.
template <int V, int T, RowWhat WHAT>
constexpr int kResident = T > 32 || V == 1 ? 1 : WHAT == kNormQ8 ? 3 : WHAT == kQuantize ? (V == 8 ? 5 : 4) : (V == 8 ? 4 : 2);

// T threads take a row, thread i the packs i, i + T, ... (NV of them).
template <typename E, RowWhat WHAT, int V, int T, int NV, bool SHIFT>
__global__ void __launch_bounds__(kThreads<T>, kResident<V, T, WHAT>) row_kernel(const RowParams p) {
    extern __shared__ float shared_weight[];   // with SHIFT
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
    const bool add = WHAT != kQuantize && p.residual != nullptr;
    if (add) {
        const E* r = static_cast<const E*>(p.residual) + row * p.residual_stride;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            pr[i] = load_pack<E, V>(r, i * T * V + c0, n, SHIFT && may_over(row, p.rows, p.residual_stride, V));
    }
    if constexpr (SHIFT && T <= 32 && WHAT != kQuantize) {   // while the rows are on their way
        share_weight<V>(p.weight, shared_weight, p.cols);
        __syncthreads();
    }
    if (T == 32 && !some) return;
    float h[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) h[i][j] = add ? to_f(px[i].e[j]) + to_f(pr[i].e[j]) : to_f(px[i].e[j]);
    if (p.residual_out != nullptr) {
        E* ho = static_cast<E*>(p.residual_out) + row * p.residual_out_stride;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            Pack<E, V> o;
#pragma unroll
            for (int j = 0; j < V; ++j) o.e[j] = from_f<E>(h[i][j]);
            store_pack<E, V>(ho, i * T * V + c0, n, o);
        }
    }
    float sum = 0.0f;
    unsigned top = 0;   // |.| as bits: orders like the values, infinities and NaN on top
    float w[V];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (WHAT == kNormQ8) load_weight<V, SHIFT, T <= 32>(p.weight, shared_weight, i * T * V + c0, i * T + t, shift, n, w);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            if (WHAT != kQuantize) sum = fmaf(h[i][j], h[i][j], sum);
            if (WHAT == kNormQ8) h[i][j] *= w[j];   // 8 bits are made of h w
            if (WHAT != kNorm) top = max(top, __float_as_uint(h[i][j]) & 0x7fffffffu);
        }
    }
    float ftop = __uint_as_float(top);
    reduce_row<T, true>(sum, ftop);
    const float s = WHAT == kQuantize ? 1.0f : rsqrtf(sum / (float)n + p.eps);
    if constexpr (WHAT == kNorm) {
        E* out = static_cast<E*>(p.out) + row * p.out_stride;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            load_weight<V, SHIFT, T <= 32>(p.weight, shared_weight, i * T * V + c0, i * T + t, shift, n, w);
            Pack<E, V> o;
#pragma unroll
            for (int j = 0; j < V; ++j) o.e[j] = from_f<E>(h[i][j] * s * w[j]);
            store_pack<E, V>(out, i * T * V + c0, n, o);
        }
    } else {
        const float a = __float_as_uint(ftop) >= 0x7f800000u ? __uint_as_float(0x7fffffffu) : s * ftop;
        const bool finite = fabsf(a) < __uint_as_float(0x7f800000u);
        const float k = finite && a >= kTiny ? 127.0f / a : 0.0f;
        if (t == 0 && some) p.scale[row] = !finite ? __uint_as_float(0x7fffffffu) : a >= kTiny ? a / 127.0f : 0.0f;
        int8_t* out = static_cast<int8_t*>(p.out) + row * p.out_stride;
        const uint32_t keep = finite ? 0xffffffffu : 0u;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            Pack<int8_t, V> o;
            uint32_t b[V];
#pragma unroll
            for (int j = 0; j < V; ++j)
                b[j] = round_bits(__fmul_rn(WHAT == kNormQ8 ? h[i][j] * s : h[i][j], k)) & keep;
            if constexpr (V >= 4) {
                uint32_t* words = reinterpret_cast<uint32_t*>(&o.word);
#pragma unroll
                for (int j = 0; j < V; j += 4)
                    words[j / 4] = __byte_perm(__byte_perm(b[j], b[j + 1], 0x0040), __byte_perm(b[j + 2], b[j + 3], 0x0040), 0x5410);
            } else {
                o.e[0] = (int8_t)b[0];
            }
            store_pack<int8_t, V>(out, i * T * V + c0, n, o);
        }
    }
}


template <typename E, RowWhat WHAT, int V, int T, int EPT, bool SHIFT>
int start_rows(const RowParams& p, cudaStream_t st) {
    const long long per = kThreads<T> / T;
    const size_t smem = SHIFT && T <= 32 && WHAT != kQuantize ? V * shift_pitch<V>(p.cols) * sizeof(float) : 0;
    return launch_row_kernel("row kernel", row_kernel<E, WHAT, V, T, EPT / V, SHIFT>, (unsigned)((p.rows + per - 1) / per),
                             kThreads<T>, smem, st, p);
}

// Threads for a row, and values for a thread, by the row's length alone.
template <typename E, RowWhat WHAT, int V, bool SHIFT>
int pick_rows(const RowParams& p, cudaStream_t st) {
    const int n = p.cols + (SHIFT ? V - 1 : 0);
    if (n <= 64) return start_rows<E, WHAT, V, 8, 8, SHIFT>(p, st);
    if (n <= 128) return start_rows<E, WHAT, V, 8, 16, SHIFT>(p, st);
    if (n <= 256) return start_rows<E, WHAT, V, 32, 8, SHIFT>(p, st);
    if (n <= 512) return start_rows<E, WHAT, V, 32, 16, SHIFT>(p, st);
    if (n <= 768) return start_rows<E, WHAT, V, 32, 24, SHIFT>(p, st);
    if (n <= 1024) return start_rows<E, WHAT, V, 32, 32, SHIFT>(p, st);
    if (n <= 2048) return start_rows<E, WHAT, V, 128, 16, SHIFT>(p, st);
    if (n <= 128 * 24) return start_rows<E, WHAT, V, 128, 24, SHIFT>(p, st);
    if (n <= 4096) return start_rows<E, WHAT, V, 128, 32, SHIFT>(p, st);
    if (SHIFT || n <= 8192) return start_rows<E, WHAT, V, SHIFT ? 512 : 256, SHIFT ? 24 : 32, SHIFT>(p, st);
    if constexpr (!SHIFT) {
        if (n <= 16384) return start_rows<E, WHAT, V, 512, 32, SHIFT>(p, st);
        return start_rows<E, WHAT, V, 1024, 32, SHIFT>(p, st);
    }
    return TR_ERR_NOT_SUPPORTED;   // not reached
}

template <typename E, RowWhat WHAT>
int align_rows(const RowParams& p, cudaStream_t st) {
    constexpr int es = sizeof(E), V = 16 / es;
    Phase phase;
    phase.add(p.x, p.x_stride, es, V, p.rows);
    phase.add(p.residual, p.residual_stride, es, V, p.rows);
    phase.add(p.out, p.out_stride, WHAT == kNorm ? es : 1, V, p.rows);
    phase.add(p.residual_out, p.residual_out_stride, es, V, p.rows);
    if (phase.f == 0 && (uintptr_t)p.weight % 16 == 0) return pick_rows<E, WHAT, V, false>(p, st);
    if (phase.f >= 0 && p.cols <= kShiftCols) return pick_rows<E, WHAT, V, true>(p, st);
    return pick_rows<E, WHAT, 1, false>(p, st);
}

template <typename E>
int type_rows(const RowParams& p, RowWhat what, cudaStream_t st) {
    if (what == kNorm) return align_rows<E, kNorm>(p, st);
    if (what == kNormQ8) return align_rows<E, kNormQ8>(p, st);
    return align_rows<E, kQuantize>(p, st);
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
// through the matrix with the grid's stride.  A thread's columns are the same
// in every row, so it keeps their weights and their sums of dweight in
// registers, and the CTA writes the sums as one partial row.  (With SHIFT the
// columns depend on the row's place in a pack; the grid and the rows of a CTA
// are multiples of 8, so that this stays the same too.)  The arithmetic
// competes with HBM: it works on pairs of binary32.
//
// A thread copies its packs of the next rows into shared memory while it works
// on this one; they are its own, so no barrier is needed.  kAhead rows ahead:
// about 100 KB an SM under way, what its share of the HBM rate takes.
//
// Above 8192 columns 1024 threads leave 64 registers to a thread, and weights,
// sums and packs spill (0.5 KB a thread up to 16384 columns, 2.3 to 3.2 KB above,
// where binary32 rows are not copied ahead either): 8192 x 8192 bfloat16 99 us
// (0.80 of the copy rate), 8192 x 12288 404 us (0.29), 4096 x 32768 1303 us (0.12).
template <int V, int T, int NV> constexpr int kRowBytes = V > 1 ? 3 * NV * 16 * kThreads<T> : 0;
template <int V, int T, int NV>
constexpr int kAhead = V == 1 ? 0 : (V == 8 ? 3 : 2) * kRowBytes<V, T, NV> <= 200 * 1024 ? (V == 8 ? 3 : 2) : 200 * 1024 / kRowBytes<V, T, NV>;

template <typename E, int V, int T, int NV, bool SHIFT>
__global__ void __launch_bounds__(kThreads<T>) grad_kernel(const GradParams p) {
    constexpr int R = kThreads<T> / T, N = NV * V;   // N values to a thread
    static_assert(N % 2 == 0, "values are taken in pairs");
    constexpr int AHEAD = kAhead<V, T, NV>;
    extern __shared__ __align__(16) uint8_t dynamic[];
    wait_for_previous();
    uint4* const mine = reinterpret_cast<uint4*>(dynamic) + threadIdx.x;   // AHEAD x 3 NV packs, kThreads<T> apart
    const int t = threadIdx.x % T, n = p.cols;
    const long long row0 = (long long)blockIdx.x * R + threadIdx.x / T, step = (long long)gridDim.x * R;
    const int c0 = t * V - (SHIFT ? (int)((row0 * p.h_stride) & (V - 1)) : 0);
    auto column = [&](int e) { return e / V * (T * V) + c0 + e % V; };
    auto in_row = [&](int e) { return column(e) >= 0 && column(e) < n; };
    // packs inside the row, and (SHIFT) those across its ends, which are read whole but in the last row
    bool inside[NV], across[NV];
    const bool strides_over = p.dy_stride >= V && p.h_stride >= V && (p.dresidual == nullptr || p.dresidual_stride >= V);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = i * T * V + c0;
        inside[i] = c >= 0 && c + V <= n;
        across[i] = SHIFT && strides_over && !inside[i] && c < n;
    }
    const E* dy_next = static_cast<const E*>(p.dy) + row0 * p.dy_stride + c0;
    const E* h_next = static_cast<const E*>(p.h) + row0 * p.h_stride + c0;
    const E* r_next = static_cast<const E*>(p.dresidual) + (p.dresidual != nullptr ? row0 * p.dresidual_stride + c0 : 0);
    long long row_next = row0;
    auto fetch = [&](int slot) {
        if constexpr (AHEAD > 0) {
            if (row_next < p.rows) {
                const bool over = row_next + 1 < p.rows;
                uint32_t to = (uint32_t)__cvta_generic_to_shared(mine) + slot * (3 * NV * 16 * kThreads<T>);
                auto one = [&](const E* from) {
#pragma unroll
                    for (int i = 0; i < NV; ++i)
                        if (inside[i] || (across[i] && over))
                            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + i * (16 * kThreads<T>)),
                                         "l"(from + i * T * V)
                                         : "memory");
                    to += NV * 16 * kThreads<T>;
                };
                one(dy_next);
                one(h_next);
                if (p.dresidual != nullptr) one(r_next);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
            row_next += step;
            dy_next += step * p.dy_stride;
            h_next += step * p.h_stride;
            if (p.dresidual != nullptr) r_next += step * p.dresidual_stride;
        }
    };
    // a pack that was copied, or one across an end of the last row
    auto take = [&](const void* base, long long stride, int m, int i, long long row, bool over, int slot) {
        const int c = i * T * V + c0;
        if constexpr (AHEAD > 0) {
            if (inside[i] || (across[i] && over)) {
                Pack<E, V> pack;
                *reinterpret_cast<uint4*>(&pack.word) = mine[((slot * 3 + m) * NV + i) * kThreads<T>];
                if (SHIFT && !inside[i])
#pragma unroll
                    for (int j = 0; j < V; ++j)
                        if (c + j < 0 || c + j >= n) pack.e[j] = from_f<E>(0.0f);
                return pack;
            }
        }
        return load_pack<E, V>(static_cast<const E*>(base) + row * stride, c, n, false);
    };
    Two acc[N / 2], w[N / 2];
#pragma unroll
    for (int e = 0; e < N; e += 2) {
        acc[e / 2] = two(0.0f, 0.0f);
        w[e / 2] = two(p.weight != nullptr && in_row(e) ? p.weight[column(e)] : 1.0f,
                       p.weight != nullptr && in_row(e + 1) ? p.weight[column(e + 1)] : 1.0f);
    }
    for (int a = 0; a < AHEAD; ++a) fetch(a);
    E* dx = static_cast<E*>(p.dx) + row0 * p.dx_stride;
    int slot = 0;
    for (long long row = row0; row < p.rows; row += step) {
        const bool over = row + 1 < p.rows;
        Pack<E, V> py[NV], ph[NV], pr[NV];
        if constexpr (AHEAD > 0) asm volatile("cp.async.wait_group %0;" ::"n"(AHEAD - 1) : "memory");
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            py[i] = take(p.dy, p.dy_stride, 0, i, row, over, slot);
            ph[i] = take(p.h, p.h_stride, 1, i, row, over, slot);
            if (p.dresidual != nullptr) pr[i] = take(p.dresidual, p.dresidual_stride, 2, i, row, over, slot);
        }
        auto pair = [&](const Pack<E, V> (&v)[NV], int e) {
            return two(to_f(v[e / V].e[e % V]), to_f(v[(e + 1) / V].e[(e + 1) % V]));
        };
        Two hh2 = two(0.0f, 0.0f), gh2 = two(0.0f, 0.0f);
#pragma unroll
        for (int e = 0; e < N; e += 2) {
            const Two h = pair(ph, e);
            hh2 = fma_two(h, h, hh2);
            gh2 = fma_two(mul_two(pair(py, e), w[e / 2]), h, gh2);
        }
        fetch(slot);   // the packs are in registers
        if (++slot >= AHEAD) slot = 0;
        float hh = apart(hh2).x + apart(hh2).y, gh = apart(gh2).x + apart(gh2).y;
        reduce_row<T, false>(hh, gh);
        // dx = s g - (s^3 gh / n) h + dres
        const float s = rsqrtf(hh / (float)n + p.eps), along = -(gh / (float)n * s * s * s);
        const Two s2 = two(s, s), along2 = two(along, along);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            Pack<E, V> o;
#pragma unroll
            for (int j = 0; j < V; j += 2) {
                // (V = 1: pairs are of two packs; the second pack's half is made with it)
                const int e = V > 1 ? i * V + j : i / 2 * 2;
                const Two h = pair(ph, e), y = pair(py, e);
                const Two r = p.dresidual != nullptr ? pair(pr, e) : two(0.0f, 0.0f);
                const float2 d = apart(fma_two(s2, mul_two(y, w[e / 2]), fma_two(along2, h, r)));
                if constexpr (V > 1) {
                    o.e[j] = from_f<E>(d.x);
                    o.e[j + 1] = from_f<E>(d.y);
                    acc[e / 2] = fma_two(y, mul_two(h, s2), acc[e / 2]);
                } else {
                    o.e[0] = from_f<E>(i % 2 ? d.y : d.x);
                    if (i % 2 == 0) acc[e / 2] = fma_two(y, mul_two(h, s2), acc[e / 2]);
                }
            }
            store_pack<E, V>(dx, i * T * V + c0, n, o);
        }
        dx += step * p.dx_stride;
    }
    if (p.partial == nullptr) return;
    float* part = p.partial + (long long)blockIdx.x * n;
    if constexpr (R > 1) {
        // the sums of the CTA's row groups, one after the other
        // (place c + c / 32: the threads' values, V columns apart, in different banks)
        __shared__ float sums[padded(N * T)];
        for (int g = 0; g < R; ++g) {
            if (threadIdx.x / T == g) {
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    const float v = e % 2 ? apart(acc[e / 2]).y : apart(acc[e / 2]).x;
                    if (in_row(e)) sums[padded(column(e))] = g == 0 ? v : sums[padded(column(e))] + v;
                }
            }
            __syncthreads();
        }
        for (int c = threadIdx.x; c < n; c += kThreads<T>) part[c] = sums[padded(c)];
    } else {
#pragma unroll
        for (int e = 0; e < N; ++e)
            if (in_row(e)) part[column(e)] = e % 2 ? apart(acc[e / 2]).y : apart(acc[e / 2]).x;
    }
}

template <typename E, int V, int T, int EPT, bool SHIFT>
int start_grad(const GradParams& p, int parts, cudaStream_t st) {
    constexpr int NV = EPT / V;
    const size_t smem = (size_t)kAhead<V, T, NV> * kRowBytes<V, T, NV>;
    if (smem > 40 * 1024) {   // with the static part, beyond what needs no opt-in
        const cudaError_t e = cudaFuncSetAttribute(grad_kernel<E, V, T, NV, SHIFT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   (int)smem);
        if (e != cudaSuccess) return cuda_failed("row gradient kernel set-up", (int)e);
    }
    return launch_row_kernel("row gradient kernel", grad_kernel<E, V, T, NV, SHIFT>, (unsigned)parts, kThreads<T>, smem, st, p);
}

template <typename E, int V, bool SHIFT>
int pick_grad(const GradParams& p, int parts, cudaStream_t st) {
    const int n = p.cols + (SHIFT ? V - 1 : 0);
    if (n <= 256) return start_grad<E, V, 32, 8, SHIFT>(p, parts, st);
    if (n <= 512) return start_grad<E, V, 32, 16, SHIFT>(p, parts, st);
    if (n <= 1024) return start_grad<E, V, 64, 16, SHIFT>(p, parts, st);
    if (n <= 2048) return start_grad<E, V, 128, 16, SHIFT>(p, parts, st);
    if (n <= 4096) return start_grad<E, V, 256, 16, SHIFT>(p, parts, st);
    if (n <= 8192) return start_grad<E, V, 512, 16, SHIFT>(p, parts, st);
    if (SHIFT || n <= 16384) return start_grad<E, V, 1024, 16, SHIFT>(p, parts, st);
    if constexpr (!SHIFT) return start_grad<E, V, 1024, 32, SHIFT>(p, parts, st);
    return TR_ERR_NOT_SUPPORTED;   // not reached
}

template <typename E>
int type_grad(const GradParams& p, int parts, cudaStream_t st) {
    constexpr int es = sizeof(E), V = 16 / es;
    Phase phase;
    phase.add(p.dy, p.dy_stride, es, V, p.rows);
    phase.add(p.h, p.h_stride, es, V, p.rows);
    phase.add(p.dresidual, p.dresidual_stride, es, V, p.rows);
    phase.add(p.dx, p.dx_stride, es, V, p.rows);
    if (phase.f == 0 && (uintptr_t)p.weight % 16 == 0) return pick_grad<E, V, false>(p, parts, st);
    if (phase.f >= 0 && p.cols <= kShiftCols) return pick_grad<E, V, true>(p, parts, st);
    return pick_grad<E, 1, false>(p, parts, st);
}

// A warp takes kSpan values of a row, V to a lane at a time, the loads first.
constexpr int kSpan = 1024;
template <typename E, int V>
__global__ void __launch_bounds__(256) dequant_kernel(const int8_t* q, const float* scale, E* out, unsigned spans,
                                                      long long q_stride, long long out_stride, int cols,
                                                      unsigned spans_a_row) {
    constexpr int NV = V == 1 ? 4 : kSpan / (32 * V), LOOPS = kSpan / (32 * V * NV);
    wait_for_previous();
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

// Rows of equal distance in q and out as one line, in packs of V values whose
// places are on boundaries of the access whatever the rows' length; a pack may
// hold the end of one row and the start of the next.  Four packs to a thread.
template <typename E, int V, typename Index>
__global__ void __launch_bounds__(256) dequant_line_kernel(const int8_t* q, const float* scale, E* out, Index packs,
                                                           Index length, Index stride, int cols) {
    wait_for_previous();
    Pack<int8_t, V> in[4];
    Index at[4], row[4];
    int c[4];
    bool one[4], two_rows[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const Index i = ((Index)blockIdx.x * 4 + u) * 256 + threadIdx.x;
        at[u] = i * V;
        row[u] = i < packs ? at[u] / stride : 0;
        c[u] = (int)(at[u] - row[u] * stride < (Index)cols ? at[u] - row[u] * stride : cols);   // past the row: none
        one[u] = i < packs && c[u] + V <= cols;
        // the rest of a row and the start of the next, without a gap
        two_rows[u] = i < packs && !one[u] && stride == (Index)cols && cols >= V && at[u] + V <= length;
        if (one[u] || two_rows[u]) in[u].word = *reinterpret_cast<const typename Word<V>::T*>(q + at[u]);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        if (one[u] || two_rows[u]) {
            const float s0 = scale[row[u]], s1 = two_rows[u] ? scale[row[u] + 1] : s0;
            Pack<E, V> o;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const uint32_t b = (uint32_t)(uint8_t)in[u].e[j] ^ 0x80u;
                o.e[j] = from_f<E>((__uint_as_float(0x4B000000u | b) - 8388736.0f) * (c[u] + j < cols ? s0 : s1));
            }
            *reinterpret_cast<typename Word<sizeof(E) * V>::T*>(out + at[u]) = o.word;
        } else if (at[u] < length) {
            for (int j = 0; j < V && at[u] + j < length; ++j) {
                const Index f = at[u] + j, r = f / stride;
                if (f - r * stride < (Index)cols) out[f] = from_f<E>((float)q[f] * scale[r]);
            }
        }
    }
}

template <typename E, typename Index>
int start_line(const DequantArgs& a, cudaStream_t st) {
    constexpr int V = 16 / sizeof(E);
    const Index length = (Index)(a.rows - 1) * (Index)a.q_stride + (Index)a.cols, packs = (length + V - 1) / V;
    const Index ctas = (packs + 1023) / 1024;
    if (ctas > 0x7fffffffu) return TR_ERR_NOT_SUPPORTED;
    return launch_row_kernel("dequantisation kernel", dequant_line_kernel<E, V, Index>, (unsigned)ctas, 256, 0, st, a.q, a.scale,
                             static_cast<E*>(a.out), packs, length, (Index)a.q_stride, a.cols);
}

template <typename E>
int type_dequant(const DequantArgs& a, cudaStream_t st) {
    constexpr int V = 16 / sizeof(E);
    // Short rows, and rows without gaps off the boundaries, as one line (41241 x 69 binary16: 19.6 us by
    // spans, 3.6 as a line; 20000 x 1001: 19.1 and 12.8; with gaps, 37248 x 176 in rows of 192, 7.0 and 11.2;
    // aligned rows without, 50176 x 768, 18.8 and 22.3).
    const bool starts = (uintptr_t)a.q % V == 0 && (uintptr_t)a.out % 16 == 0, line = a.q_stride == a.out_stride && starts;
    const bool dense = a.q_stride == a.cols;
    if (line && ((dense && (a.cols < 512 || a.cols % V != 0)) || (a.cols < 128 && a.q_stride <= 2 * (long long)a.cols))) {
        const double length = (double)a.rows * (double)a.q_stride;
        if (length < 4.0e9) return start_line<E, unsigned>(a, st);
        if (length < 1.0e12) return start_line<E, unsigned long long>(a, st);
    }
    const bool wide = on_pack(a.q, a.q_stride, 1, V, a.rows) && on_pack(a.out, a.out_stride, sizeof(E), V, a.rows);
    const long long spans_a_row = (a.cols + kSpan - 1) / kSpan;
    // rows beyond a grid's reach in further launches
    for (long long r0 = 0; r0 < a.rows;) {
        const long long most = (1LL << 31) / spans_a_row, rows = a.rows - r0 < most ? a.rows - r0 : most;
        const unsigned spans = (unsigned)(rows * spans_a_row), grid = (spans + 7) / 8;
        const int8_t* q = a.q + r0 * a.q_stride;
        E* out = static_cast<E*>(a.out) + r0 * a.out_stride;
        const int rc = launch_row_kernel("dequantisation kernel", wide ? dequant_kernel<E, V> : dequant_kernel<E, 1>, grid, 256, 0,
                                         st, q, a.scale + r0, out, spans, a.q_stride, a.out_stride, a.cols, (unsigned)spans_a_row);
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
    if (a.dtype == TR_ELEM_F32) return type_rows<float>(p, a.what, st);
    if (a.dtype == TR_ELEM_F16) return type_rows<__half>(p, a.what, st);
    return type_rows<__nv_bfloat16>(p, a.what, st);
}

int row_grad_parts(long long rows, long long cols) {
    // The CTAs that 152 SMs hold at once, a row for each of their row groups at least; a multiple of 8, so that
    // the rows of one are all at the same place in a pack.  By the length alone, so that the workspace is known
    // before the matrices are.  The last lengths up to 512 (506 and more in 16 bits, 510 in binary32) are an
    // exception: off the boundaries their packs spread over more than 512 places, a CTA has 64 threads and one
    // row, and a third of the CTAs that fit are launched (50176 x 511 binary16 201 us, x 504 45 us).
    const long long per = cols <= 512 ? 8 : 1;
    const long long want = 152 * (cols <= 512 ? 2 : cols <= 1024 ? 6 : cols <= 2048 ? 4 : cols <= 4096 ? 2 : 1);
    const long long most = ((rows + per - 1) / per + 7) / 8 * 8;
    return (int)(most < want ? (most < 1 ? 8 : most) : want);
}

int launch_row_grad(const RowGradArgs& a) {
    GradParams p{a.dy, a.h, a.weight, a.dresidual, a.dx, a.dweight != nullptr ? a.partial : nullptr, a.rows,
                 a.dy_stride, a.h_stride, a.dresidual_stride, a.dx_stride, a.cols, a.eps};
    cudaStream_t st = static_cast<cudaStream_t>(a.stream);
    const int parts = row_grad_parts(a.rows, a.cols);
    const int rc = a.dtype == TR_ELEM_F32   ? type_grad<float>(p, parts, st)
                   : a.dtype == TR_ELEM_F16 ? type_grad<__half>(p, parts, st)
                                            : type_grad<__nv_bfloat16>(p, parts, st);
    if (rc != TR_OK || a.dweight == nullptr) return rc;
    return launch_row_kernel("weight gradient sum kernel", grad_sum_kernel, (unsigned)((a.cols + kSumCols - 1) / kSumCols),
                             kSumCols * kSumRows, 0, st, a.partial, a.dweight, nullptr, parts, a.cols, a.cols);
}

int launch_dequant(const DequantArgs& a) {
    cudaStream_t st = static_cast<cudaStream_t>(a.stream);
    if (a.dtype == TR_ELEM_F32) return type_dequant<float>(a, st);
    if (a.dtype == TR_ELEM_F16) return type_dequant<__half>(a, st);
    return type_dequant<__nv_bfloat16>(a, st);
}

}  // namespace trfn
