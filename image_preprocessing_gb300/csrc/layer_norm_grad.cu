// Gradients of the layer norm (layer_norm.cu has the forward pass).
//
// Mathematics, for a row h of n values with mean m and s = 1/sqrt(sum_c (h_c - m)^2 / n + eps),
// u_c = h_c - m and g_c = dy_c w_c:
//     dx_c = s (g_c - sum_j g_j / n - u_c s^2 (sum_j g_j u_j) / n) + dres_c
//     dw_c = sum_rows dy_c u_c s,  db_c = sum_rows dy_c
//
// Bound by HBM and, beside it, by the instructions (56 % of the issue slots with
// 17 % of the warps) and the two reductions that a row needs one after the other.
// Measured (of the copy rate): 50176 x 1024 binary16 79 us (0.77), 12544 x 4096
// bfloat16 96 us (0.63), 50176 x 768 82 us (0.56), 50176 x 511 104 us (0.22: shifted packs, CTAs of one row).  Above 8192
// columns 1024 threads leave 64 registers to a thread and sums spill.
#include "row_parts.h"

namespace trfn {
namespace {

struct LayerGradParams {
    const void* dy;
    const void* h;
    const float* weight;
    const void* dresidual;
    void* dx;
    float* partial;   // gridDim.x rows of 2 cols (weight, bias), or null
    long long rows, dy_stride, h_stride, dresidual_stride, dx_stride;
    int cols;
    float eps;
};

// Rows that a CTA takes at a time, and the packs of the next rows that its
// threads copy into shared memory meanwhile, as in the RMS norm's gradient.
template <int V, int T, int NV> constexpr int kLayerRowBytes = V > 1 ? 3 * NV * 16 * kThreads<T> : 0;
template <int V, int T, int NV>
constexpr int kLayerAhead = V == 1 ? 0 : (V == 8 ? 3 : 2) * kLayerRowBytes<V, T, NV> <= 190 * 1024
                                             ? (V == 8 ? 3 : 2)
                                             : 190 * 1024 / kLayerRowBytes<V, T, NV>;

// Weights lie in shared memory, each thread's own beside its packs: in registers they cost the residency of a CTA
// (50176 x 1024: 161 registers against 128).  Rows of 1024 threads have no room for them there.
template <int T> constexpr bool kSharedWeights = T <= 512;

// CTAs that an SM is to hold, one wave of which is launched (24 values a thread take the registers of two).
template <int T> constexpr int kGradResident = T == 32 ? 2 : T == 64 ? 6 : T == 128 ? 4 : T == 256 ? 2 : 1;

// T threads take a row, T = 32 eight rows to a CTA at a time, which goes
// through the matrix with the grid's stride.  A thread's columns are the same
// in every row (with SHIFT too: the grid and the rows of a CTA are multiples of
// 8), so it keeps their sums of dweight and dbias in registers, and the CTA writes the sums as one partial row.  Two reductions:
// of (h, g), then of ((h - m)^2, g (h - m)).
template <typename E, int V, int T, int NV, bool SHIFT>
__global__ void __launch_bounds__(kThreads<T>, T == 32 && V * NV > 16 ? 1 : kGradResident<T>) layer_grad_kernel(const LayerGradParams p) {
    constexpr int R = kThreads<T> / T, N = NV * V;   // N values to a thread
    static_assert(N % 2 == 0 && N <= 32, "values are taken in pairs, and have a bit each");
    constexpr int AHEAD = kLayerAhead<V, T, NV>;
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
    uint32_t mask = 0;   // this thread's values that are in the row
#pragma unroll
    for (int e = 0; e < N; ++e) mask |= (uint32_t)in_row(e) << e;
    const bool whole = mask == (N == 32 ? 0xffffffffu : (1u << (N & 31)) - 1);
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
    __shared__ float2 between[2][2][kRowWarps<T>];   // of the two reductions, for even and odd rows
    int turn = 0;
    constexpr bool SHARED = kSharedWeights<T>;
    Two dw[N / 2], db[N / 2], own[SHARED ? 1 : N / 2];
    Two* const shared = reinterpret_cast<Two*>(dynamic + AHEAD * kLayerRowBytes<V, T, NV>) + threadIdx.x;   // kThreads<T> apart
#pragma unroll
    for (int e = 0; e < N; e += 2) {
        dw[e / 2] = db[e / 2] = two(0.0f, 0.0f);
        const Two v = two(p.weight != nullptr && in_row(e) ? p.weight[column(e)] : 1.0f,
                          p.weight != nullptr && in_row(e + 1) ? p.weight[column(e + 1)] : 1.0f);
        if (SHARED) shared[e / 2 * kThreads<T>] = v;
        else own[SHARED ? 0 : e / 2] = v;
    }
    auto w = [&](int e) { return SHARED ? shared[e / 2 * kThreads<T>] : own[SHARED ? 0 : e / 2]; };
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
        Two u[N / 2], y[N / 2];
        Two h2 = two(0.0f, 0.0f), g2 = two(0.0f, 0.0f);
#pragma unroll
        for (int e = 0; e < N; e += 2) {
            u[e / 2] = pair(ph, e);
            y[e / 2] = pair(py, e);
            h2 = add_two(u[e / 2], h2);
            g2 = fma_two(y[e / 2], w(e), g2);
        }
        fetch(slot);   // the packs are in registers
        if (++slot >= AHEAD) slot = 0;
        const float2 first = row_sums<T>(apart(h2).x + apart(h2).y, apart(g2).x + apart(g2).y, between[turn][0]);
        const float mean = first.x / (float)n, gs = first.y;
        const Two less = two(-mean, -mean);
        Two uu2 = two(0.0f, 0.0f), gu2 = two(0.0f, 0.0f);
#pragma unroll
        for (int e = 0; e < N; e += 2) {
            u[e / 2] = add_two(u[e / 2], less);
            if (!whole) {
                const float2 v = apart(u[e / 2]);
                u[e / 2] = two(mask >> e & 1 ? v.x : 0.0f, mask >> (e + 1) & 1 ? v.y : 0.0f);
            }
            uu2 = fma_two(u[e / 2], u[e / 2], uu2);
            gu2 = fma_two(mul_two(y[e / 2], w(e)), u[e / 2], gu2);
        }
        const float2 next = row_sums<T>(apart(uu2).x + apart(uu2).y, apart(gu2).x + apart(gu2).y, between[turn][1]);
        const float uu = next.x, gu = next.y;
        turn ^= 1;
        // dx = s g - (s^3 gu / n) u + (dres - s gs / n)
        const float s = rsqrtf(uu / (float)n + p.eps), along = -(gu / (float)n * s * s * s), level = -(gs / (float)n * s);
        const Two s2 = two(s, s), along2 = two(along, along), level2 = two(level, level);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            Pack<E, V> o;
#pragma unroll
            for (int j = 0; j < V; j += 2) {
                // (V = 1: pairs are of two packs; the second pack's half is made with it)
                const int e = V > 1 ? i * V + j : i / 2 * 2;
                const Two r = p.dresidual != nullptr ? add_two(pair(pr, e), level2) : level2;
                const float2 d = apart(fma_two(s2, mul_two(y[e / 2], w(e)), fma_two(along2, u[e / 2], r)));
                if constexpr (V > 1) {
                    o.e[j] = from_f<E>(d.x);
                    o.e[j + 1] = from_f<E>(d.y);
                } else {
                    o.e[0] = from_f<E>(i % 2 ? d.y : d.x);
                }
                if (V > 1 || i % 2 == 0) {
                    dw[e / 2] = fma_two(y[e / 2], mul_two(u[e / 2], s2), dw[e / 2]);
                    db[e / 2] = add_two(y[e / 2], db[e / 2]);
                }
            }
            store_pack<E, V>(dx, i * T * V + c0, n, o);
        }
        dx += step * p.dx_stride;
    }
    if (p.partial == nullptr) return;
    float* part = p.partial + (long long)blockIdx.x * (2 * n);
    auto value = [](const Two (&v)[N / 2], int e) { return e % 2 ? apart(v[e / 2]).y : apart(v[e / 2]).x; };
    if constexpr (R > 1) {
        // the sums of the CTA's row groups, one after the other
        // (place c + c / 32: the threads' values, V columns apart, in different banks)
        constexpr int half = padded(N * T);
        __shared__ float sums[2 * half];
        for (int g = 0; g < R; ++g) {
            if (threadIdx.x / T == g) {
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    if (!in_row(e)) continue;
                    const int c = padded(column(e));
                    sums[c] = g == 0 ? value(dw, e) : sums[c] + value(dw, e);
                    sums[half + c] = g == 0 ? value(db, e) : sums[half + c] + value(db, e);
                }
            }
            __syncthreads();
        }
        for (int c = threadIdx.x; c < n; c += kThreads<T>) {
            part[c] = sums[padded(c)];
            part[n + c] = sums[half + padded(c)];
        }
    } else {
#pragma unroll
        for (int e = 0; e < N; ++e) {
            if (!in_row(e)) continue;
            part[column(e)] = value(dw, e);
            part[n + column(e)] = value(db, e);
        }
    }
}

// CTAs of T threads a row: those that 152 SMs hold at once, a row for each of
// their row groups at least; a multiple of 8, so that the rows of one are all at
// the same place in a pack.
int layer_grad_ctas(long long rows, int T) {
    const long long per = kThreads<32> / 32;
    const long long want = 152 * (T == 32 ? 2 : T == 64 ? 6 : T == 128 ? 4 : T == 256 ? 2 : 1);
    const long long most = ((T == 32 ? (rows + per - 1) / per : rows) + 7) / 8 * 8;
    return (int)(most < want ? (most < 1 ? 8 : most) : want);
}

template <typename E, int V, int T, int EPT, bool SHIFT>
int start_layer_grad(const LayerGradParams& p, int* parts, cudaStream_t st) {
    constexpr int NV = EPT / V;
    *parts = layer_grad_ctas(p.rows, T);
    const size_t smem = (size_t)kLayerAhead<V, T, NV> * kLayerRowBytes<V, T, NV> + (kSharedWeights<T> ? NV * V * kThreads<T> * 4 : 0);
    if (smem > 40 * 1024) {   // with the static part, beyond what needs no opt-in
        const cudaError_t e = cudaFuncSetAttribute(layer_grad_kernel<E, V, T, NV, SHIFT>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return cuda_failed("layer norm gradient kernel set-up", (int)e);
    }
    return launch_row_kernel("layer norm gradient kernel", layer_grad_kernel<E, V, T, NV, SHIFT>, (unsigned)*parts, kThreads<T>,
                             smem, st, p);
}

template <typename E, int V, bool SHIFT>
int pick_layer_grad(const LayerGradParams& p, int* parts, cudaStream_t st) {
    const int n = p.cols + (SHIFT ? V - 1 : 0);
    if (n <= 256) return start_layer_grad<E, V, 32, 8, SHIFT>(p, parts, st);
    if (n <= 512) return start_layer_grad<E, V, 32, 16, SHIFT>(p, parts, st);
    if (n <= 768) return start_layer_grad<E, V, 32, 24, SHIFT>(p, parts, st);
    if (n <= 1024) return start_layer_grad<E, V, 64, 16, SHIFT>(p, parts, st);
    if (n <= 2048) return start_layer_grad<E, V, 128, 16, SHIFT>(p, parts, st);
    if (n <= 4096) return start_layer_grad<E, V, 256, 16, SHIFT>(p, parts, st);
    if (n <= 8192) return start_layer_grad<E, V, 512, 16, SHIFT>(p, parts, st);
    if (SHIFT || n <= 16384) return start_layer_grad<E, V, 1024, 16, SHIFT>(p, parts, st);
    if constexpr (!SHIFT) return start_layer_grad<E, V, 1024, 32, SHIFT>(p, parts, st);
    return TR_ERR_NOT_SUPPORTED;   // not reached
}

template <typename E>
int type_layer_grad(const LayerGradParams& p, int* parts, cudaStream_t st) {
    constexpr int es = sizeof(E), V = 16 / es;
    Phase phase;
    phase.add(p.dy, p.dy_stride, es, V, p.rows);
    phase.add(p.h, p.h_stride, es, V, p.rows);
    phase.add(p.dresidual, p.dresidual_stride, es, V, p.rows);
    phase.add(p.dx, p.dx_stride, es, V, p.rows);
    if (phase.f == 0) return pick_layer_grad<E, V, false>(p, parts, st);
    if (phase.f >= 0 && p.cols <= kShiftCols) return pick_layer_grad<E, V, true>(p, parts, st);
    return pick_layer_grad<E, 1, false>(p, parts, st);
}

}  // namespace

int layer_norm_grad_parts(long long rows, long long cols) {
    // by the length alone, so that the workspace is known before the matrices are: off the boundaries the last
    // lengths below each change of threads a row (up to 7 packs' values of them) take the next layout
    auto threads = [](long long n) { return n <= 768 ? 32 : n <= 1024 ? 64 : n <= 2048 ? 128 : n <= 4096 ? 256 : 512; };
    const int a = layer_grad_ctas(rows, threads(cols)), b = layer_grad_ctas(rows, threads(cols + 7));
    return a > b ? a : b;
}

int launch_layer_norm_grad(const RowGradArgs& a) {
    const bool sums = a.dweight != nullptr || a.dbias != nullptr;
    LayerGradParams p{a.dy, a.h, a.weight, a.dresidual, a.dx, sums ? a.partial : nullptr, a.rows,
                      a.dy_stride, a.h_stride, a.dresidual_stride, a.dx_stride, a.cols, a.eps};
    cudaStream_t st = static_cast<cudaStream_t>(a.stream);
    int parts = 0;
    const int rc = a.dtype == TR_ELEM_F32   ? type_layer_grad<float>(p, &parts, st)
                   : a.dtype == TR_ELEM_F16 ? type_layer_grad<__half>(p, &parts, st)
                                            : type_layer_grad<__nv_bfloat16>(p, &parts, st);
    if (rc != TR_OK || !sums) return rc;
    return launch_row_kernel("weight gradient sum kernel", grad_sum_kernel, (unsigned)((2 * a.cols + kSumCols - 1) / kSumCols),
                             kSumCols * kSumRows, 0, st, a.partial, a.dweight, a.dbias, parts, a.cols, 2 * a.cols);
}

}  // namespace trfn
