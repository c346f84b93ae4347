// y[m][n] = (sum_k x[m][k] w[n][k]) sx[m] sw[n] + bias[n] over int8 x and w:
// the kernel for few tokens, and the choice between it and int8_gemm.cu's.
//
// Arithmetic.  sm_103a has no int8 kind of tcgen05.mma, and its int8 mma.sync
// runs at a fraction of the binary16 rate; int8 values are exact in binary16,
// their products exact in the tensor cores, and sums of at most 1024 of them
// (2^14 * 2^10 = 2^24) exact in binary32.  So every kernel multiplies in
// binary16, sums 1024 products in binary32, and adds those sums as integers.
#include "int8_parts.h"
#include "token_ops.h"

namespace trfn {
namespace {

// Few tokens: bound by reading w once.  A CTA of 8 warps makes 16 R CG
// channels x 8 J tokens: warp = (channel group of 16 R, part of K).  A warp
// loads 64 bytes of each of its rows at a time, straight into the fragments
// of mma.m16n8k16: a sum over k takes its terms in any order, so lane t of a
// quad takes bytes 16 t .. 16 t + 15 of w's and x's rows alike and calls its
// word j the fragment of the j-th of four products.  Nothing passes through
// shared memory but the sums, which the warps add there as integers.
constexpr int kWarps = 8;

struct DotParams {
    ByteRows x, w;
    const float* x_scale;
    const float* w_scale;
    const float* bias;
    void* y;
    long long y_stride;
};

__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <typename E, int J, int R, int CG, int DEPTH, bool ON16>
__global__ void __launch_bounds__(kWarps * 32) dot_kernel(const DotParams p) {
    constexpr int NT = 16 * R * CG, MT = 8 * J, KS = kWarps / CG, S = NT + 4;   // S = 4 mod 16: no bank conflicts
    __shared__ int sums[MT * S];
    for (int i = threadIdx.x; i < MT * S; i += kWarps * 32) sums[i] = 0;
    __syncthreads();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int cg = warp % CG, ks = warp / CG;
    // tiles of one channel block are neighbours: w is read from HBM once
    const int m_tiles = (p.x.rows + MT - 1) / MT;
    const int n0 = (int)(blockIdx.x / m_tiles) * NT, m0 = (int)(blockIdx.x % m_tiles) * MT;
    const int wrow = n0 + cg * 16 * R + g, xrow = m0 + g;
    const int slices = (p.x.K + 63) >> 6;
    float acc[R][J][4];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[r][j][i] = 0.0f;

    uint4 wv[DEPTH][2 * R], xv[DEPTH][J];
    auto load = [&](int s, uint4 (&w)[2 * R], uint4 (&x)[J]) {
        const int k = s * 64 + t * 16;
        const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < 2 * R; ++i)
            w[i] = (s < slices && wrow + 8 * i < p.w.rows) ? load16<ON16>(p.w, wrow + 8 * i, k) : zero;
#pragma unroll
        for (int j = 0; j < J; ++j)
            x[j] = (s < slices && xrow + 8 * j < p.x.rows) ? load16<ON16>(p.x, xrow + 8 * j, k) : zero;
    };
    auto flush = [&]() {
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int j = 0; j < J; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int token = 8 * j + 2 * t + (i & 1), ch = (cg * R + r) * 16 + g + 8 * (i >> 1);
                    atomicAdd(&sums[token * S + ch], __float2int_rn(acc[r][j][i]));
                    acc[r][j][i] = 0.0f;
                }
    };
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) load(ks + d * KS, wv[d], xv[d]);
    int since = 0;
    for (int s0 = ks; s0 < slices; s0 += DEPTH * KS) {
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) {
            const int s = s0 + d * KS;
            if (s < slices) {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint32_t a[R][4];
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        int8_to_half((&wv[d][2 * r].x)[q], a[r][0], a[r][2]);
                        int8_to_half((&wv[d][2 * r + 1].x)[q], a[r][1], a[r][3]);
                    }
#pragma unroll
                    for (int j = 0; j < J; ++j) {
                        uint32_t b0, b1;
                        int8_to_half((&xv[d][j].x)[q], b0, b1);
#pragma unroll
                        for (int r = 0; r < R; ++r) mma_16816(acc[r][j], a[r][0], a[r][1], a[r][2], a[r][3], b0, b1);
                    }
                }
                load(s + DEPTH * KS, wv[d], xv[d]);
                if (++since == 16) {   // 1024 products: the last exact binary32 sum
                    flush();
                    since = 0;
                }
            }
        }
    }
    if (since > 0) flush();
    __syncthreads();
    E* y = static_cast<E*>(p.y);
    for (int i = threadIdx.x; i < MT * NT; i += kWarps * 32) {
        const int token = i / NT, ch = i % NT;
        const int m = m0 + token, n = n0 + ch;
        if (m < p.x.rows && n < p.w.rows) {
            float v = (float)sums[token * S + ch] * p.x_scale[m] * p.w_scale[n];
            if (p.bias != nullptr) v += p.bias[n];
            y[m * p.y_stride + n] = out_value<E>(v);
        }
    }
}

template <typename E, int J, int R, int CG, int DEPTH>
void start_dot(const DotParams& p, bool on16, cudaStream_t st) {
    const unsigned grid = (unsigned)((p.w.rows + 16 * R * CG - 1) / (16 * R * CG)) * ((p.x.rows + 8 * J - 1) / (8 * J));
    if (on16) dot_kernel<E, J, R, CG, DEPTH, true><<<grid, kWarps * 32, 0, st>>>(p);
    else dot_kernel<E, J, R, CG, DEPTH, false><<<grid, kWarps * 32, 0, st>>>(p);
}

template <typename E>
void pick_dot(const DotParams& p, bool on16, cudaStream_t st) {
    const int M = p.x.rows;
    if (M <= 8) start_dot<E, 1, 1, 1, 4>(p, on16, st);
    else if (M <= 16) start_dot<E, 2, 1, 1, 4>(p, on16, st);
    else if (M <= 32) start_dot<E, 4, 1, 1, 2>(p, on16, st);
    else start_dot<E, 8, 2, 4, 1>(p, on16, st);
}

}  // namespace

bool dot_takes(long long M, long long N, long long K) {
    return M <= 64 || (double)M * (double)N * (double)K <= (double)(1 << 30);
}

int launch_int8_dot(const MatmulArgs& a) {
    DotParams p;
    p.x = ByteRows{a.x, a.x_stride, a.x + (a.M - 1) * a.x_stride + a.K, a.M, a.K};
    p.w = ByteRows{a.w, a.w_stride, a.w + (a.N - 1) * a.w_stride + a.K, a.N, a.K};
    p.x_scale = a.x_scale;
    p.w_scale = a.w_scale;
    p.bias = a.bias;
    p.y = a.y;
    p.y_stride = a.y_stride;
    const bool on16 = (uintptr_t)a.x % 16 == 0 && (uintptr_t)a.w % 16 == 0 && (a.M <= 1 || a.x_stride % 16 == 0) &&
                      (a.N <= 1 || a.w_stride % 16 == 0);
    cudaStream_t st = static_cast<cudaStream_t>(a.stream);
    if (a.out_dtype == TR_ELEM_F32) pick_dot<float>(p, on16, st);
    else if (a.out_dtype == TR_ELEM_F16) pick_dot<__half>(p, on16, st);
    else pick_dot<__nv_bfloat16>(p, on16, st);
    return launched("int8 dot kernel");
}

size_t int8_matmul_workspace(long long M, long long N, long long K) {
    return dot_takes(M, N, K) ? 0 : int8_gemm_workspace(M, N, K);
}

int launch_int8_matmul(const MatmulArgs& a) {
    return dot_takes(a.M, a.N, a.K) ? launch_int8_dot(a) : launch_int8_gemm(a);
}

}  // namespace trfn
