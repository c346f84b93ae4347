// y[m][n] = (sum_k x[m][k] w[n][k]) sx[m] sw[n] + bias[n] over int8 x and w:
// the kernel for one or two tokens, and the choice between the product's kernels.
//
// Arithmetic of the others (int8_mid.cu, int8_gemm.cu).  sm_103a has no int8
// kind of tcgen05.mma, and its int8 mma.sync runs at a fraction of the
// binary16 rate; int8 values are exact in binary16, their products exact in
// the tensor cores, and sums of at most 1024 of them (2^14 * 2^10 = 2^24)
// exact in binary32.  So they multiply in binary16, sum 1024 products in
// binary32, and add those sums as integers.
#include "int8_parts.h"
#include "token_ops.h"

namespace trfn {
namespace {

// One or two tokens: bound by reading w once.  A warp takes kRows channels and
// one of KP parts of K: its lanes read 512 bytes of each channel's row at a
// time, kDepth such steps ahead, and sum four products an instruction
// (__dp4a); the lanes' sums are added by one redux each, the parts' in shared
// memory.  Integer sums have no order.  __dp4a runs at about 16 lanes a cycle
// and SM here, so that two tokens take as long as w's bytes and three go to the
// tensor cores.  Measured: 1 x 4096 x 4096 5.2 us, 1 x 16384 x 4096 14.3 us (4.7
// TB/s): 1024 CTAs in somewhat over two waves, each of which starts with nothing
// under way.
constexpr int kWarps = 8, kRows = 4, kDepth = 2, kStep = 512;

struct FewParams {
    ByteRows x, w;
    const float* x_scale;
    const float* w_scale;
    const float* bias;
    void* y;
    long long y_stride;
};

template <typename E, int M, int KP, bool ON16>
__global__ void __launch_bounds__(kWarps * 32) few_kernel(const FewParams p) {
    constexpr int NT = kWarps / KP * kRows;   // channels of a CTA
    __shared__ int sums[KP][M][NT];
    asm volatile("griddepcontrol.wait;" ::: "memory");   // for the kernel before this one in the stream
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int part = warp % KP, group = warp / KP;
    const int n0 = blockIdx.x * NT;
    // rows past the end repeat the last: their sums are not written
    const int8_t* wr[kRows];
    const int8_t* xr[M];
#pragma unroll
    for (int r = 0; r < kRows; ++r) wr[r] = p.w.p + min(n0 + group * kRows + r, p.w.rows - 1) * p.w.stride;
#pragma unroll
    for (int m = 0; m < M; ++m) xr[m] = p.x.p + min(m, p.x.rows - 1) * p.x.stride;
    const int steps = (p.x.K + kStep - 1) / kStep;
    Piece<ON16> wv[kDepth][kRows];
    auto fetch = [&](int step, Piece<ON16> (&v)[kRows]) {
#pragma unroll
        for (int r = 0; r < kRows; ++r) v[r].fetch(p.w, wr[r], step * kStep + lane * 16);
    };
#pragma unroll
    for (int d = 0; d < kDepth; ++d) fetch(part + d * KP, wv[d]);
    int acc[kRows][M];
#pragma unroll
    for (int r = 0; r < kRows; ++r)
#pragma unroll
        for (int m = 0; m < M; ++m) acc[r][m] = 0;
    for (int s0 = part; s0 < steps; s0 += kDepth * KP) {
#pragma unroll
        for (int d = 0; d < kDepth; ++d) {
            const int step = s0 + d * KP, k = step * kStep + lane * 16;
            if (step < steps) {
                Piece<ON16> xv[M];
#pragma unroll
                for (int m = 0; m < M; ++m) xv[m].fetch(p.x, xr[m], k);
                uint4 w[kRows];
#pragma unroll
                for (int r = 0; r < kRows; ++r) w[r] = wv[d][r].value(p.w, wr[r], k, false);
#pragma unroll
                for (int m = 0; m < M; ++m) {
                    const uint4 x = xv[m].value(p.x, xr[m], k, false);
#pragma unroll
                    for (int r = 0; r < kRows; ++r) {
                        acc[r][m] = __dp4a((int)w[r].x, (int)x.x, acc[r][m]);
                        acc[r][m] = __dp4a((int)w[r].y, (int)x.y, acc[r][m]);
                        acc[r][m] = __dp4a((int)w[r].z, (int)x.z, acc[r][m]);
                        acc[r][m] = __dp4a((int)w[r].w, (int)x.w, acc[r][m]);
                    }
                }
                fetch(step + kDepth * KP, wv[d]);
            }
        }
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r)
#pragma unroll
        for (int m = 0; m < M; ++m) {
            const int sum = __reduce_add_sync(0xffffffffu, acc[r][m]);
            if (lane == 0) sums[part][m][group * kRows + r] = sum;
        }
    __syncthreads();
    if (threadIdx.x < M * NT) {
        const int m = threadIdx.x / NT, c = threadIdx.x % NT, n = n0 + c;
        if (m < p.x.rows && n < p.w.rows) {
            int sum = 0;
#pragma unroll
            for (int i = 0; i < KP; ++i) sum += sums[i][m][c];
            float v = (float)sum * p.x_scale[m] * p.w_scale[n];
            if (p.bias != nullptr) v += p.bias[n];
            static_cast<E*>(p.y)[m * p.y_stride + n] = out_value<E>(v);
        }
    }
}

template <typename E, int M, int KP>
int start_few(const FewParams& p, bool on16, cudaStream_t st) {
    constexpr int NT = kWarps / KP * kRows;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)((p.w.rows + NT - 1) / NT));
    cfg.blockDim = dim3(kWarps * 32);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];   // its CTAs may be set up while the kernel before ends
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return launched("int8 product kernel (few tokens)",
                    (int)cudaLaunchKernelEx(&cfg, on16 ? few_kernel<E, M, KP, true> : few_kernel<E, M, KP, false>, p));
}

template <typename E, int M>
int part_few(const FewParams& p, bool on16, cudaStream_t st) {
    // K in 2 parts, 16 channels a CTA, where that gives each SM a CTA; else in 8, 4 channels a CTA.  In 2 and in 8
    // parts: 1 x 1216 x 4096 2.7 and 1.8 us, 1 x 2432 x 4096 4.5 and 4.7, 1 x 4096 x 4096 5.2 and 6.4, 1 x 16384 x
    // 4096 14.3 and 17.4.  (A longer K moves the place where they meet, 1 x 4096 x 16384 14.6 and 14.1, a shorter
    // one back, 1 x 1216 x 1024 1.6 and 1.7.)
    if (p.w.rows >= 152 * kWarps * kRows / 2) return start_few<E, M, 2>(p, on16, st);
    return start_few<E, M, 8>(p, on16, st);
}

template <typename E>
int pick_few(const FewParams& p, bool on16, cudaStream_t st) {
    return p.x.rows == 1 ? part_few<E, 1>(p, on16, st) : part_few<E, 2>(p, on16, st);
}

int launch_few(const MatmulArgs& a) {
    FewParams p;
    p.x = ByteRows{a.x, a.x_stride, a.x + (a.M - 1) * a.x_stride + a.K, a.M, a.K};
    p.w = ByteRows{a.w, a.w_stride, a.w + (a.N - 1) * a.w_stride + a.K, a.N, a.K};
    p.x_scale = a.x_scale;
    p.w_scale = a.w_scale;
    p.bias = a.bias;
    p.y = a.y;
    p.y_stride = a.y_stride;
    const bool on16 = rows_on16(a.x, a.x_stride, a.M) && rows_on16(a.w, a.w_stride, a.N);
    cudaStream_t st = static_cast<cudaStream_t>(a.stream);
    if (a.out_dtype == TR_ELEM_F32) return pick_few<float>(p, on16, st);
    if (a.out_dtype == TR_ELEM_F16) return pick_few<__half>(p, on16, st);
    return pick_few<__nv_bfloat16>(p, on16, st);
}

// By shape alone, so that the workspace is known before the matrices are.  A sum of nothing (K = 0) goes to the
// kernel that takes no copies, whatever the size: there would be no blocks to copy.
bool mid_takes(long long M, long long N, long long K) {
    return K == 0 || int8_mid_cycles(M, N, K) <= int8_gemm_cycles(M, N, K);
}

}  // namespace

size_t int8_matmul_workspace(long long M, long long N, long long K) {
    return M <= 2 || mid_takes(M, N, K) ? 0 : int8_gemm_workspace(M, N, K);
}

// Both estimates grow with M.  So where the kernel without copies is estimated at M no longer than the other at
// the fewest tokens, it takes every M up to this one; else the copies of M tokens have room for those of fewer.
// (Of 3000 random shapes 33 get a size here that no M up to theirs needs.)
size_t int8_matmul_workspace_up_to(long long M, long long N, long long K) {
    return M <= 2 || K == 0 || int8_mid_cycles(M, N, K) <= int8_gemm_cycles(3, N, K) ? 0 : int8_gemm_workspace(M, N, K);
}

int launch_int8_matmul(const MatmulArgs& a) {
    if (a.M <= 2) return launch_few(a);
    return mid_takes(a.M, a.N, a.K) ? launch_int8_mid(a) : launch_int8_gemm(a);
}

}  // namespace trfn
