// y[m][n] = (sum_k x[m][k] w[n][k]) sx[m] sw[n] + bias[n] over int8 x and w.
//
// A CTA makes 64 tokens x 64 channels from 64-byte slices of both matrices in
// shared memory; a thread makes 4 x 4 of them with four-way integer dot
// products, so the sums are exact.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "token_ops.h"

namespace trfn {
namespace {

template <typename T> __device__ __forceinline__ T from_f(float v);
template <> __device__ __forceinline__ float from_f<float>(float v) { return v; }
template <> __device__ __forceinline__ __half from_f<__half>(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

template <typename E>
__global__ void __launch_bounds__(256) dot_kernel(const MatmulArgs a) {
    __shared__ __align__(16) int8_t xs[64][68], ws[64][68];
    const long long m0 = (long long)blockIdx.y * 64, n0 = (long long)blockIdx.x * 64;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    int acc[4][4] = {};
    for (int k0 = 0; k0 < a.K; k0 += 64) {
        for (int i = threadIdx.x; i < 64 * 64; i += 256) {
            const int r = i >> 6, k = i & 63;
            const bool in = k0 + k < a.K;
            xs[r][k] = in && m0 + r < a.M ? a.x[(m0 + r) * a.x_stride + k0 + k] : (int8_t)0;
            ws[r][k] = in && n0 + r < a.N ? a.w[(n0 + r) * a.w_stride + k0 + k] : (int8_t)0;
        }
        __syncthreads();
#pragma unroll 4
        for (int k = 0; k < 64; k += 4) {
            int xv[4], wv[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                xv[i] = *reinterpret_cast<const int*>(&xs[ty + 16 * i][k]);
                wv[i] = *reinterpret_cast<const int*>(&ws[tx + 16 * i][k]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = __dp4a(xv[i], wv[j], acc[i][j]);
        }
        __syncthreads();
    }
    E* y = static_cast<E*>(a.y);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const long long m = m0 + ty + 16 * i;
        if (m >= a.M) continue;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const long long n = n0 + tx + 16 * j;
            if (n >= a.N) continue;
            float v = (float)acc[i][j] * a.x_scale[m] * a.w_scale[n];
            if (a.bias != nullptr) v += a.bias[n];
            y[m * a.y_stride + n] = from_f<E>(v);
        }
    }
}

}  // namespace

size_t int8_matmul_workspace(long long, long long, long long) { return 0; }

int launch_int8_matmul(const MatmulArgs& a) {
    cudaStream_t st = static_cast<cudaStream_t>(a.stream);
    const unsigned gx = (unsigned)(((long long)a.N + 63) / 64), gy = (unsigned)(((long long)a.M + 63) / 64);
    if (gy > 65535) return TR_ERR_NOT_SUPPORTED;
    const dim3 grid(gx, gy);
    if (a.out_dtype == TR_ELEM_F32) dot_kernel<float><<<grid, 256, 0, st>>>(a);
    else if (a.out_dtype == TR_ELEM_F16) dot_kernel<__half><<<grid, 256, 0, st>>>(a);
    else dot_kernel<__nv_bfloat16><<<grid, 256, 0, st>>>(a);
    return launched("int8 product kernel");
}

}  // namespace trfn
