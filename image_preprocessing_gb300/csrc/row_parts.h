// Device parts shared by the kernels that take rows of values (norms,
// quantisation, their gradients): packs of 16 bytes at any phase, reductions
// over a row's threads, launches, and the sum of partial weight gradients.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "f32_pairs.h"
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

// Values c .. c+V-1 of a row of n, zeros outside 0 .. n-1.  V > 1 only where
// the row's value c lies on a boundary of the access.  `over`: the bytes next to
// the row, up to the boundary, belong to the matrix too and may be read (they
// are not used, so it does not matter whether another CTA writes them meanwhile).
template <typename E, int V>
__device__ __forceinline__ Pack<E, V> load_pack(const E* row, int c, int n, bool over) {
    Pack<E, V> p;
    const bool whole = c >= 0 && c + V <= n;
    if (whole || (over && c < n)) {
        p.word = *reinterpret_cast<const typename Word<sizeof(E) * V>::T*>(row + c);
        if (!whole)
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (c + j < 0 || c + j >= n) p.e[j] = from_f<E>(0.0f);
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) p.e[j] = (c + j >= 0 && c + j < n) ? row[c + j] : from_f<E>(0.0f);
    }
    return p;
}
// Whether packs of row `row` may be read over its ends: another row lies beyond (a stride below a pack, as of
// one row that is repeated, says no).
__device__ __forceinline__ bool may_over(long long row, long long rows, long long stride, int V) {
    return row + 1 < rows && stride >= V;
}

template <typename E, int V>
__device__ __forceinline__ void store_pack(E* row, int c, int n, const Pack<E, V>& p) {
    if (c >= 0 && c + V <= n) {
        *reinterpret_cast<typename Word<sizeof(E) * V>::T*>(row + c) = p.word;
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (c + j >= 0 && c + j < n) row[c + j] = p.e[j];
    }
}

// Weights of shifted packs lie in shared memory as V rows: value c at row c mod V, place c / V + 1, zeros
// around them.  The j-th values of the lanes' packs are then neighbours in one row, without bounds to look at.
constexpr int kShiftCols = 8192;   // rows with shifted packs are this long at most
template <int V> __host__ __device__ constexpr int shift_pitch(int cols) { return cols / V + 3; }

template <int V>
__device__ __forceinline__ void share_weight(const float* w, float* shared, int n, float none = 1.0f) {
    const int pitch = shift_pitch<V>(n);
    for (int k = threadIdx.x; k < pitch; k += blockDim.x)
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = (k - 1) * V + v;
            shared[v * pitch + k] = c >= 0 && c < n ? (w != nullptr ? w[c] : none) : 0.0f;
        }
}

// Weights of the pack that starts at column c = pack * V - s, s < V.  (Packs past the row's end read the last
// place: their values are not used.)
// SHARED: from shared memory; else, for rows that have a CTA each, one value at a time.
template <int V, bool SHIFT, bool SHARED>
__device__ __forceinline__ void load_weight(const float* w, const float* shared, int c, int pack, int s, int n, float (&v)[V],
                                            float none = 1.0f) {
    if constexpr (SHIFT && SHARED) {
        const int place = min(pack, shift_pitch<V>(n) - 2);
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] = shared[((j - s) & (V - 1)) * shift_pitch<V>(n) + (j < s ? 0 : 1) + place];
        return;
    }
    if (w == nullptr) {
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] = none;
        return;
    }
    if constexpr (V >= 4 && !SHIFT) {
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
    for (int j = 0; j < V; ++j) v[j] = (c + j >= 0 && c + j < n) ? w[c + j] : 0.0f;
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
    if constexpr (T < 32) {
#pragma unroll
        for (int o = T / 2; o > 0; o >>= 1) {
            a += __shfl_xor_sync(0xffffffffu, a, o);
            const float c = __shfl_xor_sync(0xffffffffu, b, o);
            b = Q ? __uint_as_float(max(__float_as_uint(b), __float_as_uint(c))) : b + c;
        }
        return;
    }
    __shared__ float sa[T < 32 ? 1 : T / 32], sb[T < 32 ? 1 : T / 32];
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

// Sum over the T threads of a row, and likewise the largest bits and two sums, in a fixed order.  Rows of several
// warps pass through `between`, one of its own for each reduction that may follow before all threads have read
// it: one barrier each.
template <int T>
__device__ __forceinline__ float row_sum(float v, float* between) {
#pragma unroll
    for (int o = (T < 32 ? T : 32) / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if constexpr (T > 32) {
        if ((threadIdx.x & 31) == 0) between[threadIdx.x >> 5] = v;
        __syncthreads();
        v = between[0];
#pragma unroll
        for (int i = 1; i < T / 32; ++i) v += between[i];
    }
    return v;
}
template <int T>
__device__ __forceinline__ unsigned row_top(unsigned v, float* between) {
    if constexpr (T < 32) {
#pragma unroll
        for (int o = T / 2; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
    } else {
        v = __reduce_max_sync(0xffffffffu, v);
    }
    if constexpr (T > 32) {
        if ((threadIdx.x & 31) == 0) between[threadIdx.x >> 5] = __uint_as_float(v);
        __syncthreads();
        v = __float_as_uint(between[0]);
#pragma unroll
        for (int i = 1; i < T / 32; ++i) v = max(v, __float_as_uint(between[i]));
    }
    return v;
}
template <int T>
__device__ __forceinline__ float2 row_sums(float a, float b, float2* between) {
#pragma unroll
    for (int o = (T < 32 ? T : 32) / 2; o > 0; o >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, o);
        b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    if constexpr (T > 32) {
        if ((threadIdx.x & 31) == 0) between[threadIdx.x >> 5] = make_float2(a, b);
        __syncthreads();
        float2 v = between[0];
#pragma unroll
        for (int i = 1; i < T / 32; ++i) {
            const float2 w = between[i];
            v.x += w.x;
            v.y += w.y;
        }
        return v;
    }
    return make_float2(a, b);
}
template <int T> constexpr int kRowWarps = T > 32 ? T / 32 : 1;

// v rounded to the nearest integer, ties to even, for |v| <= 2^22: the low bits of v + 1.5 * 2^23 (the
// conversion instruction takes several times as long).
__device__ __forceinline__ uint32_t round_bits(float v) { return __float_as_uint(__fadd_rn(v, 12582912.0f)); }

// Every kernel here is launched so that its CTAs may be set up while the kernel before it in the stream ends,
// and waits for that kernel before it touches memory (50176 x 768 quantised and read back: 41.0 -> 36.2 us).
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <typename... P, typename... A>
int launch_row_kernel(const char* what, void (*kernel)(P...), unsigned grid, unsigned block, size_t smem, cudaStream_t st,
                      A&&... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return launched(what, (int)cudaLaunchKernelEx(&cfg, kernel, P(args)...));
}

// Rows of T = 8 or 32 threads share a CTA of 256; longer rows have a CTA each.
template <int T> constexpr int kThreads = T <= 32 ? 256 : T;

__host__ __device__ constexpr int padded(int c) { return c + (c >> 5); }

// How the rows of a matrix lie on packs of V values of es bytes: 0 all of them
// on boundaries, f > 0 row r starts f r mod V values into a pack, -1 neither.
int phase_of(const void* p, long long stride, int es, int V, long long rows) {
    if ((uintptr_t)p % (unsigned)(es * V) != 0) return -1;
    return rows <= 1 ? 0 : (int)(stride & (V - 1));
}
// The phase that all matrices of a call share, else -1.
struct Phase {
    int f = -2;
    void add(const void* p, long long stride, int es, int V, long long rows) {
        if (p == nullptr) return;
        const int g = phase_of(p, stride, es, V, rows);
        f = f == -2 || f == g ? g : -1;
    }
};
// Whether packs of V values of es bytes can be accessed whole.
bool on_pack(const void* p, long long stride, int es, int V, long long rows) { return phase_of(p, stride, es, V, rows) == 0; }

// dweight = sum of the partial rows: 8 columns (a sector of a row) to a CTA,
// 128 threads each summing every 128th partial in order, then the 128 sums in
// order, 16 at a time.  Columns past the first `cols` go to `second`.
constexpr int kSumCols = 8, kSumRows = 128;
__global__ void __launch_bounds__(kSumCols * kSumRows) grad_sum_kernel(const float* partial, float* first, float* second,
                                                                       int parts, int cols, int all) {
    __shared__ float sm[kSumRows][kSumCols + 1];
    wait_for_previous();   // the partial rows are that kernel's
    const int x = threadIdx.x % kSumCols, y = threadIdx.x / kSumCols, c = blockIdx.x * kSumCols + x;
    float v = 0.0f;
    if (c < all) {
#pragma unroll 8
        for (int r = y; r < parts; r += kSumRows) v += partial[(long long)r * all + c];
    }
    sm[y][x] = v;
    __syncthreads();
    if (y < kSumRows / 16) {
        v = sm[y * 16][x];
#pragma unroll
        for (int i = 1; i < 16; ++i) v += sm[y * 16 + i][x];
    }
    __syncthreads();
    if (y < kSumRows / 16) sm[y][x] = v;
    __syncthreads();
    if (y == 0 && c < all) {
#pragma unroll
        for (int i = 1; i < kSumRows / 16; ++i) v += sm[i][x];
        float* const to = c < cols ? first : second;
        if (to != nullptr) to[c < cols ? c : c - cols] = v;
    }
}

}  // namespace
}  // namespace trfn
