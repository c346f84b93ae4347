// Device parts shared by the int8 product's kernels: reading 16 bytes of a row
// at any alignment, and int8 as binary16.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace trfn {

// A row-major int8 matrix and the byte range that may be read of it.
struct ByteRows {
    const int8_t* p;
    long long stride;
    const int8_t* end;   // one past the last row's last byte
    int rows, K;
};

// Bytes k .. k+15 of row r, zeros at and past K.  Rows on 16-byte boundaries
// (ON16) take one load; others two aligned loads and a byte shift, where both
// lie inside the matrix, else single bytes.
template <bool ON16>
__device__ __forceinline__ uint4 load16(const ByteRows& m, long long r, int k) {
    const int8_t* a = m.p + r * m.stride + k;
    const int left = m.K - k;
    if (ON16 && left >= 16) return *reinterpret_cast<const uint4*>(a);
    if (left <= 0) return make_uint4(0, 0, 0, 0);
    uint4 v;
    const int s = (int)((uintptr_t)a & 15);
    const int8_t* lo = a - s;
    if (!ON16 && lo >= m.p && lo + 32 <= m.end) {
        const uint4 b = *reinterpret_cast<const uint4*>(lo), c = *reinterpret_cast<const uint4*>(lo + 16);
        // shift the 32 bytes down by s: by words, then by bytes
        uint32_t w[8] = {b.x, b.y, b.z, b.w, c.x, c.y, c.z, c.w};
#pragma unroll
        for (int i = 0; i < 6; ++i) w[i] = (s & 8) ? w[i + 2] : w[i];
#pragma unroll
        for (int i = 0; i < 5; ++i) w[i] = (s & 4) ? w[i + 1] : w[i];
        const uint32_t sel = 0x3210u + 0x1111u * (uint32_t)(s & 3);
        v = make_uint4(__byte_perm(w[0], w[1], sel), __byte_perm(w[1], w[2], sel), __byte_perm(w[2], w[3], sel),
                       __byte_perm(w[3], w[4], sel));
    } else {
        uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (i < left) w[i >> 2] |= (uint32_t)(uint8_t)a[i] << (8 * (i & 3));
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    if (left < 16) {   // clear the bytes at and past K
        uint32_t* w = &v.x;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int n = left - 4 * i;
            w[i] = n >= 4 ? w[i] : n <= 0 ? 0u : w[i] & ((1u << (8 * n)) - 1u);
        }
    }
    return v;
}

// Four int8 as four binary16: with u = x + 128 (the sign bit flipped), the
// bytes {u, 0x64} are 1024 + u, and 1024 + u - 1152 = x exactly.
__device__ __forceinline__ void int8_to_half(uint32_t v, uint32_t& lo, uint32_t& hi) {
    const uint32_t u = v ^ 0x80808080u;
    const __half2 base = __half2half2(__ushort_as_half(0x6480));   // 1152
    uint32_t a = __byte_perm(u, 0x64646464u, 0x4140u), b = __byte_perm(u, 0x64646464u, 0x4342u);
    const __half2 x = __hsub2(*reinterpret_cast<__half2*>(&a), base), y = __hsub2(*reinterpret_cast<__half2*>(&b), base);
    lo = *reinterpret_cast<const uint32_t*>(&x);
    hi = *reinterpret_cast<const uint32_t*>(&y);
}

template <typename T> __device__ __forceinline__ T out_value(float v);
template <> __device__ __forceinline__ float out_value<float>(float v) { return v; }
template <> __device__ __forceinline__ __half out_value<__half>(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 out_value<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

}  // namespace trfn
