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

// Loads 16 bytes into v where `in` is true and leaves it otherwise: a
// predicated load without a branch, so that a thread's loads leave together.
__device__ __forceinline__ void load_if(uint4& v, const int8_t* p, bool in) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.u32 p, %5, 0;\n\t"
        "@p ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
        : "+r"(v.x), "+r"(v.y), "+r"(v.z), "+r"(v.w)
        : "l"(p), "r"((uint32_t)in));
}

// Bytes k .. k+15 of a row, zeros at and past K, in two steps: fetch issues
// the loads, value waits for them.  Rows on 16-byte boundaries (ON16) take one
// load; others the two aligned pieces that hold the bytes, shifted.  What an
// aligned load may not touch (bytes outside the matrix) or would have to mask
// (bytes past K) is read byte by byte in value: the ends of rows only.
// `inner`: the caller knows that k + 16 <= K.
template <bool ON16> struct Piece;

static __device__ __noinline__ uint4 single_bytes(const int8_t* a, int left) {
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 16; ++i)
        if (i < left) w[i >> 2] |= (uint32_t)(uint8_t)a[i] << (8 * (i & 3));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <> struct Piece<true> {
    uint4 v;
    // `row`: address of the row's byte 0
    __device__ __forceinline__ void fetch(const ByteRows& m, const int8_t* row, int k) {
        load_if(v, row + k, k + 16 <= m.K);
    }
    __device__ __forceinline__ uint4 value(const ByteRows& m, const int8_t* row, int k, bool inner) {
        if (!inner) {
            const int left = m.K - k;
            if (left < 16) v = left > 0 ? single_bytes(row + k, left) : make_uint4(0, 0, 0, 0);
        }
        return v;
    }
};

template <> struct Piece<false> {
    uint4 b, c;
    __device__ __forceinline__ static bool inside(const ByteRows& m, const int8_t* lo) {
        return lo >= m.p && lo + 32 <= m.end;
    }
    __device__ __forceinline__ void fetch(const ByteRows& m, const int8_t* row, int k) {
        const int8_t* lo = row + k - ((uintptr_t)(row + k) & 15);
        const bool in = k + 16 <= m.K && inside(m, lo);
        load_if(b, lo, in);
        load_if(c, lo + 16, in);
    }
    __device__ __forceinline__ uint4 value(const ByteRows& m, const int8_t* row, int k, bool) {
        const int left = m.K - k;
        const int s = (int)((uintptr_t)(row + k) & 15);
        if (left <= 0) return make_uint4(0, 0, 0, 0);
        if (left < 16 || !inside(m, row + k - s)) return single_bytes(row + k, left);
        // the 32 bytes moved down by s: by words, then by bytes
        uint32_t w[8] = {b.x, b.y, b.z, b.w, c.x, c.y, c.z, c.w};
#pragma unroll
        for (int i = 0; i < 6; ++i) w[i] = (s & 8) ? w[i + 2] : w[i];
#pragma unroll
        for (int i = 0; i < 5; ++i) w[i] = (s & 4) ? w[i + 1] : w[i];
        const uint32_t sel = 0x3210u + 0x1111u * (uint32_t)(s & 3);
        return make_uint4(__byte_perm(w[0], w[1], sel), __byte_perm(w[1], w[2], sel), __byte_perm(w[2], w[3], sel),
                          __byte_perm(w[3], w[4], sel));
    }
};

// Whether a matrix's rows start on 16-byte boundaries.
inline bool rows_on16(const int8_t* p, long long stride, long long rows) {
    return (uintptr_t)p % 16 == 0 && (rows <= 1 || stride % 16 == 0);
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
