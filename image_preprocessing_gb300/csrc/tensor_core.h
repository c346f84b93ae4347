// PTX forms shared by the tcgen05 kernels: mbarriers with bounded waits,
// operand descriptors, reading TMEM.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace trfn {

constexpr unsigned kStatusTimeout = 1u;            // bit of a device status word
constexpr uint64_t kWaitLimitNs = 1000000000ull;   // 1 s

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ uint64_t now_ns() {
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.b32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
// Waits for the phase with this parity; false after about a second, or as soon
// as another thread of the CTA gave up.
static __device__ __noinline__ bool bar_wait_slow(uint32_t bar, uint32_t parity, volatile int* given_up, unsigned* status) {
    uint64_t t0 = 0;   // reading the timer takes longer than a product: not before the wait is a long one
    for (uint32_t i = 1; i < (1u << 28); ++i) {
        if (bar_try(bar, parity)) return true;
        if ((i & 255u) == 0) {
            if (*given_up) return false;
            if (t0 == 0) t0 = now_ns();
            else if (now_ns() - t0 > kWaitLimitNs) break;
        }
    }
    *given_up = 1;
    atomicOr(status, kStatusTimeout);
    return false;
}
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, volatile int* given_up, unsigned* status) {
    return bar_try(bar, parity) || bar_wait_slow(bar, parity, given_up, status);
}
// The same where a CTA ends, for what is in flight: whatever became of the
// other threads' waits, and without a word if it runs out.
static __device__ __noinline__ void bar_drain(uint32_t bar, uint32_t parity) {
    uint64_t t0 = 0;
    for (uint32_t i = 1; i < (1u << 28) && !bar_try(bar, parity); ++i) {
        if ((i & 255u) != 0) continue;
        if (t0 == 0) t0 = now_ns();
        else if (now_ns() - t0 > kWaitLimitNs) return;
    }
}
__device__ __forceinline__ void tmem_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }

// Operand rows of 128 bytes (64 binary16 along K), 128-byte swizzle, 8 rows
// (1024 bytes) to a swizzle atom.
__device__ __forceinline__ uint64_t operand(uint32_t addr) {
    return (uint64_t)((addr >> 4) & 0x3FFF) | (1ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}
// 16 columns of this warp's 32 lanes; v holds them after tmem_wait.
__device__ __forceinline__ void tmem_load16(uint32_t addr, uint32_t* v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(addr));
}
// 4, 8 or 16 columns, likewise.
template <int N>
__device__ __forceinline__ void tmem_load(uint32_t addr, uint32_t (&v)[N]) {
    static_assert(N == 4 || N == 8 || N == 16, "columns of one load");
    if constexpr (N == 16) {
        tmem_load16(addr, v);
    } else if constexpr (N == 8) {
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                     : "r"(addr));
    } else {
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                     : "r"(addr));
    }
}
// Waits for the loads; the values pass through it, so that none is used before.
template <int N>
__device__ __forceinline__ void tmem_wait(uint32_t (&v)[N]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+r"(v[i]));
}

}  // namespace trfn
