// The int8 product for up to some hundred tokens (int8_matmul.cu says why it
// multiplies in binary16).
//
// Bound by reading w once while tokens are few, by converting it after.  The
// weights are the product's 128 rows, so that a tile of 16 to 128 tokens fills
// it whatever their number: a CTA, one to an SM, makes 128 channels x T tokens
// over a part of K, in blocks of 64 values.  Three or four groups of four warps
// take the blocks in turn: they copy int8 into shared memory, 70 KB ahead and
// more (what one SM must have under way to get its share of the HBM rate), and
// write what has landed as binary16 into swizzled stages, of which each group
// has two, so that it converts while its last block is multiplied; a thread
// copies and converts the same bytes, so the copies need no barrier.  Each group
// has a thread more that issues its tcgen05 products of 128 x T x 16 (one thread
// for all takes 500 cycles a block, the HBM rate allows 300), into sums of its
// own in TMEM.  Where the tiles are fewer than the SMs, a cluster of up to 8
// CTAs shares a tile, a part of K each, and adds its sums through distributed
// shared memory.  All of these are added as integers, which have no order.
//
// Measured: 16 x 16384 x 4096 17.7 us (67 MB of weights: 3.8 TB/s), 64 x 4096 x
// 4096 10.4 us, 196 x 4096 x 1024 10.4 us; rows off 16 bytes, 16 x 16384 x 4095,
// 38.4 us.  What is left: a block takes a CTA 380
// cycles where its share of HBM allows 300, and start, first block and epilogue
// are 8000 cycles whatever the size.
#include <atomic>
#include <climits>
#include <cmath>
#include <type_traits>

#include "int8_parts.h"
#include "tensor_core.h"
#include "token_ops.h"

namespace trfn {
namespace {

constexpr int kRows = 128, kBlockK = 64, kExactBlocks = 1024 / kBlockK;
constexpr int kGroup = 128;                                    // threads of a group
template <int T> constexpr int kGroups = T == 16 || T == 128 ? 4 : 3;
template <int T> constexpr int kConvert = kGroups<T> * kGroup;
// warps that issue products, each into T columns of TMEM, and all threads
template <int T> constexpr int kIssuers = T == 128 ? 2 : kGroups<T>;
template <int T> constexpr int kThreads = kConvert<T> + 32 * kIssuers<T>;
// blocks to a sum of 1024 products in every issuer's columns
template <int T> constexpr int kPartBlocks = kExactBlocks * kIssuers<T>;

struct MidParams {
    ByteRows x, w;
    const float* x_scale;
    const float* w_scale;
    const float* bias;
    void* y;
    long long y_stride;
    int tokens, m_tiles, split, blocks;   // of a tile (a multiple of 16), CTAs of a cluster, blocks of K in each
    int wide;                             // groups of 4 channels of y take one store
    int missing;                          // test hook: arrivals that the first stage waits for in vain
    unsigned* status;                     // the product's status word
};

// A stage holds a block in binary16, rows of 128 bytes; the ring holds several in int8, 16 bytes at a time in
// the threads' order.
template <int T> constexpr int kStageBytes = (kRows + T) * 128;
template <int T> constexpr int kRingBytes = (kRows + T) * kBlockK;
template <int T> constexpr int kSlots = T == 128 ? 1 : 2;                  // stages of a group
template <int T> constexpr int kStages = kGroups<T> * kSlots<T>;
template <int T> constexpr int kDeep = T == 32 ? 3 : T == 128 ? 1 : 2;     // blocks of the ring for a group
template <int T> constexpr int kSmemBytes = 1024 + kStages<T> * kStageBytes<T> + kGroups<T> * kDeep<T> * kRingBytes<T>;
// What a CTA of a cluster gives for sums that a wait has kept it from; the sums themselves stay above -2^31 + 2^14.
constexpr int kNoSum = INT_MIN;
constexpr int kPass = kGroup / 4;                                                     // rows of a group's threads
template <int T> constexpr int kPieces = T < kPass ? 1 : T / kPass;                   // of x, for a thread and block

// Issued by the whole warp for its one elected thread: a branch around it would leave the compiler without
// the knowledge that its operands are the warp's (measured: 85 cycles a product instead of some).
__device__ __forceinline__ void mma_one(uint32_t d, uint64_t a, uint64_t b, uint32_t shape, uint32_t add) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(shape), "r"(add)
        : "memory");
}
// Arrives on `bar` when the products issued so far are done.
__device__ __forceinline__ void commit(uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
        : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// 16 bytes at this CTA's address `addr` in another CTA of the cluster, or zeros.
__device__ __forceinline__ int4 load_peer(uint32_t addr, uint32_t rank, bool in) {
    int4 v = make_int4(0, 0, 0, 0);
    asm volatile(
        "{\n\t.reg .b32 a;\n\t.reg .pred p;\n\t"
        "setp.ne.u32 p, %6, 0;\n\t"
        "@p mapa.shared::cluster.u32 a, %4, %5;\n\t"
        "@p ld.shared::cluster.v4.s32 {%0, %1, %2, %3}, [a];\n\t}"
        : "+r"(v.x), "+r"(v.y), "+r"(v.z), "+r"(v.w)
        : "r"(addr), "r"(rank), "r"((uint32_t)in)
        : "memory");
    return v;
}

__device__ __forceinline__ void copy16(uint32_t dst, const int8_t* src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// ONE: at most 1024 products to each sum in TMEM.  ON16: rows on 16-byte
// boundaries; others pass through registers, two blocks ahead.
template <typename E, int T, bool ONE, bool ON16>
__global__ void __launch_bounds__(kThreads<T>, 1) mid_kernel(const MidParams p) {
    constexpr int WP = kRows / kPass, XP = kPieces<T>, DEEP = kDeep<T>, NI = kIssuers<T>, PART = kPartBlocks<T>;
    constexpr int GR = kGroups<T>, SL = kSlots<T>, ST = kStages<T>, CONVERT = kConvert<T>, COLS = T == 16 || NI == 2 ? NI * T : 4 * T;
    extern __shared__ uint8_t smem_raw[];
    // full[ST] empty[ST] sums freed
    __shared__ __align__(8) uint64_t bars[2 * ST + 2];
    __shared__ uint32_t tmem_at;
    __shared__ volatile int given_up;
    __shared__ float x_scale[T];
    __shared__ float2 channel[kRows];   // scale and bias
    uint8_t* const stages = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t* const ring = stages + ST * kStageBytes<T>;
    const uint32_t bar0 = smem_u32(bars);
    auto full = [&](int s) { return bar0 + 8u * s; };
    auto empty = [&](int s) { return bar0 + 8u * (ST + s); };
    const uint32_t sums = bar0 + 8u * (2 * ST), freed = bar0 + 8u * (2 * ST + 1);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = p.split > 1 ? (int)cluster_rank() : 0;
    const int tile = blockIdx.x / p.split;
    const int m0 = tile % p.m_tiles * p.tokens, n0 = tile / p.m_tiles * kRows;
    const int kb0 = rank * p.blocks;
    const int nkb = max(0, min((p.x.K + kBlockK - 1) / kBlockK - kb0, p.blocks));
    const int parts = (nkb + PART - 1) / PART;

    // a thread's pieces of a block: 16 bytes of every 32nd row of w and of x.  A warp takes 64 bytes of 8 rows:
    // neither loads nor stores conflict
    const int group = tid / kGroup, me = tid % kGroup, q = tid & 3, row0 = me >> 2;
    const int8_t* wr[WP];
    const int8_t* xr[XP];
    Piece<false> wv[WP], xv[XP];   // unused with ON16
    auto x_mine = [&](int j) { return row0 + kPass * j < p.tokens; };
    // block i is the group's (i / GR)th, in its stage i / GR % SL
    auto slot = [&](int i) { return (group * DEEP + i / GR % DEEP) * kRingBytes<T> + me * 16; };
    auto fetch = [&](int i) {
        const int k = (kb0 + i) * kBlockK + q * 16;
        if constexpr (ON16) {
            if (i < nkb) {
                const int bytes = max(0, min(16, p.w.K - k));   // the rest is zeros
                const long long at = bytes > 0 ? k : 0;
                const uint32_t to = smem_u32(ring) + slot(i);
#pragma unroll
                for (int j = 0; j < WP; ++j) copy16(to + j * kGroup * 16, wr[j] + at, bytes);
#pragma unroll
                for (int j = 0; j < XP; ++j)
                    if (x_mine(j)) copy16(to + (WP + j) * kGroup * 16, xr[j] + at, bytes);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        } else {
            const int kk = i < nkb ? k : p.w.K;
#pragma unroll
            for (int j = 0; j < WP; ++j) wv[j].fetch(p.w, wr[j], kk);
#pragma unroll
            for (int j = 0; j < XP; ++j) xv[j].fetch(p.x, xr[j], x_mine(j) ? kk : p.x.K);
        }
    };
    if (tid < CONVERT) {
        // what the kernel before this one in the stream writes may be x or w, and what it reads y
        asm volatile("griddepcontrol.wait;" ::: "memory");
        // rows past the end repeat the last: their sums are not written
#pragma unroll
        for (int j = 0; j < WP; ++j) wr[j] = p.w.p + (long long)min(n0 + row0 + kPass * j, p.w.rows - 1) * p.w.stride;
#pragma unroll
        for (int j = 0; j < XP; ++j) xr[j] = p.x.p + (long long)min(m0 + row0 + kPass * j, p.x.rows - 1) * p.x.stride;
#pragma unroll 1
        for (int d = 0; d < (ON16 ? DEEP : 1); ++d) fetch(group + GR * d);
    } else if (warp == CONVERT / 32) {
        if (lane == 0) {
            given_up = 0;
            for (int s = 0; s < ST; ++s) {
                bar_init(full(s), kGroup / 32 + (s == 0 && blockIdx.x == 0 ? p.missing : 0));
                bar_init(empty(s), 1);
            }
            bar_init(sums, NI);
            bar_init(freed, CONVERT / 32);
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        }
        __syncwarp();
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_at)),
                     "r"(COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        tmem_fence_before();
    }
    __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = tmem_at;
    bool ok = true;

    if (warp >= CONVERT / 32) {
        const int issuer = warp - CONVERT / 32;   // takes blocks issuer, issuer + NI, ...
        const uint32_t shape = (1u << 4) | ((uint32_t)(p.tokens / 8) << 17) | (8u << 24);   // f16 x f16 -> f32, 128 x tokens
        const uint64_t w0 = operand(smem_u32(stages)), x0 = operand(smem_u32(stages) + kRows * 128);
        const uint32_t d = tmem + issuer * T;
        int s = issuer * SL, slot_of = 0;   // stages in the order of the blocks: slot 0 of each group, slot 1 ...
        uint32_t phase = 0;
        uint32_t last = 0, last_phase = 0;        // the stage whose products were issued last
        for (int part = 0; part < parts && ok; ++part) {
            if (part > 0) ok = __all_sync(0xffffffffu, bar_wait(freed, (part - 1) & 1, &given_up, p.status));
            if (!ok) break;
            tmem_fence_after();
            const int i0 = part * PART + issuer, i1 = min(nkb, (part + 1) * PART);
            for (int i = i0; i < i1; i += NI) {
                ok = __all_sync(0xffffffffu, bar_wait(full(s), phase, &given_up, p.status));
                if (!ok) break;
                tmem_fence_after();
                const uint32_t at = s * (kStageBytes<T> / 16);   // descriptors count in 16 bytes
#pragma unroll
                for (int k = 0; k < kBlockK / 16; ++k) mma_one(d, w0 + at + 2 * k, x0 + at + 2 * k, shape, i > i0 || k > 0);
                commit(empty(s));
                last = empty(s);
                last_phase = phase;
                if constexpr (NI == GR) {        // one group's stages in turn
                    if (++slot_of == SL) { slot_of = 0; phase ^= 1u; }
                    s = issuer * SL + slot_of;
                } else {                         // every second group's one stage
                    s += NI;
                    if (s >= ST) { s = issuer; phase ^= 1u; }
                }
            }
            if (ok) commit(sums);   // (else they are not whole: nobody gets them)
        }
        if (last != 0) bar_drain(last, last_phase);   // what was issued is done before TMEM is freed
        __syncwarp();
    }

    // a warp reads a quarter of the channels, and every GR-th G tokens
    constexpr int G = T / 4 < 16 ? T / 4 : 16, U = (T / G + GR - 1) / GR;
    const int quarter = warp & 3, ch = quarter * 32 + lane;
    const uint32_t tmem_mine = tmem + ((uint32_t)(quarter * 32) << 16);
    auto column = [&](int u) { return ((warp >> 2) + GR * u) * G; };
    // the sum of the issuers' sums of one part at columns c .. c+G-1; an issuer without blocks
    // in the part has written none
    auto read_sums = [&](int c, int blocks, int (&v)[G]) {
        uint32_t f[NI][G];
#pragma unroll
        for (int j = 0; j < NI; ++j)
            if (j < blocks) tmem_load(tmem_mine + j * T + c, f[j]);
#pragma unroll
        for (int j = 0; j < NI; ++j) tmem_wait(f[j]);
#pragma unroll
        for (int i = 0; i < G; ++i) {
            v[i] = 0;
#pragma unroll
            for (int j = 0; j < NI; ++j)
                if (j < blocks) v[i] += __float2int_rn(__uint_as_float(f[j][i]));
        }
    };
    int acc[ONE ? 1 : U][G];
    if (tid < CONVERT) {
        // scales are on their way while the sums are made
        const float my_scale = tid < p.tokens && m0 + tid < p.x.rows ? p.x_scale[m0 + tid] : 0.0f;
        float2 my_channel = make_float2(0.0f, 0.0f);
        if (tid < kRows && n0 + tid < p.w.rows)
            my_channel = make_float2(p.w_scale[n0 + tid], p.bias != nullptr ? p.bias[n0 + tid] : 0.0f);
        int at = group * SL;
        uint32_t phase = 1;   // of the group's stages, free at first
        for (int i = group; i < nkb; i += GR) {
            const int k = (kb0 + i) * kBlockK + q * 16;
            if constexpr (ON16) asm volatile("cp.async.wait_group %0;" ::"n"(DEEP - 1) : "memory");
            ok = __all_sync(0xffffffffu, bar_wait(empty(at), phase, &given_up, p.status));
            if (!ok) break;
            uint8_t* const stage = stages + at * kStageBytes<T>;
            auto put = [&](uint8_t* rows, int r, const uint4& v) {
                uint4 a, b;
                int8_to_half(v.x, a.x, a.y);
                int8_to_half(v.y, a.z, a.w);
                int8_to_half(v.z, b.x, b.y);
                int8_to_half(v.w, b.z, b.w);
                const int c = (2 * q) ^ (r & 7);
                *reinterpret_cast<uint4*>(rows + r * 128 + c * 16) = a;
                *reinterpret_cast<uint4*>(rows + r * 128 + (c ^ 1) * 16) = b;
            };
            const uint8_t* from = ring + slot(i);
#pragma unroll
            for (int j = 0; j < WP; ++j)
                put(stage, row0 + kPass * j,
                    ON16 ? *reinterpret_cast<const uint4*>(from + j * kGroup * 16) : wv[j].value(p.w, wr[j], k, false));
#pragma unroll
            for (int j = 0; j < XP; ++j)
                if (x_mine(j))
                    put(stage + kRows * 128, row0 + kPass * j,
                        ON16 ? *reinterpret_cast<const uint4*>(from + (WP + j) * kGroup * 16)
                             : xv[j].value(p.x, xr[j], k, false));
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // the tensor cores read it next
            __syncwarp();
            if (lane == 0) bar_arrive(full(at));
            if (++at == (group + 1) * SL) { at = group * SL; phase ^= 1u; }
            fetch(i + GR * (ON16 ? DEEP : 1));
            if constexpr (!ONE) {
                const int done = i / PART + 1;   // parts converted, when this was the group's last block of one
                if (i % PART >= PART - GR && done * PART < nkb) {
                    // sums of 1024 products, and more to come
                    ok = __all_sync(0xffffffffu, bar_wait(sums, (done - 1) & 1, &given_up, p.status));
                    if (!ok) break;
                    tmem_fence_after();
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        if (column(u) >= p.tokens) continue;
                        int v[G];
                        read_sums(column(u), PART, v);
#pragma unroll
                        for (int j = 0; j < G; ++j) acc[u][j] = done == 1 ? v[j] : acc[u][j] + v[j];
                    }
                    tmem_fence_before();
                    __syncwarp();
                    if (lane == 0) bar_arrive(freed);
                }
            }
        }
        if constexpr (ON16) asm volatile("cp.async.wait_all;" ::: "memory");
        if (ok && parts > 0) ok = bar_wait(sums, (parts - 1) & 1, &given_up, p.status);
        ok = __all_sync(0xffffffffu, ok);
        if (tid < p.tokens) x_scale[tid] = my_scale;
        if (tid < kRows) channel[tid] = my_channel;
        // every thread is done with its part of the stages and the ring, where a cluster's sums go
        asm volatile("bar.sync 1, %0;" ::"n"(CONVERT) : "memory");
        if (ok) {
            tmem_fence_after();
            const int n = n0 + ch;
            const float sw = channel[ch].x, bias = channel[ch].y;
            E* y = static_cast<E*>(p.y) + m0 * p.y_stride + n;
            int* const dump = reinterpret_cast<int*>(stages);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int c = column(u);
                if (c >= p.tokens) continue;
                int v[G];
                read_sums(c, nkb - max(parts - 1, 0) * PART, v);
#pragma unroll
                for (int j = 0; j < G; ++j) {
                    const int token = c + j;
                    int sum = v[j];
                    if constexpr (!ONE)
                        if (parts > 1) sum += acc[u][j];
                    if (p.split > 1) dump[token * kRows + ch] = sum;
                    else if (n < p.w.rows && m0 + token < p.x.rows)
                        y[token * p.y_stride] = out_value<E>((float)sum * x_scale[token] * sw + bias);
                }
            }
            tmem_fence_before();
        } else if (p.split > 1) {
            int* const dump = reinterpret_cast<int*>(stages);
#pragma unroll
            for (int u = 0; u < U; ++u)
                for (int j = 0; j < G && column(u) < p.tokens; ++j) dump[(column(u) + j) * kRows + ch] = kNoSum;
        }
    }
    if (p.split > 1) {
        __syncwarp();
        cluster_sync();   // every CTA's sums are in its shared memory
        if (tid < CONVERT) {
            const int c4 = (tid & 31) * 4, n = n0 + c4;
            float sw[4], bias[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) { sw[j] = channel[c4 + j].x; bias[j] = channel[c4 + j].y; }
            for (int i = warp; rank + p.split * i < p.tokens; i += CONVERT / 32) {
                const int token = rank + p.split * i, m = m0 + token;
                if (m >= p.x.rows) break;
                const uint32_t at = smem_u32(stages) + (token * kRows + c4) * 4;
                // all CTAs' sums on their way together
                int4 v[8];
#pragma unroll
                for (int r = 0; r < 8; ++r) v[r] = load_peer(at, r, r < p.split);
                int4 sum = v[0];
                bool lost = v[0].x == kNoSum;
#pragma unroll
                for (int r = 1; r < 8; ++r) {
                    lost |= v[r].x == kNoSum;
                    sum.x += v[r].x; sum.y += v[r].y; sum.z += v[r].z; sum.w += v[r].w;
                }
                if (lost) continue;
                const float sx = x_scale[token];
                union { typename std::conditional<sizeof(E) == 4, uint4, uint2>::type word; E e[4]; } o;
                o.e[0] = out_value<E>((float)sum.x * sx * sw[0] + bias[0]);
                o.e[1] = out_value<E>((float)sum.y * sx * sw[1] + bias[1]);
                o.e[2] = out_value<E>((float)sum.z * sx * sw[2] + bias[2]);
                o.e[3] = out_value<E>((float)sum.w * sx * sw[3] + bias[3]);
                E* y = static_cast<E*>(p.y) + m * p.y_stride + n;
                if (p.wide && n + 4 <= p.w.rows) {
                    *reinterpret_cast<decltype(o.word)*>(y) = o.word;
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (n + j < p.w.rows) y[j] = o.e[j];
                }
            }
        }
        __syncwarp();
        // no CTA leaves while another reads its sums; relaxed: a release would wait for the stores to y
        asm volatile("barrier.cluster.arrive.relaxed.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
    }
    __syncthreads();
    if (warp == CONVERT / 32) {
        tmem_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(COLS) : "memory");
    }
}

long long pieces_of(long long v, long long of) { return (v + of - 1) / of; }

template <typename E, int T, bool ONE, bool ON16>
int start_mid(const MidParams& q, cudaStream_t st) {
    MidParams p = q;
    static std::atomic<bool> set_up[kMaxDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || dev < 0 || dev >= kMaxDevices) return cuda_failed("cudaGetDevice", (int)e);
    const int rc = product_status_word(dev, &p.status);
    if (rc != TR_OK) return rc;
    std::atomic<bool>& ready = set_up[dev];
    if (!ready.load(std::memory_order_relaxed)) {
        e = cudaFuncSetAttribute(mid_kernel<E, T, ONE, ON16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   kSmemBytes<T>);
        if (e != cudaSuccess) return cuda_failed("int8 product kernel set-up", (int)e);
        ready.store(true, std::memory_order_relaxed);
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(pieces_of(p.w.rows, kRows) * p.m_tiles * p.split));
    cfg.blockDim = dim3(kThreads<T>);
    cfg.dynamicSmemBytes = kSmemBytes<T>;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)p.split;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    // barriers and TMEM are set up while the kernel before ends
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return launched("int8 product kernel", (int)cudaLaunchKernelEx(&cfg, mid_kernel<E, T, ONE, ON16>, p));
}

template <typename E, int T>
int pick_mid(const MidParams& p, bool on16, cudaStream_t st) {
    if (p.blocks <= kPartBlocks<T>) return on16 ? start_mid<E, T, true, true>(p, st) : start_mid<E, T, true, false>(p, st);
    return on16 ? start_mid<E, T, false, true>(p, st) : start_mid<E, T, false, false>(p, st);
}

template <typename E>
int tile_mid(const MidParams& p, int T, bool on16, cudaStream_t st) {
    switch (T) {
        case 16: return pick_mid<E, 16>(p, on16, st);
        case 32: return pick_mid<E, 32>(p, on16, st);
        case 64: return pick_mid<E, 64>(p, on16, st);
        default: return pick_mid<E, 128>(p, on16, st);
    }
}

// Tile and split by an estimate in cycles, fitted to measurements from 9 x 300 x 300 to 4096 x 16384 x 4096:
// a start, a cost for each block of K, and for adding a cluster's sums.
struct MidPlan { int T, split; double cycles; };
MidPlan plan_mid(long long M, long long N, long long K) {
    MidPlan best{0, 1, 0.0};
    constexpr int tiles[4] = {16, 32, 64, 128}, cost[4] = {380, 430, 520, 1000};
    constexpr int splits[4] = {1, 2, 4, 8}, room[4] = {152, 152, 144, 120};   // CTAs that run at once in such clusters
    const double blocks = std::ceil((double)K / kBlockK), n_tiles = std::ceil((double)N / kRows);
    // contiguous rows off 16-byte boundaries; that strides put others off them is not known here (16 x 16384 x
    // 4095 38.4 us, x 4096 17.7)
    const double slow = K % 16 == 0 ? 1.0 : 2.0;
    for (int i = 0; i < 4; ++i) {
        const double at = std::ceil((double)M / tiles[i]) * n_tiles;
        for (int j = 0; j < 4 && (j == 0 || blocks >= 4 * splits[j]); ++j) {
            const double c = std::ceil(at * splits[j] / room[j]) *
                             (5000 + std::ceil(blocks / splits[j]) * cost[i] * slow + (j > 0 ? 2000 + 30 * tiles[i] : 0) +
                              tiles[i] * 8);
            if (best.T == 0 || c < best.cycles) best = MidPlan{tiles[i], splits[j], c};
        }
    }
    return best;
}

}  // namespace

int launch_int8_mid(const MatmulArgs& a) {
    MidParams p;
    p.x = ByteRows{a.x, a.x_stride, a.x + (a.M - 1) * a.x_stride + a.K, a.M, a.K};
    p.w = ByteRows{a.w, a.w_stride, a.w + (a.N - 1) * a.w_stride + a.K, a.N, a.K};
    p.x_scale = a.x_scale;
    p.w_scale = a.w_scale;
    p.bias = a.bias;
    p.y = a.y;
    p.y_stride = a.y_stride;
    p.missing = test_waits();
    const MidPlan plan = plan_mid(a.M, a.N, a.K);
    p.m_tiles = (int)pieces_of(a.M, plan.T);
    p.tokens = (int)pieces_of(pieces_of(a.M, p.m_tiles), 16) * 16;
    p.split = plan.split;
    p.blocks = (int)pieces_of(pieces_of(a.K, kBlockK), p.split);
    if (pieces_of(a.N, kRows) * p.m_tiles * p.split > INT_MAX) return TR_ERR_NOT_SUPPORTED;
    const int es = a.out_dtype == TR_ELEM_F32 ? 4 : 2;
    p.wide = (uintptr_t)a.y % (4 * es) == 0 && (a.y_stride % 4 == 0 || a.M <= 1);
    const bool on16 = rows_on16(a.x, a.x_stride, a.M) && rows_on16(a.w, a.w_stride, a.N);
    cudaStream_t st = static_cast<cudaStream_t>(a.stream);
    if (a.out_dtype == TR_ELEM_F32) return tile_mid<float>(p, plan.T, on16, st);
    if (a.out_dtype == TR_ELEM_F16) return tile_mid<__half>(p, plan.T, on16, st);
    return tile_mid<__nv_bfloat16>(p, plan.T, on16, st);
}

double int8_mid_cycles(long long M, long long N, long long K) { return plan_mid(M, N, K).cycles; }

}  // namespace trfn
