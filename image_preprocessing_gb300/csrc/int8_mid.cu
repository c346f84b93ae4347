// The int8 product for up to some hundred tokens (int8_matmul.cu says why it
// multiplies in binary16).
//
// Bound by reading w once while tokens are few, by converting it after.  The
// weights are the product's 128 rows, so that a tile of 16 to 128 tokens fills
// it whatever their number: a CTA, one to an SM, makes 128 channels x T tokens
// over a part of K, in blocks of 64 values.  Four groups of four warps take
// every fourth block: they copy its int8 into shared memory, 100 KB ahead (what
// one SM must have under way to get its share of the HBM rate), and write what
// has landed as binary16 into their swizzled stage; a thread copies and
// converts the same bytes, so the copies need no barrier.  One more thread
// issues tcgen05 products of 128 x T x 16 into TMEM.  Where the tiles are fewer
// than the SMs, a cluster of up to 8 CTAs shares a tile, a part of K each, and
// adds its sums through distributed shared memory as integers, which have no
// order.
#include <atomic>
#include <climits>
#include <type_traits>

#include "int8_parts.h"
#include "tensor_core.h"
#include "token_ops.h"

namespace trfn {
namespace {

__device__ unsigned int g_mid_status;

constexpr int kRows = 128, kBlockK = 64, kExactBlocks = 1024 / kBlockK;
constexpr int kGroups = 4, kGroup = 128;                                  // groups of converting threads
constexpr int kConvert = kGroups * kGroup, kThreads = kConvert + 32;      // and a warp that issues

struct MidParams {
    ByteRows x, w;
    const float* x_scale;
    const float* w_scale;
    const float* bias;
    void* y;
    long long y_stride;
    int tokens, m_tiles, split, blocks;   // of a tile (a multiple of 16), CTAs of a cluster, blocks of K in each
    int wide;                             // groups of 4 channels of y take one store
};

// A stage holds a block in binary16, rows of 128 bytes; the ring holds several in int8, 16 bytes at a time in
// the threads' order.
template <int T> constexpr int kStageBytes = (kRows + T) * 128;
template <int T> constexpr int kRingBytes = (kRows + T) * kBlockK;
template <int T> constexpr int kDeep = T == 16 ? 4 : T == 32 ? 3 : T == 64 ? 2 : 1;   // blocks of the ring for a group
template <int T> constexpr int kSmemBytes = 1024 + kGroups * (kStageBytes<T> + kDeep<T> * kRingBytes<T>);
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

// ONE: at most 1024 products to a sum of this CTA.  ON16: rows on 16-byte
// boundaries; others pass through registers, two blocks ahead.
template <typename E, int T, bool ONE, bool ON16>
__global__ void __launch_bounds__(kThreads, 1) mid_kernel(const MidParams p) {
    constexpr int WP = kRows / kPass, XP = kPieces<T>, DEEP = kDeep<T>, COLS = T < 32 ? 32 : T;
    extern __shared__ uint8_t smem_raw[];
    // full[4] empty[4] sums freed
    __shared__ __align__(8) uint64_t bars[2 * kGroups + 2];
    __shared__ uint32_t tmem_at;
    __shared__ volatile int given_up;
    __shared__ float x_scale[T];
    uint8_t* const stages = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t* const ring = stages + kGroups * kStageBytes<T>;
    const uint32_t bar0 = smem_u32(bars);
    auto full = [&](int s) { return bar0 + 8u * s; };
    auto empty = [&](int s) { return bar0 + 8u * (kGroups + s); };
    const uint32_t sums = bar0 + 8u * (2 * kGroups), freed = bar0 + 8u * (2 * kGroups + 1);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = p.split > 1 ? (int)cluster_rank() : 0;
    const int tile = blockIdx.x / p.split;
    const int m0 = tile % p.m_tiles * p.tokens, n0 = tile / p.m_tiles * kRows;
    const int kb0 = rank * p.blocks;
    const int nkb = max(0, min((p.x.K + kBlockK - 1) / kBlockK - kb0, p.blocks));
    const int parts = (nkb + kExactBlocks - 1) / kExactBlocks;

    // a thread's pieces of a block: 16 bytes of every 32nd row of w and of x.  A warp takes 64 bytes of 8 rows:
    // neither loads nor stores conflict
    const int group = tid / kGroup, me = tid % kGroup, q = tid & 3, row0 = me >> 2;
    const int8_t* wr[WP];
    const int8_t* xr[XP];
    Piece<false> wv[WP], xv[XP];   // unused with ON16
    auto x_mine = [&](int j) { return row0 + kPass * j < p.tokens; };
    // block i is the group's (i / 4)th
    auto slot = [&](int i) { return (group * DEEP + i / kGroups % DEEP) * kRingBytes<T> + me * 16; };
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
    if (tid < kConvert) {
        // rows past the end repeat the last: their sums are not written
#pragma unroll
        for (int j = 0; j < WP; ++j) wr[j] = p.w.p + (long long)min(n0 + row0 + kPass * j, p.w.rows - 1) * p.w.stride;
#pragma unroll
        for (int j = 0; j < XP; ++j) xr[j] = p.x.p + (long long)min(m0 + row0 + kPass * j, p.x.rows - 1) * p.x.stride;
#pragma unroll 1
        for (int d = 0; d < (ON16 ? DEEP : 1); ++d) fetch(group + kGroups * d);
        if (tid < p.tokens) x_scale[tid] = m0 + tid < p.x.rows ? p.x_scale[m0 + tid] : 0.0f;
    } else {
        if (lane == 0) {
            given_up = 0;
            for (int s = 0; s < kGroups; ++s) {
                bar_init(full(s), kGroup / 32);
                bar_init(empty(s), 1);
            }
            bar_init(sums, 1);
            bar_init(freed, kConvert / 32);
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

    if (warp == kConvert / 32) {
        const uint32_t shape = (1u << 4) | ((uint32_t)(p.tokens / 8) << 17) | (8u << 24);   // f16 x f16 -> f32, 128 x tokens
        const uint64_t w0 = operand(smem_u32(stages)), x0 = operand(smem_u32(stages) + kRows * 128);
        int s = 0;
        uint32_t phase = 0;
        for (int part = 0; part < parts && ok; ++part) {
            if (part > 0) ok = __all_sync(0xffffffffu, bar_wait(freed, (part - 1) & 1, &given_up, &g_mid_status));
            if (!ok) break;
            tmem_fence_after();
            const int i0 = part * kExactBlocks, i1 = min(nkb, i0 + kExactBlocks);
            for (int i = i0; i < i1; ++i) {
                ok = __all_sync(0xffffffffu, bar_wait(full(s), phase, &given_up, &g_mid_status));
                if (!ok) break;
                tmem_fence_after();
                const uint32_t at = s * (kStageBytes<T> / 16);   // descriptors count in 16 bytes
#pragma unroll
                for (int k = 0; k < kBlockK / 16; ++k) mma_one(tmem, w0 + at + 2 * k, x0 + at + 2 * k, shape, i > i0 || k > 0);
                commit(empty(s));
                if (++s == kGroups) { s = 0; phase ^= 1u; }
            }
            commit(sums);
            // after a wait that ran out: what was issued is done before TMEM is freed
            if (!ok)
                for (int n = 0; n < (1 << 20) && !bar_try(sums, part & 1); ++n) {}
        }
        __syncwarp();
    }

    constexpr int QT = T / 4, G = QT < 16 ? QT : 16;   // tokens of a warp, columns read at a time
    const int quarter = warp & 3, c_warp = (warp >> 2) * QT, ch = quarter * 32 + lane;
    const uint32_t tmem_mine = tmem + c_warp + ((uint32_t)(quarter * 32) << 16);
    int acc[ONE ? 1 : QT];
    if (tid < kConvert) {
        uint32_t phase = 1;   // of the group's stage, free at first
        uint8_t* const stage = stages + group * kStageBytes<T>;
        for (int i = group; i < nkb; i += kGroups) {
            const int k = (kb0 + i) * kBlockK + q * 16;
            if constexpr (ON16) asm volatile("cp.async.wait_group %0;" ::"n"(DEEP - 1) : "memory");
            ok = __all_sync(0xffffffffu, bar_wait(empty(group), phase, &given_up, &g_mid_status));
            if (!ok) break;
            phase ^= 1u;
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
            if (lane == 0) bar_arrive(full(group));
            fetch(i + kGroups * (ON16 ? DEEP : 1));
            if constexpr (!ONE) {
                const int done = i / kExactBlocks + 1;   // parts converted when this was the group's last block of one
                if (i % kExactBlocks >= kExactBlocks - kGroups && done * kExactBlocks < nkb) {
                    // a sum of 1024 products, and more to come
                    ok = __all_sync(0xffffffffu, bar_wait(sums, (done - 1) & 1, &given_up, &g_mid_status));
                    if (!ok) break;
                    tmem_fence_after();
#pragma unroll
                    for (int c = 0; c < QT; c += G) {
                        uint32_t v[G];
                        tmem_load(tmem_mine + c, v);
                        tmem_wait(v);
#pragma unroll
                        for (int j = 0; j < G; ++j) {
                            const int sum = __float2int_rn(__uint_as_float(v[j]));
                            acc[c + j] = done == 1 ? sum : acc[c + j] + sum;
                        }
                    }
                    tmem_fence_before();
                    __syncwarp();
                    if (lane == 0) bar_arrive(freed);
                }
            }
        }
        if constexpr (ON16) asm volatile("cp.async.wait_all;" ::: "memory");
        if (ok && parts > 0) ok = bar_wait(sums, (parts - 1) & 1, &given_up, &g_mid_status);
        ok = __all_sync(0xffffffffu, ok);
        // the sums of several CTAs go over stages and ring: every thread is done with its part of them
        if (p.split > 1) asm volatile("bar.sync 1, 512;" ::: "memory");
        if (ok) {
            tmem_fence_after();
            const int n = n0 + ch;
            float sw = 0.0f, bias = 0.0f;
            if (p.split == 1 && n < p.w.rows) {
                sw = p.w_scale[n];
                if (p.bias != nullptr) bias = p.bias[n];
            }
            E* y = static_cast<E*>(p.y) + m0 * p.y_stride + n;
            int* const dump = reinterpret_cast<int*>(stages);
#pragma unroll
            for (int c = 0; c < QT; c += G) {
                if (c_warp + c >= p.tokens) break;
                uint32_t v[G];
                if (parts > 0) {
                    tmem_load(tmem_mine + c, v);
                    tmem_wait(v);
                }
#pragma unroll
                for (int j = 0; j < G; ++j) {
                    const int token = c_warp + c + j;
                    int sum = parts > 0 ? __float2int_rn(__uint_as_float(v[j])) : 0;
                    if constexpr (!ONE)
                        if (parts > 1) sum += acc[c + j];
                    if (p.split > 1) dump[token * kRows + ch] = sum;
                    else if (n < p.w.rows && m0 + token < p.x.rows)
                        y[token * p.y_stride] = out_value<E>((float)sum * x_scale[token] * sw + bias);
                }
            }
            tmem_fence_before();
        }
    }
    if (p.split > 1) {
        __syncwarp();
        cluster_sync();   // every CTA's sums are in its shared memory
        if (tid < kConvert) {
            const int c4 = (tid & 31) * 4, n = n0 + c4;
            float sw[4], bias[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                sw[j] = n + j < p.w.rows ? p.w_scale[n + j] : 0.0f;
                bias[j] = n + j < p.w.rows && p.bias != nullptr ? p.bias[n + j] : 0.0f;
            }
            for (int i = warp; rank + p.split * i < p.tokens; i += kConvert / 32) {
                const int token = rank + p.split * i, m = m0 + token;
                if (m >= p.x.rows) break;
                const uint32_t at = smem_u32(stages) + (token * kRows + c4) * 4;
                // all CTAs' sums on their way together
                int4 v[8];
#pragma unroll
                for (int r = 0; r < 8; ++r) v[r] = load_peer(at, r, r < p.split);
                int4 sum = v[0];
#pragma unroll
                for (int r = 1; r < 8; ++r) {
                    sum.x += v[r].x; sum.y += v[r].y; sum.z += v[r].z; sum.w += v[r].w;
                }
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
    if (warp == kConvert / 32) {
        tmem_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(COLS) : "memory");
    }
}

long long pieces_of(long long v, long long of) { return (v + of - 1) / of; }

template <typename E, int T, bool ONE, bool ON16>
int start_mid(const MidParams& p, cudaStream_t st) {
    static std::atomic<bool> ready{false};
    if (!ready.load(std::memory_order_relaxed)) {
        const cudaError_t e = cudaFuncSetAttribute(mid_kernel<E, T, ONE, ON16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   kSmemBytes<T>);
        if (e != cudaSuccess) {
            set_last_error("int8 product kernel set-up", (int)e);
            return TR_ERR_CUDA;
        }
        ready.store(true, std::memory_order_relaxed);
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(pieces_of(p.w.rows, kRows) * p.m_tiles * p.split));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmemBytes<T>;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)p.split;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, mid_kernel<E, T, ONE, ON16>, p);
    if (e != cudaSuccess) {
        set_last_error("cudaLaunchKernelEx(int8 product)", (int)e);
        return TR_ERR_CUDA;
    }
    return launched("int8 product kernel");
}

template <typename E, int T>
int pick_mid(const MidParams& p, bool on16, cudaStream_t st) {
    if (p.blocks <= kExactBlocks) return on16 ? start_mid<E, T, true, true>(p, st) : start_mid<E, T, true, false>(p, st);
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

// Tile and split by an estimate in cycles: a start, a cost for each block, and for adding a cluster's sums.
struct MidPlan { int T, split; long long cycles; };
MidPlan plan_mid(long long M, long long N, long long K) {
    MidPlan best{0, 1, 0};
    const int tiles[4] = {16, 32, 64, 128}, cost[4] = {300, 310, 330, 450};
    const int splits[4] = {1, 2, 4, 8}, room[4] = {152, 152, 144, 120};   // CTAs that run at once in such clusters
    for (int i = 0; i < 4; ++i) {
        const long long at = pieces_of(M, tiles[i]) * pieces_of(N, kRows), blocks = pieces_of(K, kBlockK);
        for (int j = 0; j < 4 && (j == 0 || blocks >= 4 * splits[j]); ++j) {
            const long long waves = pieces_of(at * splits[j], room[j]);
            const long long c = waves * (5000 + pieces_of(blocks, splits[j]) * cost[i] + (j > 0 ? 2000 + 30 * tiles[i] : 0) +
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

int read_mid_status(int* flags, bool clear) {
    unsigned v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_mid_status, sizeof v);
    if (e == cudaSuccess && clear && v != 0) {
        const unsigned zero = 0;
        e = cudaMemcpyToSymbol(g_mid_status, &zero, sizeof zero);
    }
    if (e != cudaSuccess) {
        set_last_error("tr_device_status (int8 product)", (int)e);
        return TR_ERR_CUDA;
    }
    *flags = (int)v;
    return TR_OK;
}

}  // namespace trfn
