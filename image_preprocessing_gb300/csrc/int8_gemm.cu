// The int8 product for many tokens: binary16 copies of x and w, then a
// tcgen05 product of the copies (int8_matmul.cu says why that is exact).
//
// Copies.  Both matrices go into the workspace as blocks of 128 rows x 64
// values: 16 KB, rows of 128 bytes whose 16-byte pieces are swizzled (piece c
// of row r at c ^ (r & 7)) as the tensor cores read them from shared memory.
// A block is then one contiguous bulk copy, whatever the alignment of x and w.
//
// Product.  Bound by the tensor cores.  Two CTAs (a cluster on two SMs) make a
// tile of 256 tokens x BN channels with cta_group::2 products of 256 x BN x 16:
// each holds 128 tokens of x and BN/2 channels of w in a ring of shared-memory
// stages, and 128 x BN binary32 sums in TMEM.  One thread copies, one (in the
// even CTA) issues the products, eight warps read the sums: sums of 1024
// products are read into integer registers while the other half of TMEM
// takes the next 1024, so the reading is hidden.
#include <atomic>

#include "int8_parts.h"
#include "token_ops.h"

namespace trfn {
namespace {

__device__ unsigned int g_gemm_status;
constexpr unsigned kStatusTimeout = 1u;
constexpr uint64_t kWaitLimitNs = 1000000000ull;   // 1 s

constexpr int kBlockRows = 128, kBlockK = 64, kBlockBytes = kBlockRows * kBlockK * 2;
constexpr int kExactBlocks = 1024 / kBlockK;       // blocks of K summed in binary32
constexpr int kEpilogueWarps = 8;
constexpr int kThreads = 32 * (4 + kEpilogueWarps);

// ------------------------------------------------------------- PTX forms ---

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
// Arrives on the even CTA's barrier at this CTA's address `bar`.
__device__ __forceinline__ void bar_arrive_even(uint32_t bar) {
    asm volatile(
        "{\n\t.reg .b32 a;\n\t"
        "mapa.shared::cluster.u32 a, %0, 0;\n\t"
        "mbarrier.arrive.release.cluster.shared::cluster.b64 _, [a];\n\t}" ::"r"(bar)
        : "memory");
}
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.b32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
// Waits for the phase with this parity; false after about a second, or as soon
// as another thread of the CTA gave up.
__device__ __noinline__ bool bar_wait_slow(uint32_t bar, uint32_t parity, volatile int* given_up) {
    const uint64_t t0 = now_ns();
    for (uint32_t i = 0; i < (1u << 28); ++i) {
        if (bar_try(bar, parity)) return true;
        if (*given_up) return false;
        if ((i & 63u) == 63u && now_ns() - t0 > kWaitLimitNs) break;
    }
    *given_up = 1;
    atomicOr(&g_gemm_status, kStatusTimeout);
    return false;
}
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, volatile int* given_up) {
    return bar_try(bar, parity) || bar_wait_slow(bar, parity, given_up);
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void tmem_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }

// Operand rows of 128 bytes (64 binary16 along K), 128-byte swizzle, 8 rows
// (1024 bytes) to a swizzle atom.
__device__ __forceinline__ uint64_t operand(uint32_t addr) {
    return (uint64_t)((addr >> 4) & 0x3FFF) | (1ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}
__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t shape, uint32_t add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(shape), "r"(add)
        : "memory");
}
// Arrives on `bar` of both CTAs when the products issued so far are done.
__device__ __forceinline__ void commit_both(uint32_t bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"((uint16_t)3)
        : "memory");
}
__device__ __forceinline__ void tmem_load32(uint32_t addr, uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
          "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
          "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(addr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// ---------------------------------------------------------------- copies ---

struct CopyParams {
    ByteRows x, w;
    uint4* xh;
    uint4* wh;
    long long x_pieces, w_pieces;   // 16-value pieces, of whole blocks
    int k_blocks;
};

// A thread copies 16 values; four threads a block row, eight rows a warp, so a
// warp writes a swizzle atom of 1 KB.
template <bool ON16>
__global__ void __launch_bounds__(256) copy_kernel(const CopyParams p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const long long all = p.x_pieces + p.w_pieces, step = (long long)gridDim.x * blockDim.x;
    for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < all; i += step) {
        const bool of_w = i >= p.x_pieces;
        const long long j = of_w ? i - p.x_pieces : i;
        const int q = (int)(j & 3), r = (int)(j >> 2) & (kBlockRows - 1);
        const long long block = j >> 9;
        const long long row = block / p.k_blocks * kBlockRows + r;
        const int k = (int)(block % p.k_blocks) * kBlockK + q * 16;
        const ByteRows m{of_w ? p.w.p : p.x.p, of_w ? p.w.stride : p.x.stride, of_w ? p.w.end : p.x.end,
                         of_w ? p.w.rows : p.x.rows, p.x.K};
        uint4 v = make_uint4(0, 0, 0, 0);
        if (row < m.rows) v = load16<ON16>(m, row, k);
        uint4 a, b;
        int8_to_half(v.x, a.x, a.y);
        int8_to_half(v.y, a.z, a.w);
        int8_to_half(v.z, b.x, b.y);
        int8_to_half(v.w, b.z, b.w);
        uint4* line = (of_w ? p.wh : p.xh) + block * (kBlockBytes / 16) + r * 8;
        line[(2 * q) ^ (r & 7)] = a;
        line[(2 * q + 1) ^ (r & 7)] = b;
    }
}

// --------------------------------------------------------------- product ---

struct GemmParams {
    const uint8_t* xh;        // blocks of x, then of w
    const uint8_t* wh;
    const float* x_scale;
    const float* w_scale;
    const float* bias;
    void* y;
    long long y_stride;
    int M, N, k_blocks, m_tiles, n_tiles, wide;   // wide: rows of y take 16-byte stores
};

template <int BN> constexpr int kStageBytes = kBlockBytes + BN / 2 * 128;
template <int BN> constexpr int kStages = BN == 256 ? 6 : 8;
template <int BN> constexpr int kSmemBytes = kStages<BN> * kStageBytes<BN> + 1024;

template <typename E, int BN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1) gemm_kernel(const GemmParams p) {
    constexpr int ST = kStages<BN>;
    extern __shared__ uint8_t smem_raw[];
    // full[ST] peer[ST] empty[ST] sums_full[2] sums_empty[2]
    __shared__ __align__(8) uint64_t bars[3 * ST + 4];
    __shared__ uint32_t tmem_at;
    __shared__ volatile int given_up;
    const uint32_t ring = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t bar0 = smem_u32(bars);
    auto full = [&](int s) { return bar0 + 8u * s; };
    auto peer = [&](int s) { return bar0 + 8u * (ST + s); };
    auto empty = [&](int s) { return bar0 + 8u * (2 * ST + s); };
    auto sums_full = [&](int s) { return bar0 + 8u * (3 * ST + s); };
    auto sums_empty = [&](int s) { return bar0 + 8u * (3 * ST + 2 + s); };
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();

    if (threadIdx.x == 0) {
        given_up = 0;
        for (int s = 0; s < ST; ++s) {
            bar_init(full(s), 1);
            bar_init(peer(s), 1);
            bar_init(empty(s), 1);
        }
        for (int s = 0; s < 2; ++s) {
            bar_init(sums_full(s), 1);
            bar_init(sums_empty(s), 2 * kEpilogueWarps);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 2) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_at)),
                     "r"(2 * BN)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        tmem_fence_before();
    }
    __syncthreads();
    cluster_sync();
    tmem_fence_after();
    const uint32_t tmem = tmem_at;

    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    const int tiles = p.m_tiles * p.n_tiles;
    const int parts = (p.k_blocks + kExactBlocks - 1) / kExactBlocks;

    if (warp == 0) {
        if (lane == 0) {
            asm volatile("griddepcontrol.wait;" ::: "memory");   // the copies are made by the kernel before
            int s = 0, issued = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int tile = pair; tile < tiles && ok; tile += pairs) {
                const long long mt = tile / p.n_tiles, nt = tile % p.n_tiles;
                const uint8_t* xb = p.xh + (mt * 2 + rank) * p.k_blocks * kBlockBytes;
                // this CTA's BN/2 channels: a block, or half of one
                const long long ch = nt * BN + (long long)rank * (BN / 2);
                const uint8_t* wb = p.wh + (ch >> 7) * p.k_blocks * kBlockBytes + (ch & 127) * 128;
                for (int kb = 0; kb < p.k_blocks; ++kb) {
                    if (!bar_wait(empty(s), phase ^ 1u, &given_up)) { ok = false; break; }
                    const uint32_t at = ring + s * kStageBytes<BN>;
                    bar_expect(full(s), kStageBytes<BN>);
                    bulk_load(at, xb + (long long)kb * kBlockBytes, kBlockBytes, full(s));
                    bulk_load(at + kBlockBytes, wb + (long long)kb * kBlockBytes, BN / 2 * 128, full(s));
                    issued = issued < ST ? issued + 1 : ST;
                    if (++s == ST) { s = 0; phase ^= 1u; }
                }
            }
            // copies in flight land before the CTA ends, whatever became of the others
            for (int i = 0; i < issued; ++i) {
                s = s == 0 ? ST - 1 : s - 1;
                if (s == ST - 1) phase ^= 1u;
                for (int n = 0; n < (1 << 20) && !bar_try(full(s), phase); ++n) {}
            }
        }
    } else if (warp == 1 && rank == 0) {
        if (lane == 0) {
            constexpr uint32_t shape = (1u << 4) | ((uint32_t)(BN / 8) << 17) | (16u << 24);   // f16 x f16 -> f32, 256 x BN
            int s = 0, half = 0;
            uint32_t phase = 0, half_phase = 0;
            bool ok = true;
            for (int tile = pair; tile < tiles && ok; tile += pairs) {
                for (int part = 0; part < parts && ok; ++part) {
                    ok = bar_wait(sums_empty(half), half_phase ^ 1u, &given_up);
                    if (!ok) break;
                    tmem_fence_after();
                    const uint32_t d = tmem + half * BN;
                    const int kb0 = part * kExactBlocks, kb1 = min(p.k_blocks, kb0 + kExactBlocks);
                    for (int kb = kb0; kb < kb1; ++kb) {
                        ok = bar_wait(full(s), phase, &given_up) && bar_wait(peer(s), phase, &given_up);
                        if (!ok) break;
                        tmem_fence_after();
                        const uint32_t at = ring + s * kStageBytes<BN>;
#pragma unroll
                        for (int k = 0; k < kBlockK / 16; ++k)
                            mma_pair(d, operand(at + 32 * k), operand(at + kBlockBytes + 32 * k), shape, kb > kb0 || k > 0);
                        commit_both(empty(s));
                        if (++s == ST) { s = 0; phase ^= 1u; }
                    }
                    commit_both(sums_full(half));
                    if (++half == 2) { half = 0; half_phase ^= 1u; }
                }
            }
            // the last products are done before TMEM is freed: their arrival on sums_full of the half before
            const int last = half ^ 1;
            const uint32_t last_phase = half == 0 ? half_phase ^ 1u : half_phase;
            if (pair < tiles)
                for (int n = 0; n < (1 << 20) && !bar_try(sums_full(last), last_phase); ++n) {}
        }
    } else if (warp == 1) {
        if (lane == 0) {   // tells the even CTA that this one's half of a stage has landed
            int s = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int tile = pair; tile < tiles && ok; tile += pairs)
                for (int kb = 0; kb < p.k_blocks; ++kb) {
                    ok = bar_wait(full(s), phase, &given_up);
                    if (!ok) break;
                    bar_arrive_even(peer(s));
                    if (++s == ST) { s = 0; phase ^= 1u; }
                }
        }
    } else if (warp >= 4) {
        constexpr int W = BN / 2;                                  // channels of a warp
        const int quarter = warp & 3, col0 = (warp - 4) / 4 * W;
        int half = 0;
        uint32_t half_phase = 0;
        bool ok = true;
        for (int tile = pair; tile < tiles && ok; tile += pairs) {
            const int mt = tile / p.n_tiles, nt = tile % p.n_tiles;
            int acc[W];
            for (int part = 0; part < parts; ++part) {
                ok = bar_wait(sums_full(half), half_phase, &given_up);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tmem_fence_after();
                const uint32_t at = tmem + half * BN + col0 + ((uint32_t)(quarter * 32) << 16);
#pragma unroll
                for (int c = 0; c < W; c += 32) {
                    uint32_t v[32];
                    tmem_load32(at + c, v);
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        const int sum = __float2int_rn(__uint_as_float(v[i]));
                        acc[c + i] = part == 0 ? sum : acc[c + i] + sum;
                    }
                }
                tmem_fence_before();
                __syncwarp();
                if (lane == 0) bar_arrive_even(sums_empty(half));
                if (++half == 2) { half = 0; half_phase ^= 1u; }
            }
            if (!ok) break;
            const long long m = (long long)mt * 256 + rank * 128 + quarter * 32 + lane;
            const int n0 = nt * BN + col0;
            if (m < p.M) {
                const float sx = p.x_scale[m];
                E* y = static_cast<E*>(p.y) + m * p.y_stride + n0;
                constexpr int V = 16 / sizeof(E);
#pragma unroll
                for (int c = 0; c < W; c += V) {
                    union { uint4 word; E e[V]; } o;
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const int n = n0 + c + i;
                        float v = 0.0f;
                        if (n < p.N) {
                            v = (float)acc[c + i] * sx * p.w_scale[n];
                            if (p.bias != nullptr) v += p.bias[n];
                        }
                        o.e[i] = out_value<E>(v);
                    }
                    if (p.wide && n0 + c + V <= p.N) {
                        *reinterpret_cast<uint4*>(y + c) = o.word;
                    } else {
#pragma unroll
                        for (int i = 0; i < V; ++i)
                            if (n0 + c + i < p.N) y[c + i] = o.e[i];
                    }
                }
            }
        }
    }
    __syncthreads();
    __syncwarp();
    cluster_sync();   // neither CTA leaves while the other may use its shared memory or TMEM
    if (warp == 2) {
        tmem_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(2 * BN) : "memory");
    }
}

int pieces_of(int v, int of) { return (int)(((long long)v + of - 1) / of); }

template <typename E, int BN>
int start_gemm(const GemmParams& q, cudaStream_t st) {
    GemmParams p = q;
    p.m_tiles = pieces_of(p.M, 256);
    p.n_tiles = pieces_of(p.N, BN);
    const long long tiles = (long long)p.m_tiles * p.n_tiles;
    if (tiles > (1LL << 30)) return TR_ERR_NOT_SUPPORTED;
    cudaLaunchConfig_t cfg{};
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmemBytes<BN>;
    cfg.stream = st;
    // the pairs of SMs that can run at once, asked for once
    static std::atomic<int> pairs{0};
    int n = pairs.load(std::memory_order_relaxed);
    if (n == 0) {
        cfg.gridDim = dim3(2);
        cudaError_t e = cudaFuncSetAttribute(gemm_kernel<E, BN>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes<BN>);
        if (e == cudaSuccess) e = cudaOccupancyMaxActiveClusters(&n, gemm_kernel<E, BN>, &cfg);
        if (e != cudaSuccess || n < 1) {
            set_last_error("int8 product kernel set-up", (int)e);
            return TR_ERR_CUDA;
        }
        pairs.store(n, std::memory_order_relaxed);
    }
    cfg.gridDim = dim3((unsigned)(2 * (tiles < n ? tiles : n)));
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, gemm_kernel<E, BN>, p);
    if (e != cudaSuccess) {
        set_last_error("cudaLaunchKernelEx(int8 product)", (int)e);
        return TR_ERR_CUDA;
    }
    return launched("int8 product kernel");
}

template <typename E>
int pick_gemm(const GemmParams& p, cudaStream_t st) {
    // the narrower tile where the wide one leaves pairs of SMs without any
    const long long wide = (long long)pieces_of(p.M, 256) * pieces_of(p.N, 256);
    return wide >= 76 ? start_gemm<E, 256>(p, st) : start_gemm<E, 128>(p, st);
}

}  // namespace

size_t int8_gemm_workspace(long long M, long long N, long long K) {
    const size_t kb = (size_t)((K + kBlockK - 1) / kBlockK);
    // whole tiles of 256 rows: the product reads them without looking at M and N
    return (size_t)((M + 255) / 256 + (N + 255) / 256) * 2 * kb * kBlockBytes;
}

int launch_int8_gemm(const MatmulArgs& a) {
    cudaStream_t st = static_cast<cudaStream_t>(a.stream);
    const int kb = pieces_of(a.K, kBlockK);
    CopyParams c;
    c.x = ByteRows{a.x, a.x_stride, a.x + (a.M - 1) * a.x_stride + a.K, a.M, a.K};
    c.w = ByteRows{a.w, a.w_stride, a.w + (a.N - 1) * a.w_stride + a.K, a.N, a.K};
    c.x_pieces = (long long)pieces_of(a.M, 256) * 2 * kb * (kBlockBytes / 32);
    c.w_pieces = (long long)pieces_of(a.N, 256) * 2 * kb * (kBlockBytes / 32);
    c.xh = static_cast<uint4*>(a.workspace);
    c.wh = c.xh + c.x_pieces * 2;
    c.k_blocks = kb;
    const bool on16 = (uintptr_t)a.x % 16 == 0 && (uintptr_t)a.w % 16 == 0 && a.x_stride % 16 == 0 && a.w_stride % 16 == 0;
    const long long ctas = (c.x_pieces + c.w_pieces + 255) / 256;
    const unsigned grid = (unsigned)(ctas < (1 << 30) ? ctas : (1 << 30));
    if (on16) copy_kernel<true><<<grid, 256, 0, st>>>(c);
    else copy_kernel<false><<<grid, 256, 0, st>>>(c);
    const int rc = launched("int8 copy kernel");
    if (rc != TR_OK) return rc;
    GemmParams p{};
    p.xh = reinterpret_cast<const uint8_t*>(c.xh);
    p.wh = reinterpret_cast<const uint8_t*>(c.wh);
    p.x_scale = a.x_scale;
    p.w_scale = a.w_scale;
    p.bias = a.bias;
    p.y = a.y;
    p.y_stride = a.y_stride;
    p.M = a.M; p.N = a.N; p.k_blocks = kb;
    const int es = a.out_dtype == TR_ELEM_F32 ? 4 : 2;
    p.wide = (uintptr_t)a.y % 16 == 0 && (a.y_stride * es) % 16 == 0;
    if (a.out_dtype == TR_ELEM_F32) return pick_gemm<float>(p, st);
    if (a.out_dtype == TR_ELEM_F16) return pick_gemm<__half>(p, st);
    return pick_gemm<__nv_bfloat16>(p, st);
}

int read_gemm_status(int* flags, bool clear) {
    unsigned v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_gemm_status, sizeof v);
    if (e == cudaSuccess && clear && v != 0) {
        const unsigned zero = 0;
        e = cudaMemcpyToSymbol(g_gemm_status, &zero, sizeof zero);
    }
    if (e != cudaSuccess) {
        set_last_error("tr_device_status (int8 product)", (int)e);
        return TR_ERR_CUDA;
    }
    *flags = (int)v;
    return TR_OK;
}

}  // namespace trfn
