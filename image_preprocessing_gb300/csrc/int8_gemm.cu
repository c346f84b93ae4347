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
//
// Measured: 12544 x 4096 x 4096 242 to 256 us, 1645 to 1740 TFLOP/s, by the clock
// that the power limit leaves; the copies are 34 of them (5.8 TB/s), the product
// alone runs at 1950 TFLOP/s, the rate of a plain binary16 product; 50176 x 1024 x
// 768 68 to 69 us, 21 of them copies; 50176 x 4096 x 1024 233 us, 1800 TFLOP/s;
// outputs off 16 bytes, 7168 x 8749 x 197, 54 us (93 with one row stored at a time).  Converting in the product's kernel instead would
// put half as much again through shared memory for each block; copying later
// tokens beside the product of the first measured slower (73 us).
#include <cuda.h>
#include <cudaTypedefs.h>

#include <atomic>
#include <climits>
#include <cmath>
#include <mutex>

#include "int8_parts.h"
#include "tensor_core.h"
#include "token_ops.h"

namespace trfn {
namespace {

constexpr int kBlockRows = 128, kBlockK = 64, kBlockBytes = kBlockRows * kBlockK * 2;
constexpr int kExactBlocks = 1024 / kBlockK;       // blocks of K summed in binary32
constexpr int kEpilogueWarps = 8;
constexpr int kThreads = 32 * (4 + kEpilogueWarps);

// ------------------------------------------------- PTX forms of the pair ---

// Arrives on the even CTA's barrier at this CTA's address `bar`.  Relaxed: what
// it reports is that TMEM has been read, which tcgen05.wait::ld and the tcgen05
// fence before it order; a release would wait for the thread's stores to y
// (measured: 4000 cycles a tile).
__device__ __forceinline__ void bar_arrive_even(uint32_t bar) {
    asm volatile(
        "{\n\t.reg .b32 a;\n\t"
        "mapa.shared::cluster.u32 a, %0, 0;\n\t"
        "mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [a];\n\t}" ::"r"(bar)
        : "memory");
}
// This CTA's address `bar` in the even CTA.
__device__ __forceinline__ uint32_t in_even(uint32_t bar) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"(bar));
    return a;
}
// Box of a tensor map at row `row`; the bytes count on `bar`, a barrier of
// either CTA of the pair.
__device__ __forceinline__ void tensor_load(uint32_t dst, const CUtensorMap* map, int row, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(map), "r"(0), "r"(row), "r"(bar)
        : "memory");
}
// Issued by the whole warp for its one elected thread: a branch around it would leave the compiler without
// the knowledge that its operands are the warp's (measured: 85 cycles a product instead of some).
__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t shape, uint32_t add) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(shape), "r"(add)
        : "memory");
}
// Arrives on `bar` of both CTAs when the products issued so far are done.
__device__ __forceinline__ void commit_both(uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(bar),
        "h"((uint16_t)3)
        : "memory");
}
// Barrier of the eight epilogue warps; whether any of them passed a true flag.
__device__ __forceinline__ bool epilogue_barrier(bool flag) {
    uint32_t any;
    asm volatile(
        "{\n\t.reg .pred q, p;\n\t"
        "setp.ne.u32 q, %1, 0;\n\t"
        "bar.red.or.pred p, 1, 256, q;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(any)
        : "r"((uint32_t)flag)
        : "memory");
    return any != 0;
}
// ---------------------------------------------------------------- copies ---

struct CopyParams {
    ByteRows x, w;
    uint4* xh;
    uint4* wh;
    unsigned x_blocks, blocks, k_blocks;   // blocks of x, of both, of a block row
};

// A CTA copies a block at a time, a thread 16 values of two of its rows: four
// threads a block row, eight rows a warp, so a warp writes a swizzle atom of
// 1 KB.  (One index division for a block: with one for each 16 values the
// instructions, not the bytes, are the bound.)
template <bool ON16>
__global__ void __launch_bounds__(256) copy_kernel(const CopyParams p) {
    // x and w may be of the kernel before this one in the stream, which may read the workspace
    asm volatile("griddepcontrol.wait;\n\tgriddepcontrol.launch_dependents;" ::: "memory");
    const int q = threadIdx.x & 3, r = threadIdx.x >> 2;
    for (unsigned i = blockIdx.x; i < p.blocks; i += gridDim.x) {
        const bool of_w = i >= p.x_blocks;
        const ByteRows m{of_w ? p.w.p : p.x.p, of_w ? p.w.stride : p.x.stride, of_w ? p.w.end : p.x.end,
                         of_w ? p.w.rows : p.x.rows, p.x.K};
        const unsigned block = of_w ? i - p.x_blocks : i, across = block / p.k_blocks;
        const int k = (int)(block - across * p.k_blocks) * kBlockK + q * 16;
        const long long row = (long long)across * kBlockRows + r;
        const int8_t* const at0 = m.p + row * m.stride;
        const int8_t* const at1 = at0 + 64 * m.stride;
        const bool in0 = row < m.rows, in1 = row + 64 < m.rows;
        Piece<ON16> p0, p1;
        if (in0) p0.fetch(m, at0, k);
        if (in1) p1.fetch(m, at1, k);
        uint4* line = (of_w ? p.wh : p.xh) + (long long)block * (kBlockBytes / 16) + r * 8;
        auto put = [&](uint4* to, const uint4& v) {
            uint4 a, b;
            int8_to_half(v.x, a.x, a.y);
            int8_to_half(v.y, a.z, a.w);
            int8_to_half(v.z, b.x, b.y);
            int8_to_half(v.w, b.z, b.w);
            to[(2 * q) ^ (r & 7)] = a;
            to[(2 * q + 1) ^ (r & 7)] = b;
        };
        put(line, in0 ? p0.value(m, at0, k, false) : make_uint4(0, 0, 0, 0));
        put(line + 64 * 8, in1 ? p1.value(m, at1, k, false) : make_uint4(0, 0, 0, 0));
    }
}

// --------------------------------------------------------------- product ---

struct GemmParams {
    CUtensorMap x, w;         // the copies: all block rows of 64 values, boxes of 128 and BN/2 rows
    const float* x_scale;
    const float* w_scale;
    const float* bias;
    void* y;
    long long y_stride;
    int M, N, k_blocks, m_tiles, n_tiles, wide;   // wide: rows of y take 16-byte stores
    int missing;                                  // test hook: arrivals that the first stage waits for in vain
    unsigned* status;                             // the product's status word
};

// Shared memory: the ring, 2 KB for each epilogue warp, (scale, bias) of two
// tiles' channels.
template <int BN> constexpr int kStageBytes = kBlockBytes + BN / 2 * 128;
template <int BN> constexpr int kStages = BN == 256 ? 6 : 8;
constexpr int kPassBytes = 64;   // of a row of y that pass through a warp's 2 KB at a time
template <int BN> constexpr int kSmemBytes =
    1024 + kStages<BN> * kStageBytes<BN> + kEpilogueWarps * 32 * kPassBytes + 2 * BN * 8;

// ONE: K <= 1024, one sum in TMEM for each value of y.
template <typename E, int BN, bool ONE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1) gemm_kernel(const __grid_constant__ GemmParams p) {
    constexpr int ST = kStages<BN>;
    extern __shared__ uint8_t smem_raw[];
    // full[ST] empty[ST] sums_full[2] sums_empty[2]
    __shared__ __align__(8) uint64_t bars[2 * ST + 4];
    __shared__ uint32_t tmem_at;
    __shared__ volatile int given_up;
    uint8_t* const base = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t ring = smem_u32(base);
    const uint32_t bar0 = smem_u32(bars);
    auto full = [&](int s) { return bar0 + 8u * s; };
    auto empty = [&](int s) { return bar0 + 8u * (ST + s); };
    auto sums_full = [&](int s) { return bar0 + 8u * (2 * ST + s); };
    auto sums_empty = [&](int s) { return bar0 + 8u * (2 * ST + 2 + s); };
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();

    if (threadIdx.x == 0) {
        given_up = 0;
        for (int s = 0; s < ST; ++s) {
            bar_init(full(s), s == 0 && blockIdx.x == 0 ? 1 + p.missing : 1);
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
    const int parts = ONE ? 1 : (p.k_blocks + kExactBlocks - 1) / kExactBlocks;

    if (warp == 0) {
        if (lane == 0) {
            asm volatile("griddepcontrol.wait;" ::: "memory");   // the copies are made by the kernel before
            int s = 0, issued = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int tile = pair; tile < tiles && ok; tile += pairs) {
                const int mt = tile / p.n_tiles, nt = tile % p.n_tiles;
                const int xb = (mt * 2 + (int)rank) * p.k_blocks;
                // this CTA's BN/2 channels: a block, or half of one
                const int ch = nt * BN + (int)rank * (BN / 2);
                const int wb = (ch >> 7) * p.k_blocks, sub = ch & 127;
                for (int kb = 0; kb < p.k_blocks; ++kb) {
                    if (!bar_wait(empty(s), phase ^ 1u, &given_up, p.status)) { ok = false; break; }
                    const uint32_t at = ring + s * kStageBytes<BN>;
                    // both CTAs' bytes count on the even one's barrier
                    if (rank == 0) bar_expect(full(s), 2 * kStageBytes<BN>);
                    tensor_load(at, &p.x, (xb + kb) * kBlockRows, in_even(full(s)));
                    tensor_load(at + kBlockBytes, &p.w, (wb + kb) * kBlockRows + sub, in_even(full(s)));
                    issued = issued < ST ? issued + 1 : ST;
                    if (++s == ST) { s = 0; phase ^= 1u; }
                }
            }
            // copies in flight land before the pair ends, whatever became of the others (in a run that gave
            // up, the odd CTA's may be counted nowhere: it leaves them a thousand times their duration)
            if (rank != 0 && !ok) __nanosleep(1000000);
            if (rank == 0)
                for (int i = 0; i < issued; ++i) {
                    s = s == 0 ? ST - 1 : s - 1;
                    if (s == ST - 1) phase ^= 1u;
                    bar_drain(full(s), phase);
                }
        }
    } else if (warp == 1 && rank == 0) {
        // the waits for copies are limited from here on, not from when the kernel that makes them still runs
        asm volatile("griddepcontrol.wait;" ::: "memory");
        constexpr uint32_t shape = (1u << 4) | ((uint32_t)(BN / 8) << 17) | (16u << 24);   // f16 x f16 -> f32, 256 x BN
        const uint64_t x0 = operand(ring), w0 = operand(ring + kBlockBytes);
        int s = 0, half = 0;
        uint32_t phase = 0, half_phase = 0;
        uint32_t last = 0, last_phase = 0;   // the stage whose products were issued last
        bool ok = true;
        for (int tile = pair; tile < tiles && ok; tile += pairs) {
            for (int part = 0; part < parts && ok; ++part) {
                ok = __all_sync(0xffffffffu, bar_wait(sums_empty(half), half_phase ^ 1u, &given_up, p.status));
                if (!ok) break;
                tmem_fence_after();
                const uint32_t d = tmem + half * BN;
                const int kb0 = part * kExactBlocks, kb1 = min(p.k_blocks, kb0 + kExactBlocks);
                for (int kb = kb0; kb < kb1; ++kb) {
                    ok = __all_sync(0xffffffffu, bar_wait(full(s), phase, &given_up, p.status));
                    if (!ok) break;
                    tmem_fence_after();
                    const uint32_t at = s * (kStageBytes<BN> / 16);   // descriptors count in 16 bytes
#pragma unroll
                    for (int k = 0; k < kBlockK / 16; ++k)
                        mma_pair(d, x0 + at + 2 * k, w0 + at + 2 * k, shape, kb > kb0 || k > 0);
                    commit_both(empty(s));
                    last = empty(s);
                    last_phase = phase;
                    if (++s == ST) { s = 0; phase ^= 1u; }
                }
                if (!ok) break;   // these sums are not whole: nobody gets them
                commit_both(sums_full(half));
                if (++half == 2) { half = 0; half_phase ^= 1u; }
            }
        }
        if (last != 0) bar_drain(last, last_phase);   // the last products are done before TMEM is freed
        __syncwarp();
    } else if (warp >= 4) {
        constexpr int W = BN / 2;                      // channels of a warp
        constexpr int V = 16 / sizeof(E), C = kPassBytes / sizeof(E);   // channels of 16 bytes, of a pass
        const int quarter = warp & 3, col0 = (warp - 4) / 4 * W, me = threadIdx.x - 128;
        uint8_t* const pass = base + ST * kStageBytes<BN> + (warp - 4) * 32 * kPassBytes;
        float2* const channel = reinterpret_cast<float2*>(base + ST * kStageBytes<BN> + kEpilogueWarps * 32 * kPassBytes);
        // a thread's row scale, and its channel's (scale, bias), loaded a tile ahead
        struct Scales { float sx; float2 channel; };
        auto scales_of = [&](int tile) {
            Scales v{0.0f, make_float2(0.0f, 0.0f)};
            if (tile >= tiles) return v;
            const int m = tile / p.n_tiles * 256 + (int)rank * 128 + quarter * 32 + lane, n = tile % p.n_tiles * BN + me;
            if (m < p.M) v.sx = p.x_scale[m];
            if (me < BN && n < p.N) v.channel = make_float2(p.w_scale[n], p.bias != nullptr ? p.bias[n] : 0.0f);
            return v;
        };
        // the scales, and what reads y, may be of kernels before the copies, which have waited for them
        asm volatile("griddepcontrol.wait;" ::: "memory");
        Scales ahead = scales_of(pair);
        int half = 0, buf = 0;
        uint32_t half_phase = 0;
        bool ok = true;
        for (int tile = pair; tile < tiles; tile += pairs) {
            const int mt = tile / p.n_tiles, nt = tile % p.n_tiles;
            // scale and bias of the tile's channels; the other buffer may still be in use
            buf ^= 1;
            if (me < BN) channel[buf * BN + me] = ahead.channel;
            const int m0 = mt * 256 + (int)rank * 128 + quarter * 32;
            const float sx = ahead.sx;
            if (epilogue_barrier(!ok)) break;
            ahead = scales_of(tile + pairs);
            int acc[ONE ? 1 : W];
            for (int part = 0; part < parts - 1; ++part) {
                ok = __all_sync(0xffffffffu, bar_wait(sums_full(half), half_phase, &given_up, p.status));
                if (!ok) break;
                tmem_fence_after();
                const uint32_t at = tmem + half * BN + col0 + ((uint32_t)(quarter * 32) << 16);
                if constexpr (!ONE) {
#pragma unroll
                    for (int c = 0; c < W; c += 16) {
                        uint32_t v[16];
                        tmem_load16(at + c, v);
                        tmem_wait(v);
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const int sum = __float2int_rn(__uint_as_float(v[i]));
                            acc[c + i] = part == 0 ? sum : acc[c + i] + sum;
                        }
                    }
                }
                tmem_fence_before();
                __syncwarp();
                if (lane == 0) bar_arrive_even(sums_empty(half));
                if (++half == 2) { half = 0; half_phase ^= 1u; }
            }
            if (ok) ok = __all_sync(0xffffffffu, bar_wait(sums_full(half), half_phase, &given_up, p.status));
            if (!ok) continue;   // to the barrier, where all eight warps leave together
            tmem_fence_after();
            const uint32_t at = tmem + half * BN + col0 + ((uint32_t)(quarter * 32) << 16);
            const int n0 = nt * BN + col0;
            // G columns at a time; with registers to spare, the next are on their way meanwhile
            constexpr int G = ONE ? 32 : 16;
            uint32_t v[G], next[G];
            auto fetch = [&](int c, uint32_t (&to)[G]) {
                tmem_load16(at + c, to);
                if constexpr (ONE) tmem_load16(at + c + 16, to + 16);
            };
            if (ONE) fetch(0, next);
#pragma unroll
            for (int c = 0; c < W; c += G) {
                if (!ONE) fetch(c, next);
                tmem_wait(next);
#pragma unroll
                for (int i = 0; i < G; ++i) v[i] = next[i];
                if (ONE && c + G < W) fetch(c + G, next);
                if (c + G == W) {   // TMEM is read: the next sums may go there
                    tmem_fence_before();
                    __syncwarp();
                    if (lane == 0) bar_arrive_even(sums_empty(half));
                    if (++half == 2) { half = 0; half_phase ^= 1u; }
                }
                // through the warp's 2 KB, 64 bytes of each row at a time, so that rows of y are written in
                // 64-byte runs; piece q of row r lies at q ^ (r >> 1 & 3): no bank conflicts
#pragma unroll
                for (int i = 0; i < G; i += V) {
                    union { uint4 word; E e[V]; } o;
#pragma unroll
                    for (int j = 0; j < V; j += 2) {
                        const float4 two = *reinterpret_cast<const float4*>(&channel[buf * BN + col0 + c + i + j]);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            float sum = __uint_as_float(v[i + j + h]);
                            if constexpr (!ONE)
                                if (parts > 1) sum = (float)(acc[c + i + j + h] + __float2int_rn(sum));
                            o.e[j + h] = out_value<E>(sum * sx * (h ? two.z : two.x) + (h ? two.w : two.y));
                        }
                    }
                    const int q = (c + i) % C / V;
                    *reinterpret_cast<uint4*>(pass + lane * 64 + ((q ^ (lane >> 1)) & 3) * 16) = o.word;
                    if ((c + i + V) % C != 0) continue;
                    __syncwarp();
                    const int n = n0 + c + i + V - C;
                    E* y = static_cast<E*>(p.y) + (long long)m0 * p.y_stride + n;
                    if (p.wide && n + C <= p.N) {
#pragma unroll
                        for (int d = 0; d < 4; ++d) {
                            const int r = d * 8 + (lane >> 2), part_q = lane & 3;
                            const uint4 w = *reinterpret_cast<const uint4*>(pass + r * 64 + ((part_q ^ (r >> 1)) & 3) * 16);
                            if (m0 + r < p.M) *reinterpret_cast<uint4*>(y + r * p.y_stride + part_q * V) = w;
                        }
                    } else {
                        // rows off 16 bytes: R rows of C values at a time, eight reads before the writes
                        constexpr int R = 32 / C;
                        const int e = lane % C, part_q = e / V;
                        const bool in = n + e < p.N;
#pragma unroll
                        for (int r0 = 0; r0 < 32; r0 += 8 * R) {
                            E w[8];
#pragma unroll
                            for (int u = 0; u < 8; ++u) {
                                const int r = r0 + u * R + lane / C;
                                w[u] = *(reinterpret_cast<const E*>(pass + r * 64 + ((part_q ^ (r >> 1)) & 3) * 16) + e % V);
                            }
                            E* yr = y + (long long)(r0 + lane / C) * p.y_stride + e;
#pragma unroll
                            for (int u = 0; u < 8; ++u) {
                                if (in && m0 + r0 + u * R + lane / C < p.M) *yr = w[u];
                                yr += R * p.y_stride;
                            }
                        }
                    }
                    __syncwarp();
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

// `rows` block rows of 64 binary16 at `p`, boxes of `box` of them.
int block_map(CUtensorMap* map, void* p, long long rows, int box) {
    static PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* fn = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    });
    if (encode == nullptr) return cuda_failed("cuTensorMapEncodeTiled unavailable", (int)cudaErrorNotSupported);
    const cuuint64_t dims[2] = {kBlockK, (cuuint64_t)rows}, strides[1] = {kBlockK * 2};
    const cuuint32_t boxes[2] = {kBlockK, (cuuint32_t)box}, elem[2] = {1, 1};
    const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, p, dims, strides, boxes, elem,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return cuda_failed("cuTensorMapEncodeTiled", (int)cudaErrorInvalidValue);
    return TR_OK;
}

struct Copies {
    void* xh;
    void* wh;
    long long x_rows, w_rows;   // block rows: 64 values each
};

template <typename E, int BN, bool ONE>
int start_gemm(const GemmParams& q, const Copies& c, cudaStream_t st) {
    GemmParams p = q;
    p.m_tiles = pieces_of(p.M, 256);
    p.n_tiles = pieces_of(p.N, BN);
    int rc = block_map(&p.x, c.xh, c.x_rows, kBlockRows);
    if (rc == TR_OK) rc = block_map(&p.w, c.wh, c.w_rows, BN / 2);
    if (rc != TR_OK) return rc;
    const long long tiles = (long long)p.m_tiles * p.n_tiles;
    if (tiles > (1LL << 30)) return TR_ERR_NOT_SUPPORTED;
    cudaLaunchConfig_t cfg{};
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmemBytes<BN>;
    cfg.stream = st;
    // the pairs of SMs that can run at once, asked for once on each device
    static std::atomic<int> known[kMaxDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || dev < 0 || dev >= kMaxDevices) return cuda_failed("cudaGetDevice", (int)e);
    rc = product_status_word(dev, &p.status);
    if (rc != TR_OK) return rc;
    std::atomic<int>& pairs = known[dev];
    int n = pairs.load(std::memory_order_relaxed);
    if (n == 0) {
        cfg.gridDim = dim3(2);
        e = cudaFuncSetAttribute(gemm_kernel<E, BN, ONE>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes<BN>);
        if (e == cudaSuccess) e = cudaOccupancyMaxActiveClusters(&n, gemm_kernel<E, BN, ONE>, &cfg);
        if (e != cudaSuccess || n < 1) return cuda_failed("int8 product kernel set-up", (int)e);
        pairs.store(n, std::memory_order_relaxed);
    }
    cfg.gridDim = dim3((unsigned)(2 * (tiles < n ? tiles : n)));
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return launched("int8 product kernel", (int)cudaLaunchKernelEx(&cfg, gemm_kernel<E, BN, ONE>, p));
}

template <typename E, int BN>
int pick_parts(const GemmParams& p, const Copies& c, cudaStream_t st) {
    return p.k_blocks <= kExactBlocks ? start_gemm<E, BN, true>(p, c, st) : start_gemm<E, BN, false>(p, c, st);
}

// Cycles of the product with tiles of BN channels, for a block of K: one wave of pairs takes 512 cycles of the
// tensor cores (BN = 256) or, bound by loading, 340 (BN = 128; 256 by the tensor cores).
double wave_cycles(long long M, long long N, int BN) {
    return std::ceil(std::ceil(M / 256.0) * std::ceil((double)N / BN) / 76) * (BN == 256 ? 512 : 340);
}

template <typename E>
int pick_gemm(const GemmParams& p, const Copies& c, cudaStream_t st) {
    return wave_cycles(p.M, p.N, 256) <= wave_cycles(p.M, p.N, 128) ? pick_parts<E, 256>(p, c, st) : pick_parts<E, 128>(p, c, st);
}

}  // namespace

size_t int8_gemm_workspace(long long M, long long N, long long K) {
    const size_t kb = (size_t)((K + kBlockK - 1) / kBlockK);
    // whole tiles of 256 rows: the product reads them without looking at M and N
    return (size_t)((M + 255) / 256 + (N + 255) / 256) * 2 * kb * kBlockBytes;
}

// Start of two kernels, the copies' bytes (read one, write two) at 2850 a cycle, and the product.
double int8_gemm_cycles(long long M, long long N, long long K) {
    return 9500 + 3.0 * (double)(M + N) * (double)K / 2850 +
           std::ceil((double)K / kBlockK) * std::fmin(wave_cycles(M, N, 256), wave_cycles(M, N, 128));
}

int launch_int8_gemm(const MatmulArgs& a) {
    cudaStream_t st = static_cast<cudaStream_t>(a.stream);
    const int kb = pieces_of(a.K, kBlockK);
    CopyParams c;
    c.x = ByteRows{a.x, a.x_stride, a.x + (a.M - 1) * a.x_stride + a.K, a.M, a.K};
    c.w = ByteRows{a.w, a.w_stride, a.w + (a.N - 1) * a.w_stride + a.K, a.N, a.K};
    const long long x_blocks = (long long)pieces_of(a.M, 256) * 2 * kb, w_blocks = (long long)pieces_of(a.N, 256) * 2 * kb;
    if ((x_blocks + w_blocks) * kBlockRows > INT_MAX) return TR_ERR_NOT_SUPPORTED;   // rows of a tensor map
    c.x_blocks = (unsigned)x_blocks;
    c.blocks = (unsigned)(x_blocks + w_blocks);
    c.k_blocks = (unsigned)kb;
    c.xh = static_cast<uint4*>(a.workspace);
    c.wh = c.xh + x_blocks * (kBlockBytes / 16);
    const bool on16 = rows_on16(a.x, a.x_stride, a.M) && rows_on16(a.w, a.w_stride, a.N);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(c.blocks);
    cfg.blockDim = dim3(256);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];   // its CTAs may be set up while the kernel before ends
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const int rc = launched("int8 copy kernel", (int)cudaLaunchKernelEx(&cfg, on16 ? copy_kernel<true> : copy_kernel<false>, c));
    if (rc != TR_OK) return rc;
    const Copies copies{c.xh, c.wh, x_blocks * kBlockRows, w_blocks * kBlockRows};
    GemmParams p{};
    p.x_scale = a.x_scale;
    p.w_scale = a.w_scale;
    p.bias = a.bias;
    p.y = a.y;
    p.y_stride = a.y_stride;
    p.M = a.M; p.N = a.N; p.k_blocks = kb;
    p.missing = test_waits();
    const int es = a.out_dtype == TR_ELEM_F32 ? 4 : 2;
    p.wide = (uintptr_t)a.y % 16 == 0 && (a.y_stride * es) % 16 == 0;
    if (a.out_dtype == TR_ELEM_F32) return pick_gemm<float>(p, copies, st);
    if (a.out_dtype == TR_ELEM_F16) return pick_gemm<__half>(p, copies, st);
    return pick_gemm<__nv_bfloat16>(p, copies, st);
}

}  // namespace trfn
