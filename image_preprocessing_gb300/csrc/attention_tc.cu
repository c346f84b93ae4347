// Attention on the tensor cores: binary16 and bfloat16, heads of up to 128 values
// on 16-byte boundaries (attention.cu has the mathematics and the plain kernel).
//
// A CTA on each SM goes through its share of the work (attention_plan.h).  An item
// is two tiles of 128 rows (queries x heads of one key head) over blocks of 128
// keys.  Warps: one copies (TMA: queries, then keys and values through a ring of
// stages) and says what comes next; one issues the products; one makes values that
// a row does not see harmless; four for each tile do the softmax, a thread a row.
//     S = Q K^T into TMEM; a row's thread reads it, keeps maximum and sum, writes
//     P = 2^(x - m) in 16 bits over S; O += P V in TMEM, P read from there.
// The tiles take turns: the tensor cores multiply for one while the other's
// weights are made.  O is multiplied by 2^(m_old - m_new) only where the maximum
// has grown by more than 8 (2^8 more in P is no loss: the sum is binary32); the
// thread does that itself, so there is no correction in the usual block.
//
// P is rounded to the type of v, half a unit relative to itself, as the products
// take it, and l is the sum of what they take: where one key has nearly all the
// weight, its rounding is no error (costs 2 %).  In binary16 the weights are made
// 2^6 times as large, so that the ones below 2^-14 of the largest keep more of
// their bits.
//
// What a row does not see: its weight is an exact zero, but 0 times an infinity is
// not.  In blocks that some row does not see whole, values that are not finite are
// replaced by zeros in shared memory, and a tile that meets such a block adds them
// at the end to the rows that do see them.  Keys need no care: their scores are
// replaced.
//
// A share that begins or ends inside an item leaves its sums, maxima and outputs
// in the workspace, and a second kernel joins them in the order of the keys.
//
// What bounds it: the way of one block through a tile (scores 800 cycles until the
// last is visible, weights some 1500, the products with v and the handing over)
// is longer than the 2048 cycles that the tensor cores need for both tiles' block
// at 128 values a head, and twice their time at 64.  Measured: 8192 causal queries,
// 32 heads of 128 over 8 key heads, bfloat16, 510 us, 1077 TFLOP/s (0.56 of the
// measured peak; the tensor pipe active 53 % of the cycles); 16 packed prompts of up to
// 4096 306 us (0.41); 256 x 196, 12 heads of 64, binary16, 147 us (0.31 of the copy
// rate); one token for each of 32 sequences over 42,000 keys in all 58 us (0.44 of
// the copy rate; even lengths of 4096 113 us, 0.70).
//
// Shared memory leaves L1 a few KB, so whatever a thread keeps in local memory
// comes from L2 each time: a kernel that spilled a few hundred bytes took five
// times as long.  No role has a stack frame.  Tried and slower: two threads a row
// (149 us for 138 at 4096 x 4096, 16 heads of 128), P in two halves with the
// products of the first beside the weights of the second (+ 10 %), rows through
// shared memory into bulk copies at the end (+ 7 %), P beside S for heads of 64 with
// the next scores early (163 us for 139 at 256 x 196).
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>
#include <cmath>
#include <mutex>
#include <type_traits>

#include "attention_parts.h"
#include "f32_pairs.h"
#include "tensor_core.h"

namespace trfn {
namespace {

using attention::Border;
using attention::kKeys;
using attention::kRows;

constexpr int kCtas = 152;                    // one on each SM
constexpr int kSoftmaxWarps = 8, kThreads = 32 * (4 + kSoftmaxWarps);
constexpr int kPieces = 8, kFlags = 16;       // descriptors on their way; items whose values may be under way
constexpr int kBoxRows = 64;                  // keys to a copy
constexpr float kGrowth = 8.0f;               // of a maximum, in powers of two, before O is multiplied

// What a CTA does of one item, as the copying warp tells the others.
struct Piece {
    int q0, tokens;      // its first query's row, and queries
    int head;            // key head
    int k0, keys;        // the sequence's first key's row, and keys
    int base;            // keys that its first query sees (before the bounds); causal: one more for each query
    int j0, j1;          // blocks of this piece; j0 < 0: nothing follows
    int slot;            // partial result, or -1
    int end0, end1;      // where the tiles' blocks end, up to j1
    int least;           // keys that its first query sees
    int seen0, seen1;    // keys that the tiles' last queries see
    int pad[2];
};
static_assert(sizeof(Piece) == 64, "pieces of the workspace and of shared memory");

// A partial result in the workspace.
struct Slot {
    int state;           // 0 (none), kFirst (of an item) or kNext; kFailed is added by a CTA that gave up
    int ends;            // the item's last
    int q0, tokens, head, keys, base, pad;
};
constexpr int kFirst = 1, kNext = 2, kFailed = 4;

struct TcParams {
    CUtensorMap q, k, v;
    Sequences seq;
    void* out;
    const void* values;       // v, for values that are not finite
    long long out_stride, v_stride;
    int kv_heads, group, dim, tokens;   // tokens: queries of a tile
    float scale;              // with log2(e), positive
    bool causal;
    Slot* slots;              // 2 kCtas
    float2* stats;            // 2 kCtas x slot_rows: maximum, sum
    float* parts;             // 2 kCtas x slot_rows x D
    int slot_rows;
    const Border* borders;    // kCtas + 1
    int missing;              // test hook: arrivals that the first stage waits for in vain
    unsigned* status;
};

// ------------------------------------------------------------- PTX forms ---

__device__ __forceinline__ void box_load(uint32_t dst, const CUtensorMap* map, int c, int head, int row, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(map), "r"(c), "r"(head), "r"(row), "r"(bar)
        : "memory");
}
// Four products, 64 values of K, issued by the whole warp for its one elected thread: as one piece of PTX, whose
// operands are made once (four pieces, each with an election and operands of its own, kept the tensor cores waiting
// where other warps were busy: 145 cycles a product for 64).
__device__ __forceinline__ void mma4_shared(uint32_t d, uint64_t a, uint64_t b, uint32_t shape, uint32_t add) {
    asm volatile(
        "{\n"
        "\t.reg .pred p, e, t;\n"
        "\t.reg .b64 a, b;\n"
        "\telect.sync _|e, 0xffffffff;\n"
        "\tsetp.ne.b32 p, %4, 0;\n"
        "\tsetp.eq.b32 t, 0, 0;\n"
        "\tadd.s64 a, %1, 0;\n"
        "\tadd.s64 b, %2, 0;\n"
        "\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n"
        "\tadd.s64 a, %1, 2;\n"
        "\tadd.s64 b, %2, 2;\n"
        "\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n"
        "\tadd.s64 a, %1, 4;\n"
        "\tadd.s64 b, %2, 4;\n"
        "\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n"
        "\tadd.s64 a, %1, 6;\n"
        "\tadd.s64 b, %2, 6;\n"
        "\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n"
        "}\n"::"r"(d), "l"(a), "l"(b), "r"(shape), "r"(add)
        : "memory");
}
// A in TMEM, two 16-bit values to a column; B's rows along K, 2 KB to 16 of them.
__device__ __forceinline__ void mma4_tmem(uint32_t d, uint32_t a, uint64_t b, uint32_t shape, uint32_t add) {
    asm volatile(
        "{\n"
        "\t.reg .pred p, e, t;\n"
        "\t.reg .b64 b;\n"
        "\t.reg .b32 a;\n"
        "\telect.sync _|e, 0xffffffff;\n"
        "\tsetp.ne.b32 p, %4, 0;\n"
        "\tsetp.eq.b32 t, 0, 0;\n"
        "\tadd.s32 a, %1, 0;\n"
        "\tadd.s64 b, %2, 0;\n"
        "\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, p;\n"
        "\tadd.s32 a, %1, 8;\n"
        "\tadd.s64 b, %2, 128;\n"
        "\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n"
        "\tadd.s32 a, %1, 16;\n"
        "\tadd.s64 b, %2, 256;\n"
        "\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n"
        "\tadd.s32 a, %1, 24;\n"
        "\tadd.s64 b, %2, 384;\n"
        "\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n"
        "}\n"::"r"(d), "r"(a), "l"(b), "r"(shape), "r"(add)
        : "memory");
}
// One such product.
__device__ __forceinline__ void mma_tmem(uint32_t d, uint32_t a, uint64_t b, uint32_t shape, uint32_t add) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(shape), "r"(add)
        : "memory");
}
__device__ __forceinline__ void commit(uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
        : "memory");
}
__device__ __forceinline__ void arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// Values of rows along K (shared memory: 64 of them to a row of 128 bytes, swizzled; 16 KB between
// the next 64, 1 KB between groups of 8 rows): the matrix is read transposed.
__device__ __forceinline__ uint64_t operand_across(uint32_t addr, uint32_t apart) {
    return (uint64_t)((addr >> 4) & 0x3FFF) | ((uint64_t)(apart >> 4) << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}
__device__ __forceinline__ void tmem_load32(uint32_t addr, uint32_t* v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]), "=r"(v[9]),
          "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]), "=r"(v[17]), "=r"(v[18]),
          "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]),
          "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(addr));
}
__device__ __forceinline__ void tmem_store16(uint32_t addr, const uint32_t* v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]),
        "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}
__device__ __forceinline__ void tmem_stored() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ float power2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

template <typename E> __device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <> __device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
template <> __device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
// Not 0 where one of the two values is not finite: x * 0 is then NaN.
template <typename E> __device__ __forceinline__ uint32_t not_finite2(uint32_t x);
template <> __device__ __forceinline__ uint32_t not_finite2<__half>(uint32_t x) {
    const __half2 v = __hmul2(*reinterpret_cast<const __half2*>(&x), __half2half2(__ushort_as_half(0)));
    return *reinterpret_cast<const uint32_t*>(&v) & 0x7fff7fffu;
}
template <> __device__ __forceinline__ uint32_t not_finite2<__nv_bfloat16>(uint32_t x) {
    const __nv_bfloat162 v = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&x), __bfloat162bfloat162(__ushort_as_bfloat16(0)));
    return *reinterpret_cast<const uint32_t*>(&v) & 0x7fff7fffu;
}
__device__ __forceinline__ float value_of(__half v) { return __half2float(v); }
__device__ __forceinline__ float value_of(__nv_bfloat16 v) { return __bfloat162float(v); }

// Adds both rounded values to binary32 sums.
template <typename E> __device__ __forceinline__ void add_rounded(uint32_t w, float& lo, float& hi);
template <> __device__ __forceinline__ void add_rounded<__half>(uint32_t w, float& lo, float& hi) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tadd.f32.f16 %0, a, %0;\n\tadd.f32.f16 %1, b, %1;\n\t}" : "+f"(lo), "+f"(hi) : "r"(w));
}
template <> __device__ __forceinline__ void add_rounded<__nv_bfloat16>(uint32_t w, float& lo, float& hi) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tadd.f32.bf16 %0, a, %0;\n\tadd.f32.bf16 %1, b, %1;\n\t}" : "+f"(lo), "+f"(hi) : "r"(w));
}
template <typename E> __device__ __forceinline__ E from_value(float v);
template <> __device__ __forceinline__ __half from_value<__half>(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 from_value<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// bar_wait (tensor_core.h) without its call: what a call keeps in local memory would be fetched from L2 after every
// wait, as shared memory leaves no room for it in L1.
__device__ __forceinline__ bool bar_wait_here(uint32_t bar, uint32_t parity, volatile int* given_up, unsigned* status) {
    if (bar_try(bar, parity)) return true;
    uint32_t t0 = 0;
    for (uint32_t i = 1; i < (1u << 28); ++i) {
        if (bar_try(bar, parity)) return true;
        if ((i & 255u) != 0) continue;
        if (*given_up) return false;
        const uint32_t now = (uint32_t)(now_ns() >> 10);   // about microseconds
        if (t0 == 0) t0 = now | 1u;
        else if (now - t0 > (uint32_t)(kWaitLimitNs >> 10)) break;
    }
    *given_up = 1;
    atomicOr(status, kStatusTimeout);
    return false;
}

// The exponent of the type is all ones: one value.
template <typename E> constexpr uint32_t kExponent = 0x7c00;
template <> constexpr uint32_t kExponent<__nv_bfloat16> = 0x7f80;
// Powers of two by which weights are made larger.
template <typename E> constexpr float kLift = 6.0f;
template <> constexpr float kLift<__nv_bfloat16> = 0.0f;

// ------------------------------------------------------------- the layout ---

// Shared memory, D = 64 or 128: queries of two tiles (kQ of them), the ring.
template <int D> constexpr int kTileBytes = kRows * D * 2;    // of queries, of a block of keys or values
template <int D> constexpr int kQ = D == 64 ? 2 : 1;
template <int D> constexpr int kStages = D == 64 ? 10 : 5;
template <int D> constexpr int kSmem = 1024 + kQ<D> * 2 * kTileBytes<D> + kStages<D> * kTileBytes<D>;

__device__ __forceinline__ int seen_by(const Piece& p, bool causal, int token) {
    if (!causal) return p.keys;
    const long long n = (long long)p.base + token;
    return (int)max(0LL, min(n, (long long)p.keys));
}
// Whether some row of an item, whose first query sees `least` keys, does not see the whole of block j.
__device__ __forceinline__ bool masked(int least, int j) { return (least >> 7) <= j; }
static_assert(kKeys == 128, "blocks are counted by a shift");

// ---------------------------------------------------------------- the plan ---

// The borders of all CTAs' shares, by one CTA: in the kernel that works by them each CTA would make its own, and
// the registers of that would be the products' (measured: 134 -> 166 us at 4096 x 4096, 16 x 128).
struct PlanParams {
    Sequences seq;
    Border* borders;   // kCtas + 1
    int kv_heads, tokens;
    bool causal;
};
constexpr int kPlanThreads = 256;

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const PlanParams p) {
    __shared__ long long upto[kPlanThreads], warps[kPlanThreads / 32];   // units of the chunk's sequences, up to each
    asm volatile("griddepcontrol.wait;\n\tgriddepcontrol.launch_dependents;" ::: "memory");
    const int n = p.seq.count, t = threadIdx.x;
    auto sequence = [&](int s) {
        return attention::Sequence{range_of(p.seq.q_starts, p.seq.q_lengths, s, p.seq.q_rows).length,
                                   range_of(p.seq.k_starts, p.seq.k_lengths, s, p.seq.k_rows).length, p.tokens, p.causal};
    };
    auto scan = [&](long long v) {   // leaves the sums in upto
        const int lane = t & 31;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long left = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += left;
        }
        __syncthreads();   // the last chunk's sums have been read
        if (lane == 31) warps[t >> 5] = v;
        __syncthreads();
        for (int w = 0; w < (t >> 5); ++w) v += warps[w];
        upto[t] = v;
        __syncthreads();
    };
    long long mine = 0;
    for (int s = t; s < n; s += kPlanThreads) mine += sequence(s).head_units() * p.kv_heads;
    scan(mine);
    const long long units = upto[kPlanThreads - 1];
    // at least two units to a CTA
    const int parts = (int)max(1LL, min((long long)kCtas, units / 2));
    const long long want = attention::share_start(units, parts, min(t, parts));
    if (t <= kCtas && want >= units) p.borders[t] = Border{units, n, 0, 0, 0};
    long long before = 0;
    for (int s0 = 0; s0 < n && before < units; s0 += kPlanThreads) {
        if (n > kPlanThreads) scan(s0 + t < n ? sequence(s0 + t).head_units() * p.kv_heads : 0);
        const long long all = upto[kPlanThreads - 1];
        if (t <= kCtas && want >= before && want < before + all) {
            // the first sequence that ends after it
            int lo = 0, hi = kPlanThreads - 1;
            while (lo < hi) {
                const int mid = (lo + hi) / 2;
                if (before + upto[mid] > want) hi = mid;
                else lo = mid + 1;
            }
            p.borders[t] = attention::border_in(sequence(s0 + lo), s0 + lo, p.kv_heads, before + (lo > 0 ? upto[lo - 1] : 0), want, units, parts);
        }
        before += all;
    }
}
static_assert(kCtas < kPlanThreads, "a thread for each border");

// ------------------------------------------------------------- the kernel ---

template <typename E, int D>
__global__ void __launch_bounds__(kThreads, 1) attention_kernel(const __grid_constant__ TcParams p) {
    constexpr int ST = kStages<D>, NQ = kQ<D>, COLS = D / 64;
    constexpr uint32_t kTypes = sizeof(E) == 2 && kExponent<E> == 0x7f80 ? (1u << 7) | (1u << 10) : 0u;
    constexpr uint32_t kShape = (1u << 4) | kTypes | ((kRows / 16) << 24);   // binary32 sums, 128 rows
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(16) Piece pieces[kPieces];
    __shared__ __align__(8) uint64_t bars[3 * ST + 2 * NQ + 2 * kPieces + 6];
    __shared__ uint32_t tmem_at;
    __shared__ volatile int given_up;
    __shared__ volatile int not_finite[kFlags];   // the item (by number of pieces) in whose masked blocks values were replaced
    uint8_t* const base = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t queries = smem_u32(base), ring = queries + NQ * 2 * kTileBytes<D>;
    const uint32_t bar0 = smem_u32(bars);
    auto full = [&](int s) { return bar0 + 8u * s; };
    auto empty = [&](int s) { return bar0 + 8u * (ST + s); };
    auto q_full = [&](int s) { return bar0 + 8u * (2 * ST + s); };
    auto q_empty = [&](int s) { return bar0 + 8u * (2 * ST + NQ + s); };
    auto piece_full = [&](int s) { return bar0 + 8u * (2 * ST + 2 * NQ + s); };
    auto piece_empty = [&](int s) { return bar0 + 8u * (2 * ST + 2 * NQ + kPieces + s); };
    auto scores = [&](int t) { return bar0 + 8u * (2 * ST + 2 * NQ + 2 * kPieces + t); };       // S of tile t is there
    auto weights = [&](int t) { return bar0 + 8u * (2 * ST + 2 * NQ + 2 * kPieces + 2 + t); };  // P of tile t is there
    auto summed = [&](int t) { return bar0 + 8u * (2 * ST + 2 * NQ + 2 * kPieces + 4 + t); };   // P V is in O of tile t
    auto clean = [&](int s) { return bar0 + 8u * (2 * ST + 2 * NQ + 2 * kPieces + 6 + s); };    // values of masked blocks are finite
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        given_up = 0;
        for (int s = 0; s < ST; ++s) {
            bar_init(full(s), s == 0 && blockIdx.x == 0 ? 1 + p.missing : 1);
            bar_init(empty(s), 1);
            bar_init(clean(s), 1);
        }
        for (int s = 0; s < NQ; ++s) {
            bar_init(q_full(s), 1);
            bar_init(q_empty(s), 1);
        }
        for (int s = 0; s < kPieces; ++s) {
            bar_init(piece_full(s), 1);
            bar_init(piece_empty(s), 2 + kSoftmaxWarps);   // the products' warp, the one that cleans, the softmax
        }
        for (int t = 0; t < 2; ++t) {
            bar_init(scores(t), 1);
            bar_init(weights(t), kSoftmaxWarps / 2);
            bar_init(summed(t), 1);
        }
        for (int i = 0; i < kFlags; ++i) not_finite[i] = -1;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_at)), "r"(512) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        tmem_fence_before();
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");   // the kernel before may make any of what is read here
    __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = tmem_at;
    auto wait = [&](uint32_t bar, uint32_t parity) { return bar_wait_here(bar, parity, &given_up, p.status); };
    auto wait_all = [&](uint32_t bar, uint32_t parity) { return __all_sync(0xffffffffu, bar_wait_here(bar, parity, &given_up, p.status)) != 0; };
    // Whether the piece with this number is there and not the end; and that the warp is done with it.
    auto next_piece = [&](int number) {
        return wait_all(piece_full(number % kPieces), (number / kPieces) & 1) && pieces[number % kPieces].j0 >= 0;
    };
    auto piece_done = [&](int number) {
        __syncwarp();
        if (lane == 0) arrive(piece_empty(number % kPieces));
    };

    if (warp == 0) {
        if (lane == 0) {
            Border b = p.borders[blockIdx.x];
            long long left = p.borders[blockIdx.x + 1].unit - b.unit;
            // nothing of an earlier call is left in the slots
            Slot* const slots = p.slots + 2 * blockIdx.x;
            slots[0].state = slots[1].state = 0;
            int number = 0, item = 0;   // pieces, and those with blocks
            int s = 0, issued = 0;
            uint32_t phase = 0;
            bool ok = true;
            auto stage = [&](const CUtensorMap* map, const Piece& c, int j) {
                ok = ok && wait(empty(s), phase ^ 1u);
                if (!ok) return;
                const int boxes = min(kKeys, c.keys - j * kKeys) > kBoxRows ? 2 : 1;
                const uint32_t at = ring + s * kTileBytes<D>;
                bar_expect(full(s), boxes * COLS * kBoxRows * 128);
                for (int col = 0; col < COLS; ++col)
                    for (int r = 0; r < boxes; ++r)
                        box_load(at + col * (kKeys * 128) + r * (kBoxRows * 128), map, col * 64, c.head, c.k0 + j * kKeys + r * kBoxRows,
                                 full(s));
                issued = issued < ST ? issued + 1 : ST;
                if (++s == ST) { s = 0; phase ^= 1u; }
            };
            while (left > 0 && ok) {
                while (b.s < p.seq.count && range_of(p.seq.q_starts, p.seq.q_lengths, b.s, p.seq.q_rows).length == 0) ++b.s;
                if (b.s >= p.seq.count) break;   // (not reached: what is left lies in some sequence)
                const Range rq = range_of(p.seq.q_starts, p.seq.q_lengths, b.s, p.seq.q_rows);
                const Range rk = range_of(p.seq.k_starts, p.seq.k_lengths, b.s, p.seq.k_rows);
                const attention::Sequence q{rq.length, rk.length, p.tokens, p.causal};
                while (left > 0 && ok && b.head < p.kv_heads) {
                    const attention::Step step = attention::next_step(q, b, left);
                    Piece c;
                    const int i0 = step.item * 2 * p.tokens;
                    c.q0 = rq.start + i0;
                    c.tokens = min(2 * p.tokens, rq.length - i0);
                    c.head = step.head;
                    c.k0 = rk.start;
                    c.keys = rk.length;
                    c.base = (int)((long long)i0 + 1 + rk.length - rq.length);
                    c.j0 = step.j0;
                    c.j1 = step.j1;
                    c.end0 = min(step.j1, step.n0);
                    c.end1 = min(step.j1, step.n1);
                    c.least = seen_by(c, p.causal, 0);
                    c.seen0 = seen_by(c, p.causal, min(c.tokens, p.tokens) - 1);
                    c.seen1 = seen_by(c, p.causal, c.tokens - 1);
                    c.slot = -1;
                    if (!step.begins || !step.ends) {
                        const int which = step.begins ? 1 : 0;
                        c.slot = 2 * blockIdx.x + which;
                        slots[which] = Slot{step.begins ? kFirst : kNext, step.ends, c.q0, c.tokens, c.head, c.keys, c.base, 0};
                    }
                    ok = wait(piece_empty(number % kPieces), ((number / kPieces) & 1) ^ 1u);
                    if (!ok) break;
                    pieces[number % kPieces] = c;
                    arrive(piece_full(number % kPieces));
                    ++number;
                    if (c.j1 > c.j0) {
                        const int qs = item % NQ;
                        ok = wait(q_empty(qs), ((item / NQ) & 1) ^ 1u);
                        if (!ok) break;
                        const int tiles = c.tokens > p.tokens ? 2 : 1;
                        bar_expect(q_full(qs), tiles * COLS * p.tokens * p.group * 128);
                        for (int t = 0; t < tiles; ++t)
                            for (int col = 0; col < COLS; ++col)
                                box_load(queries + (qs * 2 + t) * kTileBytes<D> + col * (kRows * 128), &p.q, col * 64, c.head * p.group,
                                         c.q0 + t * p.tokens, q_full(qs));
                        ++item;
                        for (int j = c.j0; j < c.j1 && ok; ++j) {
                            stage(&p.k, c, j);
                            stage(&p.v, c, j);
                        }
                    }
                }
                b.head = 0;
                ++b.s;
            }
            if (ok && wait(piece_empty(number % kPieces), ((number / kPieces) & 1) ^ 1u)) {
                pieces[number % kPieces].j0 = -1;
                arrive(piece_full(number % kPieces));
            }
            // copies in flight land before the CTA ends, whatever became of the others
            for (int i = 0; i < issued; ++i) {
                s = s == 0 ? ST - 1 : s - 1;
                if (s == ST - 1) phase ^= 1u;
                bar_drain(full(s), phase);
            }
            for (int i = item < NQ ? 0 : item - NQ; i < item; ++i) bar_drain(q_full(i % NQ), (i / NQ) & 1);
        }
    } else if (warp == 1) {
        int s = 0, number = 0, item = 0;
        uint32_t phase = 0, weights_phase0 = 0, weights_phase1 = 0;
        uint32_t last = 0, last_phase = 0;   // the stage whose products were issued last
        auto advance = [&] {
            commit(empty(s));
            last = empty(s);
            last_phase = phase;
            if (++s == ST) { s = 0; phase ^= 1u; }
        };
        // What the products need to know of a piece, in registers that the compiler knows to be the same in every
        // lane (a maximum over the warp is): operands of other registers cost each product a loop over lanes.
        auto same = [](int v) { return __reduce_max_sync(0xffffffffu, v); };
        const uint32_t tm = (uint32_t)same((int)tmem), queries_u = (uint32_t)same((int)queries), ring_u = (uint32_t)same((int)ring);
        int j0 = 0, j1 = 0, end0 = 0, end1 = 0, seen0 = 0, seen1 = 0;               // the piece whose P V come next
        int next_j0 = 0, next_j1 = 0, next_end0 = 0, next_end1 = 0, next_seen0 = 0, next_seen1 = 0;   // the one after it
        bool ok = true;
        // That one, and whether it has blocks.  (Not the next that has some: between them more pieces may lie than
        // there are places for, and those are free only once this piece's products are done.)
        enum { kEnd, kBlocks, kNothing };
        auto look_ahead = [&] {
            const int at = number % kPieces;
            ok = wait_all(piece_full(at), (number / kPieces) & 1);
            if (!ok) return kEnd;
            const Piece& c = pieces[at];
            next_j0 = same(c.j0);
            next_j1 = same(c.j1);
            next_end0 = same(c.end0);
            next_end1 = same(c.end1);
            next_seen0 = same(c.seen0);
            next_seen1 = same(c.seen1);
            __syncwarp();
            if (lane == 0) arrive(piece_empty(at));
            if (next_j0 < 0) return kEnd;
            ++number;
            return next_j1 > next_j0 ? kBlocks : kNothing;
        };
        auto go_on = [&] {
            j0 = next_j0;
            j1 = next_j1;
            end0 = next_end0;
            end1 = next_end1;
            seen0 = next_seen0;
            seen1 = next_seen1;
        };
        const int n_values = (p.dim + 15) / 16;
        // S of tile t for block j, of whose keys some row of the tile sees seen - 128 j
        auto score = [&](int t, int seen, int j, int qs, int stage) {
            const uint64_t a = operand(queries_u + (uint32_t)same((qs * 2 + t) * kTileBytes<D>));
            const uint64_t b = operand(ring_u + (uint32_t)same(stage * kTileBytes<D>));
            const uint32_t shape = kShape | (uint32_t)same((min(kKeys, seen - j * kKeys) + 15) / 16 << 18);
            // (all of D: what a shorter head lacks was copied as zeros)
#pragma unroll
            for (int k = 0; k < D / 64; ++k)   // 64 values lie 16 KB from the next
                mma4_shared(tm + t * kKeys, a + k * (kRows * 128 / 16), b + k * (kRows * 128 / 16), shape, k > 0);
            commit(scores(t));
        };
        auto weigh = [&](int t, int seen, int j, int stage, bool add) {
            const uint64_t b = operand_across(ring_u + (uint32_t)same(stage * kTileBytes<D>), kKeys * 128);
            const int steps = same((min(kKeys, seen - j * kKeys) + 15) / 16);
            const uint32_t shape = kShape | (1u << 16) | (uint32_t)(n_values << 18), more = (uint32_t)same(add);
            const uint32_t o = tm + 2 * kKeys + t * D, w = tm + t * kKeys;
            if (steps == kKeys / 16) {
                mma4_tmem(o, w, b, shape, more);
                mma4_tmem(o, w + 32, b + 4 * 128, shape, 1);
            } else {
#pragma unroll 1
                for (int k = 0; k < steps; ++k) mma_tmem(o, w + k * 8, b + k * 128, shape, k > 0 ? 1u : more);
            }
            commit(summed(t));
        };
        auto next = look_ahead();
        bool follows = false;   // the piece's first scores are made beside the last one's products
        while (ok) {
            while (ok && next == kNothing) next = look_ahead();
            if (!ok || next == kEnd) break;
            go_on();
            for (int j = follows ? j0 : j0 - 1; j < j1; ++j) {
                const bool begun = j >= j0;   // else the first scores alone
                const int v_stage = s;
                if (begun) ok = wait_all(full(s), phase) && wait_all(clean(s), phase);
                if (!ok) break;
                // the block whose scores come next: this piece's, or the first of the next one
                const bool inside = j + 1 < j1;
                if (!inside) next = look_ahead();
                if (!ok) break;
                const bool more = inside || next == kBlocks;
                const int then_j = inside ? j + 1 : next_j0, then_item = inside ? item : item + 1, qs = then_item % NQ;
                const int then_end0 = inside ? end0 : next_end0, then_end1 = inside ? end1 : next_end1;
                const bool turns = begun && s + 1 == ST;
                const int k_stage = begun ? (turns ? 0 : s + 1) : s;
                const uint32_t k_phase = turns ? phase ^ 1u : phase;
                if (begun && j < end0) {
                    ok = wait_all(weights(0), weights_phase0);
                    weights_phase0 ^= 1u;
                    if (!ok) break;
                    tmem_fence_after();
                    weigh(0, seen0, j, v_stage, j > j0);
                }
                if (more) {
                    ok = ((inside && begun) || wait_all(q_full(qs), (then_item / NQ) & 1)) && wait_all(full(k_stage), k_phase);
                    if (!ok) break;
                    tmem_fence_after();
                    if (then_j < then_end0) score(0, inside ? seen0 : next_seen0, then_j, qs, k_stage);
                }
                if (begun && j < end1) {
                    ok = wait_all(weights(1), weights_phase1);
                    weights_phase1 ^= 1u;
                    if (!ok) break;
                    tmem_fence_after();
                    weigh(1, seen1, j, v_stage, j > j0);
                }
                if (more && then_j < then_end1) score(1, inside ? seen1 : next_seen1, then_j, qs, k_stage);
                if (begun) advance();
                if (more) {
                    advance();
                    if (then_j + 1 == (inside ? j1 : next_j1)) commit(q_empty(qs));
                }
            }
            ++item;
            follows = next == kBlocks;
        }
        if (last != 0) bar_drain(last, last_phase);   // the last products are done before TMEM is freed
        __syncwarp();
    } else if (warp == 2) {
        // Values that a row does not see: rows of the ring beyond the keys become zeros, values that are not finite too.
        // (The products wait for this warp at every block of values, so it is never a turn of the ring ahead.)
        int s = 0, number = 0;
        uint32_t phase = 0;
        bool ok = true;
        auto done = [&] {
            __syncwarp();
            if (lane == 0) arrive(clean(s));
            if (++s == ST) { s = 0; phase ^= 1u; }
        };
        while (ok && next_piece(number)) {
            const Piece& c = pieces[number % kPieces];
            bool found = false;
            for (int j = c.j0; j < c.j1 && ok; ++j) {
                ok = wait_all(full(s), phase);   // keys
                if (!ok) break;
                done();
                ok = wait_all(full(s), phase);
                if (!ok) break;
                if (masked(c.least, j)) {
                    uint8_t* const at = base + NQ * 2 * kTileBytes<D> + s * kTileBytes<D>;
                    const int rows = min(kKeys, c.keys - j * kKeys), whole = (rows + 15) / 16 * 16;
                    bool wrote = false;
                    for (int col = 0; col < COLS; ++col)
                        for (int i = lane; i < whole * 8; i += 32) {   // 16 bytes
                            uint4* const v = reinterpret_cast<uint4*>(at + col * (kKeys * 128)) + i;
                            if (i >= rows * 8) {
                                *v = make_uint4(0, 0, 0, 0);
                                wrote = true;
                                continue;
                            }
                            const uint4 x = *v;
                            if ((not_finite2<E>(x.x) | not_finite2<E>(x.y) | not_finite2<E>(x.z) | not_finite2<E>(x.w)) == 0) continue;
                            uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                            for (int h = 0; h < 4; ++h) {
                                if ((w[h] & kExponent<E>) == kExponent<E>) w[h] &= 0xffff0000u;
                                if ((w[h] >> 16 & kExponent<E>) == kExponent<E>) w[h] &= 0xffffu;
                            }
                            *v = make_uint4(w[0], w[1], w[2], w[3]);
                            wrote = found = true;
                        }
                    if (__any_sync(0xffffffffu, found) && lane == 0) not_finite[number % kFlags] = number;
                    if (wrote) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                }
                done();
            }
            if (!ok) break;
            piece_done(number++);
        }
    } else if (warp >= 4) {
        const int tile = (warp - 4) >> 2, quarter = warp & 3, row = quarter * 32 + lane;
        const uint32_t tm = tmem + ((uint32_t)(quarter * 32) << 16);
        const int token = row / p.group;
        uint32_t products = 0;   // scores seen and products of P and V asked for, so far
        int number = 0;
        bool ok = true;
        while (ok && next_piece(number)) {
            const Piece& c = pieces[number % kPieces];
            const int here = tile * p.tokens + token;   // of the item's queries
            const bool mine = token < p.tokens && here < c.tokens;
            const bool some = __any_sync(0xffffffffu, mine);
            const int seen = mine ? seen_by(c, p.causal, here) : 0;
            const int last_seen = tile == 0 ? c.seen0 : c.seen1;
            const int e = tile == 0 ? c.end0 : c.end1, begin = c.j0, least = c.least;
            float ms = -INFINITY, l = 0.0f;   // the maximum times the scale, less the lift; the sum of the weights
            for (int j = begin; j < e; ++j) {
                ok = wait_all(scores(tile), products & 1);
                if (!ok) break;
                tmem_fence_after();
                if (some) {
                    const int cols = min(kKeys, last_seen - j * kKeys);   // of the tile
                    uint32_t x[kKeys];
                    tmem_load32(tm + tile * kKeys, x);
                    tmem_load32(tm + tile * kKeys + 32, x + 32);
                    tmem_load32(tm + tile * kKeys + 64, x + 64);
                    tmem_load32(tm + tile * kKeys + 96, x + 96);
                    tmem_wait(x);
                    if (masked(least, j)) {
                        const int sees = seen - j * kKeys;
#pragma unroll
                        for (int i = 0; i < kKeys; ++i)
                            if (i >= sees) x[i] = 0xff800000u;
                    }
                    float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int i = 0; i < kKeys; i += 8)
#pragma unroll
                        for (int u = 0; u < 4; ++u)
                            top[u] = fmaxf(top[u], fmaxf(__uint_as_float(x[i + 2 * u]), __uint_as_float(x[i + 2 * u + 1])));
                    const float high = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * p.scale - kLift<E>;
                    const bool grows = high > ms + kGrowth;
                    if (__any_sync(0xffffffffu, grows)) {
                        const float factor = grows ? power2(ms - high) : 1.0f;   // (from -infinity: 0)
                        if (grows) {
                            ms = high;
                            l *= factor;
                        }
                        if (j > begin) {
                            ok = wait_all(summed(tile), (products - 1) & 1);
                            if (!ok) break;
                            tmem_fence_after();
#pragma unroll 1
                            for (int g = 0; g < D; g += 16) {
                                uint32_t o[16];
                                tmem_load16(tm + 2 * kKeys + tile * D + g, o);
                                tmem_wait(o);
#pragma unroll
                                for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * factor);
                                tmem_store16(tm + 2 * kKeys + tile * D + g, o);
                            }
                        }
                    }
                    const float off = ms == -INFINITY ? 0.0f : ms;   // nothing seen yet: weights 0
                    const Two scale2 = two(p.scale, p.scale), off2 = two(-off, -off);
                    float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};   // of the weights as the products take them
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        if (g * 32 >= cols) continue;
                        uint32_t w[16];
#pragma unroll
                        for (int i = 0; i < 32; i += 2) {
                            const float2 y = apart(fma_two(two(__uint_as_float(x[g * 32 + i]), __uint_as_float(x[g * 32 + i + 1])), scale2, off2));
                            const float a = power2(y.x), b = power2(y.y);
                            w[i / 2] = pack2<E>(a, b);
                            add_rounded<E>(w[i / 2], sum[i & 2], sum[(i & 2) + 1]);
                        }
                        tmem_store16(tm + tile * kKeys + g * 16, w);
                    }
                    l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                    tmem_stored();
                }
                tmem_fence_before();
                __syncwarp();
                if (lane == 0) arrive(weights(tile));
                ++products;
            }
            if (!ok) break;
            if (some) {
                const bool any = e > begin;
                if (any) {
                    ok = wait_all(summed(tile), (products - 1) & 1);
                    if (!ok) break;
                    tmem_fence_after();
                }
                // what only this end of a piece needs is made here, not kept in registers meanwhile
                int me = threadIdx.x - 128;
                asm volatile("" : "+r"(me));
                const int member = (me & 127) - token * p.group;
                const bool whole = c.slot < 0;
                const int part_row = max(c.slot, 0) * p.slot_rows + tile * kRows + row;
                if (!whole && mine) p.stats[part_row] = make_float2(any ? ms : -INFINITY, any ? l : 0.0f);
                const float inverse = !any || seen == 0 ? 0.0f : whole ? 1.0f / l : 1.0f;
                char* const to = whole ? static_cast<char*>(p.out) + ((long long)(c.q0 + here) * p.out_stride +
                                                                     ((long long)c.head * p.group + member) * p.dim) * 2
                                       : reinterpret_cast<char*>(p.parts + (long long)part_row * D);
                const int until = p.dim;
                if (whole || any) {
#pragma unroll 1
                    for (int g = 0; g < until; g += 32) {
                        uint32_t o[32];
                        tmem_load32(tm + 2 * kKeys + tile * D + g, o);
                        tmem_wait(o);
                        // (a row that sees nothing gets zeros, whatever its sums are)
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = inverse == 0.0f ? 0u : __float_as_uint(__uint_as_float(o[i]) * inverse);
                        auto two_of = [&](int i) { return pack2<E>(__uint_as_float(o[i]), __uint_as_float(o[i + 1])); };
                        if (mine) {
                            if (whole) {
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    if (g + 8 * i < until)
                                        *reinterpret_cast<uint4*>(to + (g + 8 * i) * 2) =
                                            make_uint4(two_of(8 * i), two_of(8 * i + 2), two_of(8 * i + 4), two_of(8 * i + 6));
                            } else {
#pragma unroll
                                for (int i = 0; i < 8; ++i)
                                    if (g + 4 * i < until)
                                        *reinterpret_cast<uint4*>(to + (g + 4 * i) * 4) = make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                            }
                        }
                    }
                    tmem_fence_before();   // O is read: the next item's products may overwrite it
                }
                if (any && not_finite[number % kFlags] == number && mine) {
                    // values of masked blocks that are not finite, for the rows that see them: added to what was written
                    const int first = max(begin, least / kKeys) * kKeys, end = min(seen, e * kKeys);
                    char* const out = to;
#pragma unroll 1
                    for (int k = first; k < end; ++k) {
                        const E* const v = static_cast<const E*>(p.values) + (long long)(c.k0 + k) * p.v_stride + (long long)c.head * p.dim;
#pragma unroll 1
                        for (int d = 0; d < until; ++d) {
                            const float f = value_of(v[d]);
                            if (isfinite(f)) continue;
                            if (whole) {
                                E* const o = reinterpret_cast<E*>(out) + d;
                                *o = from_value<E>(value_of(*o) + f);
                            } else {
                                reinterpret_cast<float*>(out)[d] += f;
                            }
                        }
                    }
                }
            }
            piece_done(number++);
        }
    }
    __syncthreads();
    if (warp == 1) {
        tmem_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
    }
    if (threadIdx.x == 0 && given_up) {   // what this CTA was to leave is not whole
        p.slots[2 * blockIdx.x].state |= kFailed;
        p.slots[2 * blockIdx.x + 1].state |= kFailed;
    }
}

// ------------------------------------------------------------ joining pieces ---

struct JoinParams {
    const Slot* slots;
    const float2* stats;
    const float* parts;
    void* out;
    long long out_stride;
    int group, dim, tokens, slot_rows;
    bool causal;
};

constexpr int kJoinWarps = 8, kJoinBlocks = 16;

// The pieces of the item that CTA blockIdx.x of the attention kernel began and did not end; gridDim.y CTAs
// share its rows.  A warp takes a row, four values a lane; where an item has many pieces (a few rows, then),
// the CTA's warps share a row's.  Latency counts: slots, maxima and sums are read by a lane each, and the
// pieces' values four at a time.
template <typename E, int D>
__global__ void __launch_bounds__(32 * kJoinWarps) join_kernel(const JoinParams p) {
    __shared__ float sums[kJoinWarps][D + 1];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int c0 = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Slot head = p.slots[2 * c0 + 1];
    if (head.state != kFirst) return;
    // pieces: this one's slot 2 c0 + 1, then slots 2 c of the CTAs after it, up to the one that ends the item; a
    // CTA that has none of it is passed over.  Nothing is stored where a wait that ran out left one unfinished.
    int n = 0;
    for (int c = c0 + 1; c < kCtas && n == 0; c += 32) {
        int state = 0, ends = 0;
        if (c + lane < kCtas) {
            state = p.slots[2 * (c + lane)].state;
            ends = p.slots[2 * (c + lane)].ends;
        }
        const unsigned end = __ballot_sync(0xffffffffu, (state & kNext) != 0 && ends != 0);
        const unsigned upto = end != 0 ? (2u << (__ffs((int)end) - 1)) - 1 : 0xffffffffu;
        if (__ballot_sync(0xffffffffu, (state & kFailed) != 0) & upto) return;
        if (end != 0) n = c - c0 + __ffs((int)end);
    }
    if (n == 0) return;   // (not reached: some CTA ends the item)
    auto slot_of = [&](int i) { return i == 0 ? 2 * c0 + 1 : 2 * (c0 + i); };
    const bool shared = n > kJoinWarps;
    const int first = shared ? blockIdx.y : blockIdx.y * kJoinWarps + warp, step = shared ? gridDim.y : gridDim.y * kJoinWarps;
    // whether piece `lane` (the first 32) has anything of the item
    const bool there = lane == 0 || (lane < n && p.slots[slot_of(min(lane, n - 1))].state == kNext);
    for (int tile = 0; tile < 2; ++tile) {
        const int tokens = min(p.tokens, head.tokens - tile * p.tokens);
        for (int row = first; row < tokens * p.group; row += step) {
            const int token = row / p.group, member = row - token * p.group, at = tile * kRows + row;
            auto stat = [&](int i) {
                const bool has = i < n && (i < 32 ? there : p.slots[slot_of(i)].state == kNext);
                return has ? p.stats[(long long)slot_of(i) * p.slot_rows + at] : make_float2(-INFINITY, 0.0f);
            };
            // of the pieces lane, lane + 32, ...: the first's statistics stay
            const float2 mine = stat(lane);
            float top = mine.x;
            for (int i = lane + 32; i < n; i += 32) top = fmaxf(top, stat(i).x);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            float l = 0.0f, acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            for (int i0 = 0; i0 < n; i0 += 32) {
                const float2 s = i0 == 0 ? mine : stat(i0 + lane);
                // a piece whose scores are not numbers has a sum that is none; one that saw nothing has no sum, and
                // no values that could be read
                const bool none = s.y == 0.0f && s.x == -INFINITY;
                const float w = none ? 0.0f : s.x == -INFINITY ? (top == -INFINITY ? 1.0f : 0.0f) : power2(s.x - top);
                const unsigned has = __ballot_sync(0xffffffffu, !none);
                const float wl = none ? 0.0f : s.y * w;
#pragma unroll 4
                for (int i = shared ? warp : 0; i < min(32, n - i0); i += shared ? kJoinWarps : 1) {
                    const float wi = __shfl_sync(0xffffffffu, w, i);
                    l += __shfl_sync(0xffffffffu, wl, i);
                    if ((has >> i & 1) && lane * 4 < D) {
                        const float4 v = *reinterpret_cast<const float4*>(p.parts + ((long long)slot_of(i0 + i) * p.slot_rows + at) * D + lane * 4);
                        acc[0] = fmaf(v.x, wi, acc[0]);
                        acc[1] = fmaf(v.y, wi, acc[1]);
                        acc[2] = fmaf(v.z, wi, acc[2]);
                        acc[3] = fmaf(v.w, wi, acc[3]);
                    }
                }
            }
            if (shared) {   // the warps' sums in order
                __syncthreads();
                if (lane * 4 < D)
#pragma unroll
                    for (int k = 0; k < 4; ++k) sums[warp][lane * 4 + k] = acc[k];
                if (lane == 0) sums[warp][D] = l;
                __syncthreads();
                if (warp != 0) continue;
                l = 0.0f;
#pragma unroll
                for (int k = 0; k < 4; ++k) acc[k] = 0.0f;
                for (int w = 0; w < kJoinWarps; ++w) {
                    l += sums[w][D];
                    if (lane * 4 < D)
#pragma unroll
                        for (int k = 0; k < 4; ++k) acc[k] += sums[w][lane * 4 + k];
                }
            }
            Piece c;
            c.base = head.base;
            c.keys = head.keys;
            const int here = tile * p.tokens + token;
            const bool sees = seen_by(c, p.causal, here) > 0;
            const float inverse = sees ? 1.0f / l : 0.0f;
            if (lane * 4 < p.dim) {
                E* to = static_cast<E*>(p.out) + (long long)(head.q0 + here) * p.out_stride + ((long long)head.head * p.group + member) * p.dim;
                *reinterpret_cast<uint2*>(to + lane * 4) =
                    make_uint2(sees ? pack2<E>(acc[0] * inverse, acc[1] * inverse) : 0u, sees ? pack2<E>(acc[2] * inverse, acc[3] * inverse) : 0u);
            }
        }
    }
}

// -------------------------------------------------------------------- host ---

// Heads of a matrix of `rows` rows, boxes of 64 values x `heads_a_box` heads x `rows_a_box` rows.
int heads_map(CUtensorMap* map, const void* at, int dtype, long long rows, int heads, int dim, long long stride, int heads_a_box,
              int rows_a_box) {
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
    const cuuint64_t dims[3] = {(cuuint64_t)dim, (cuuint64_t)heads, (cuuint64_t)rows};
    const cuuint64_t strides[2] = {(cuuint64_t)dim * 2, (cuuint64_t)stride * 2};
    const cuuint32_t boxes[3] = {64, (cuuint32_t)heads_a_box, (cuuint32_t)rows_a_box}, elem[3] = {1, 1, 1};
    const CUresult r = encode(map, dtype == TR_ELEM_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                              const_cast<void*>(at), dims, strides, boxes, elem, CU_TENSOR_MAP_INTERLEAVE_NONE,
                              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return cuda_failed("cuTensorMapEncodeTiled", (int)cudaErrorInvalidValue);
    return TR_OK;
}

size_t slots_bytes() { return 2 * kCtas * sizeof(Slot); }
size_t borders_bytes() { return (kCtas + 1) * sizeof(Border); }
static_assert(sizeof(Border) % 8 == 0 && (kCtas + 1) * sizeof(Border) % 8 == 0, "what follows is aligned");
// Rows of a partial result: of both tiles, or where one tile takes all queries, theirs (an even number).
int slot_rows(long long q_rows, long long group) { return q_rows <= kRows / group ? (int)((q_rows * group + 1) / 2 * 2) : 2 * kRows; }
size_t stats_bytes(int rows) { return 2 * kCtas * (size_t)rows * sizeof(float2); }
int padded_dim(long long dim) { return dim <= 64 ? 64 : 128; }

template <typename E, int D>
int start_tc(TcParams& p, cudaStream_t st) {
    static std::atomic<bool> ready[kMaxDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || dev < 0 || dev >= kMaxDevices) return cuda_failed("cudaGetDevice", (int)e);
    int rc = product_status_word(dev, &p.status);
    if (rc != TR_OK) return rc;
    if (!ready[dev].load(std::memory_order_relaxed)) {
        e = cudaFuncSetAttribute(attention_kernel<E, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem<D>);
        if (e != cudaSuccess) return cuda_failed("attention kernel set-up", (int)e);
        ready[dev].store(true, std::memory_order_relaxed);
    }
    cudaLaunchConfig_t cfg{};
    cfg.stream = st;
    cudaLaunchAttribute attr[1];   // the next kernel may be set up while this one ends
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const PlanParams plan{p.seq, const_cast<Border*>(p.borders), p.kv_heads, p.tokens, p.causal};
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(kPlanThreads);
    cfg.dynamicSmemBytes = 0;
    rc = launched("attention plan kernel", (int)cudaLaunchKernelEx(&cfg, plan_kernel, plan));
    if (rc != TR_OK) return rc;
    cfg.gridDim = dim3(kCtas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem<D>;
    rc = launched("attention kernel", (int)cudaLaunchKernelEx(&cfg, attention_kernel<E, D>, p));
    if (rc != TR_OK) return rc;
    const JoinParams j{p.slots, p.stats, p.parts, p.out, p.out_stride, p.group, p.dim, p.tokens, p.slot_rows, p.causal};
    cfg.gridDim = dim3(kCtas, kJoinBlocks);
    cfg.blockDim = dim3(32 * kJoinWarps);
    cfg.dynamicSmemBytes = 0;
    return launched("attention joining kernel", (int)cudaLaunchKernelEx(&cfg, join_kernel<E, D>, j));
}

template <typename E>
int type_tc(TcParams& p, cudaStream_t st) {
    return p.dim <= 64 ? start_tc<E, 64>(p, st) : start_tc<E, 128>(p, st);
}

}  // namespace

bool attention_tc_shape(long long heads, long long kv_heads, long long dim) {
    return dim % 8 == 0 && dim <= 128 && heads / kv_heads <= 64;
}

bool attention_tc_supported(const AttentionArgs& a) {
    if (a.dtype == TR_ELEM_F32 || !attention_tc_shape(a.heads, a.kv_heads, a.dim)) return false;
    if (!(a.scale > 0.0f) || a.scale > 1e30f) return false;
    auto on16 = [](const void* p, long long stride, long long rows, long long cols) {
        return (uintptr_t)p % 16 == 0 && (rows <= 1 || (stride % 8 == 0 && stride >= cols && stride < (1LL << 38)));
    };
    const long long q_cols = (long long)a.heads * a.dim, k_cols = (long long)a.kv_heads * a.dim;
    return on16(a.q, a.q_stride, a.q_rows, q_cols) && on16(a.out, a.out_stride, a.q_rows, q_cols) &&
           (a.k_rows == 0 || (on16(a.k, a.k_stride, a.k_rows, k_cols) && on16(a.v, a.v_stride, a.k_rows, k_cols)));
}

size_t attention_tc_workspace(long long q_rows, long long heads, long long kv_heads, long long dim) {
    if (!attention_tc_shape(heads, kv_heads, dim)) return 0;
    const int rows = slot_rows(q_rows, heads / kv_heads);
    return slots_bytes() + stats_bytes(rows) + borders_bytes() + (size_t)2 * kCtas * rows * padded_dim(dim) * sizeof(float);
}

int launch_attention_tc(const AttentionArgs& a) {
    TcParams p;
    p.seq = Sequences{a.q_starts, a.k_starts, a.q_lengths, a.k_lengths, a.q_rows, a.k_rows, a.sequences};
    p.out = a.out;
    p.values = a.v;
    p.out_stride = a.out_stride;
    p.v_stride = a.v_stride;
    p.kv_heads = a.kv_heads;
    p.group = a.heads / a.kv_heads;
    p.dim = a.dim;
    p.tokens = kRows / p.group;
    p.scale = a.scale * 1.44269504088896341f;
    p.causal = a.causal;
    uint8_t* const ws = static_cast<uint8_t*>(a.workspace);
    p.slots = reinterpret_cast<Slot*>(ws);
    p.stats = reinterpret_cast<float2*>(ws + slots_bytes());
    p.slot_rows = slot_rows(a.q_rows, p.group);
    p.parts = reinterpret_cast<float*>(ws + slots_bytes() + stats_bytes(p.slot_rows));
    p.borders = reinterpret_cast<Border*>(reinterpret_cast<uint8_t*>(p.parts) + (size_t)2 * kCtas * p.slot_rows * padded_dim(a.dim) * sizeof(float));
    p.missing = test_waits();
    int rc = heads_map(&p.q, a.q, a.dtype, a.q_rows, a.heads, a.dim, a.q_stride, p.group, p.tokens);
    // (without keys nothing is copied through the other maps)
    const bool keys = a.k_rows > 0;
    if (rc == TR_OK)
        rc = keys ? heads_map(&p.k, a.k, a.dtype, a.k_rows, a.kv_heads, a.dim, a.k_stride, 1, kBoxRows)
                  : heads_map(&p.k, a.q, a.dtype, 1, a.kv_heads, a.dim, (long long)a.kv_heads * a.dim, 1, kBoxRows);
    if (rc == TR_OK)
        rc = keys ? heads_map(&p.v, a.v, a.dtype, a.k_rows, a.kv_heads, a.dim, a.v_stride, 1, kBoxRows)
                  : heads_map(&p.v, a.q, a.dtype, 1, a.kv_heads, a.dim, (long long)a.kv_heads * a.dim, 1, kBoxRows);
    if (rc != TR_OK) return rc;
    cudaStream_t st = static_cast<cudaStream_t>(a.stream);
    return a.dtype == TR_ELEM_F16 ? type_tc<__half>(p, st) : type_tc<__nv_bfloat16>(p, st);
}

}  // namespace trfn
