// Attention over packed sequences: the choice of kernel, and the plain kernel.
//
// Mathematics, for a query row: with scores x_j = scale * (q . k_j) log2(e) over the
// keys that it sees, the blocks of keys are gone through once with a running
// maximum m and sum l; a block multiplies what there is by 2^(m_old - m_new):
//     l = l 2^(m_old - m_new) + sum_j 2^(x_j - m_new),  o likewise with v_j;  o / l at the end.
// A tile's rows are the (query, head) pairs of one key head, heads of a query
// next to each other: the heads that share a key read it once, and a single
// token's heads fill a tile together.
//
// The plain kernel takes what the tensor cores' kernel (attention_tc.cu) does
// not: binary32, odd lengths of heads, rows off 16-byte boundaries.  Binary32
// products in registers, 32 rows x 32 keys at a time; bound by shared memory
// (six values read for eight products).  Measured: 8192 causal queries, 32 heads of
// 128, bfloat16, 21 ms (26 TFLOP/s); a long cache is not split among CTAs.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "attention_parts.h"
#include "row_parts.h"

namespace trfn {
namespace {

struct PlainParams {
    const void* q;
    const void* k;
    const void* v;
    void* out;
    Sequences seq;
    int kv_heads, group, dim;
    long long q_stride, k_stride, v_stride, out_stride;
    float scale;   // with log2(e)
    bool causal;
};

constexpr int kTile = 32, kPlainThreads = 128;

// Dim <= 16 * DC.
template <typename E, int DC>
__global__ void __launch_bounds__(kPlainThreads) plain_kernel(const PlainParams p) {
    constexpr int D = 16 * DC, PITCH = D + 1;
    extern __shared__ float sm[];
    float* const sq = sm;                     // kTile x PITCH
    float* const sk = sq + kTile * PITCH;
    float* const sv = sk + kTile * PITCH;
    float* const sp = sv + kTile * PITCH;     // kTile x (kTile + 1)
    __shared__ int found[3];
    wait_for_previous();
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    // the sequence of this tile: the first one with so many tiles before its end
    if (tid < 32) {
        long long before = 0;
        const long long tile = blockIdx.x;
        int s = -1, t = 0;
        for (int s0 = 0; s0 < p.seq.count && s < 0; s0 += 32) {
            long long mine = 0;
            if (s0 + tid < p.seq.count)
                mine = ((long long)range_of(p.seq.q_starts, p.seq.q_lengths, s0 + tid, p.seq.q_rows).length * p.group + kTile - 1) / kTile;
            long long upto = mine;
            for (int o = 1; o < 32; o <<= 1) {
                const long long left = __shfl_up_sync(0xffffffffu, upto, o);
                if (tid >= o) upto += left;
            }
            const unsigned in = __ballot_sync(0xffffffffu, before + upto > tile);
            if (in != 0) {
                const int lane = __ffs((int)in) - 1;
                s = s0 + lane;
                t = (int)(tile - before - __shfl_sync(0xffffffffu, upto - mine, lane));
            }
            before += __shfl_sync(0xffffffffu, upto, 31);
        }
        if (tid == 0) { found[0] = s; found[1] = t; }
    }
    __syncthreads();
    const int s = found[0];
    if (s < 0) return;
    const Range rq = range_of(p.seq.q_starts, p.seq.q_lengths, s, p.seq.q_rows);
    const Range rk = range_of(p.seq.k_starts, p.seq.k_lengths, s, p.seq.k_rows);
    const int hk = blockIdx.y, n = p.dim, d0 = hk * n;
    const long long row0 = (long long)found[1] * kTile, rows = (long long)rq.length * p.group;
    // row r of the tile: query (row0 + r) / group, head (row0 + r) % group of the group
    auto place = [&](int r, long long stride) {
        const long long row = row0 + r;
        const long long i = row / p.group;
        return (rq.start + i) * stride + ((long long)hk * p.group + (row - i * p.group)) * n;
    };
    for (int e = tid; e < kTile * D; e += kPlainThreads) {
        const int r = e / D, d = e % D;
        sq[r * PITCH + d] = row0 + r < rows && d < n ? to_f(static_cast<const E*>(p.q)[place(r, p.q_stride) + d]) : 0.0f;
    }
    int seen[4], most = 0;   // keys of this thread's rows, and of the tile's
#pragma unroll
    for (int r = 0; r < 4; ++r)
        seen[r] = row0 + ty * 4 + r < rows ? attention::keys_seen((int)((row0 + ty * 4 + r) / p.group), rq.length, rk.length, p.causal) : 0;
    const long long last = min(row0 + kTile, rows) - 1;
    most = attention::keys_seen((int)(last / p.group), rq.length, rk.length, p.causal);
    float m[4], l[4], o[4][DC];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        m[r] = -INFINITY;
        l[r] = 0.0f;
#pragma unroll
        for (int c = 0; c < DC; ++c) o[r][c] = 0.0f;
    }
    for (int j0 = 0; j0 < most; j0 += kTile) {
        __syncthreads();
        for (int e = tid; e < kTile * D; e += kPlainThreads) {
            const int r = e / D, d = e % D;
            const bool in = j0 + r < rk.length && d < n;
            const long long row = (long long)rk.start + j0 + r;
            sk[r * PITCH + d] = in ? to_f(static_cast<const E*>(p.k)[row * p.k_stride + d0 + d]) : 0.0f;
            sv[r * PITCH + d] = in ? to_f(static_cast<const E*>(p.v)[row * p.v_stride + d0 + d]) : 0.0f;
        }
        __syncthreads();
        float x[4][2] = {};
        for (int d = 0; d < n; ++d) {
            const float k0 = sk[tx * PITCH + d], k1 = sk[(tx + 16) * PITCH + d];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float a = sq[(ty * 4 + r) * PITCH + d];
                x[r][0] = fmaf(a, k0, x[r][0]);
                x[r][1] = fmaf(a, k1, x[r][1]);
            }
        }
        bool all = true;   // every row of the tile sees the whole block
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            float top = -INFINITY;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                x[r][h] = j0 + tx + 16 * h < seen[r] ? x[r][h] * p.scale : -INFINITY;
                top = fmaxf(top, x[r][h]);
            }
            all = all && j0 + kTile <= seen[r];
#pragma unroll
            for (int w = 8; w > 0; w >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
            const float now = fmaxf(m[r], top), base = now == -INFINITY ? 0.0f : now;
            const float keep = exp2f(m[r] - base);
            float sum = 0.0f;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float e = exp2f(x[r][h] - base);
                sp[(ty * 4 + r) * (kTile + 1) + tx + 16 * h] = e;
                sum += e;
            }
#pragma unroll
            for (int w = 8; w > 0; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
            l[r] = fmaf(l[r], keep, sum);
            m[r] = now;
#pragma unroll
            for (int c = 0; c < DC; ++c) o[r][c] *= keep;
        }
        __syncwarp();   // a warp's rows of sp are its own
        for (int j = 0; j < kTile && j0 + j < most; ++j) {
            float pj[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) pj[r] = sp[(ty * 4 + r) * (kTile + 1) + j];
#pragma unroll
            for (int c = 0; c < DC; ++c) {
                const float v = sv[j * PITCH + tx + 16 * c];
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (all || j0 + j < seen[r]) o[r][c] = fmaf(pj[r], v, o[r][c]);   // (0 times an infinity is none of it)
            }
        }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        if (row0 + ty * 4 + r >= rows) continue;
        E* to = static_cast<E*>(p.out) + place(ty * 4 + r, p.out_stride);
        const float inverse = seen[r] > 0 ? 1.0f / l[r] : 0.0f;
#pragma unroll
        for (int c = 0; c < DC; ++c)
            if (tx + 16 * c < n) to[tx + 16 * c] = from_f<E>(o[r][c] * inverse);
    }
}

template <typename E, int DC>
int start_plain(const PlainParams& p, cudaStream_t st) {
    constexpr int smem = (3 * kTile * (16 * DC + 1) + kTile * (kTile + 1)) * (int)sizeof(float);
    if (smem > 40 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(plain_kernel<E, DC>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return cuda_failed("attention kernel set-up", (int)e);
    }
    // at most this many tiles: each sequence's last may be short
    const long long tiles = (long long)p.seq.q_rows * p.group / kTile + p.seq.count;
    if (tiles > 0x7fffffffLL) return TR_ERR_NOT_SUPPORTED;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)tiles, (unsigned)p.kv_heads);
    cfg.blockDim = dim3(kPlainThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return launched("attention kernel", (int)cudaLaunchKernelEx(&cfg, plain_kernel<E, DC>, p));
}

template <typename E>
int type_plain(const PlainParams& p, cudaStream_t st) {
    if (p.dim <= 64) return start_plain<E, 4>(p, st);
    if (p.dim <= 128) return start_plain<E, 8>(p, st);
    return start_plain<E, 16>(p, st);
}

}  // namespace

size_t attention_workspace(long long q_rows, long long, long long heads, long long kv_heads, long long dim) {
    return attention_tc_workspace(q_rows, heads, kv_heads, dim);
}

int launch_attention(const AttentionArgs& a) {
    if (attention_tc_supported(a)) return launch_attention_tc(a);
    cudaStream_t st = static_cast<cudaStream_t>(a.stream);
    PlainParams p{a.q, a.k, a.v, a.out,
                  Sequences{a.q_starts, a.k_starts, a.q_lengths, a.k_lengths, a.q_rows, a.k_rows, a.sequences},
                  a.kv_heads, a.heads / a.kv_heads, a.dim, a.q_stride, a.k_stride, a.v_stride, a.out_stride,
                  a.scale * 1.44269504088896341f, a.causal};
    if (a.dtype == TR_ELEM_F32) return type_plain<float>(p, st);
    if (a.dtype == TR_ELEM_F16) return type_plain<__half>(p, st);
    return type_plain<__nv_bfloat16>(p, st);
}

}  // namespace trfn
