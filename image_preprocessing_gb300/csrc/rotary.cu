// Rotary positions: pairs of a head's values turned by an angle that grows with
// the token's position, and back (the gradient).
//
// Mathematics, for pair k = (a, b) of a head at position t, with frequency f_k:
//     c, s = magnitude * (cos, sin)(t f_k)
//     (a, b) -> (a c - b s, b c + a s);  inverse: s -> -s
// The pair is (k, k + rot/2) (halves) or (2k, 2k + 1) (pairs) of the head's
// first `rot` values; the rest are copied.
//
// Angles.  t f_k of far positions has no fraction left in binary32 (position
// 10^6: steps of 2^-4 radians).  f_k / 2 pi is taken modulo 1 as a 64-bit
// fraction of a turn on the host; t times it modulo 2^64 is the exact phase of
// that fraction, within 2^-33 turns for any 32-bit t, and its upper 32 bits go
// through sincospif.
//
// Bound by HBM.  A thread takes V pairs of a token and goes through heads: the
// angles are made once for all of them.  Measured: 50176 x 24 heads of 64, binary16,
// 51 us (0.89 of the copy rate); 8192 x 40 x 128, bfloat16, half of each head, 30 us
// (0.82); heads off 16-byte boundaries value by value, 8192 x 40 x 96 33 us (0.56).
#include "row_parts.h"

#include <cmath>

namespace trfn {
namespace {

constexpr int kMaxPairs = TR_MAX_ROTARY / 2;

struct RotaryParams {
    const void* x;
    void* out;
    const int32_t* positions;
    long long tokens, x_stride, out_stride, threads;
    int heads, dim, rot, slices, per_slice, groups, turned;   // groups of a head, of which the first turn
    float magnitude, sign;
    unsigned long long turns[kMaxPairs];   // a position's share of a turn, in 2^-64
};

// Heads whose packs are under way at once.
constexpr int kRotaryHeads = 4;

// A head is V values of each half of its turned part (HALVES) or 2 V values in
// a row to a group, the rest 2 V values to a group.
template <typename E, int V, bool HALVES>
__global__ void __launch_bounds__(256) rotary_kernel(const __grid_constant__ RotaryParams p) {
    wait_for_previous();
    const long long id = (long long)blockIdx.x * 256 + threadIdx.x;
    if (id >= p.threads) return;
    // neighbours take the groups of a head, then slices of heads, then tokens
    const long long rest = id / p.groups;
    const int group = (int)(id - rest * p.groups);
    const long long token = rest / p.slices;
    const int head0 = (int)(rest - token * p.slices) * p.per_slice, head1 = min(p.heads, head0 + p.per_slice);
    const bool turn = group < p.turned;
    int at0, at1;   // this group's two packs in a head
    if (turn) {
        at0 = HALVES ? group * V : group * 2 * V;
        at1 = HALVES ? at0 + p.rot / 2 : at0 + V;
    } else {
        at0 = p.rot + (group - p.turned) * 2 * V;
        at1 = at0 + V;
    }
    const bool second = at1 < p.dim;
    float c[V], s[V];
    if (turn) {
        const long long t = p.positions != nullptr ? p.positions[token] : token;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int phase = (int)(((unsigned long long)t * p.turns[group * V + j]) >> 32);   // 2^-32 turns
            sincospif((float)phase * 0x1p-31f, &s[j], &c[j]);
            c[j] *= p.magnitude;
            s[j] *= p.magnitude * p.sign;
        }
    }
    const E* x = static_cast<const E*>(p.x) + token * p.x_stride;
    E* out = static_cast<E*>(p.out) + token * p.out_stride;
    for (int h = head0; h < head1; h += kRotaryHeads) {
        Pack<E, V> a[kRotaryHeads], b[kRotaryHeads];
#pragma unroll
        for (int u = 0; u < kRotaryHeads; ++u)
            if (h + u < head1) {
                const E* from = x + (long long)(h + u) * p.dim;
                a[u].word = *reinterpret_cast<const typename Word<sizeof(E) * V>::T*>(from + at0);
                if (second) b[u].word = *reinterpret_cast<const typename Word<sizeof(E) * V>::T*>(from + at1);
            }
#pragma unroll
        for (int u = 0; u < kRotaryHeads; ++u)
            if (h + u < head1) {
                if (turn) {
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        // pair j: (a_j, b_j), or values 2j and 2j + 1 of the two packs in a row
                        E& lo = HALVES ? a[u].e[j] : 2 * j < V ? a[u].e[(2 * j) % V] : b[u].e[(2 * j) % V];
                        E& hi = HALVES ? b[u].e[j] : 2 * j + 1 < V ? a[u].e[(2 * j + 1) % V] : b[u].e[(2 * j + 1) % V];
                        const float l = to_f(lo), r = to_f(hi);
                        lo = from_f<E>(l * c[j] - r * s[j]);
                        hi = from_f<E>(r * c[j] + l * s[j]);
                    }
                }
                E* to = out + (long long)(h + u) * p.dim;
                *reinterpret_cast<typename Word<sizeof(E) * V>::T*>(to + at0) = a[u].word;
                if (second) *reinterpret_cast<typename Word<sizeof(E) * V>::T*>(to + at1) = b[u].word;
            }
    }
}

template <typename E, int V>
int start_rotary(const RotaryArgs& a, cudaStream_t st) {
    RotaryParams p;
    p.x = a.x; p.out = a.out; p.positions = a.positions;
    p.tokens = a.tokens; p.x_stride = a.x_stride; p.out_stride = a.out_stride;
    p.heads = a.heads; p.dim = a.dim; p.rot = a.rot;
    p.magnitude = a.magnitude;
    p.sign = a.inverse ? -1.0f : 1.0f;
    p.turned = a.rot / (2 * V);
    // in place the rest stays where it is
    const bool in_place = a.x == a.out;
    p.groups = p.turned + (in_place ? 0 : (a.dim - a.rot + 2 * V - 1) / (2 * V));
    for (int k = 0; k < a.rot / 2; ++k) {
        double t = a.freqs[k] * (0.5 / 3.14159265358979323846);
        t -= std::floor(t);
        p.turns[k] = t < 1.0 ? (unsigned long long)std::ldexp(t, 64) : 0;
    }
    // heads to a thread: as many as leave every SM its threads (each makes its angles again: 8192 x 40 x 128 with
    // half as many heads 33.5 us, so 31.0), up to 8 (50176 x 24 x 64: 54.6 us with 12, 50.6 with 4)
    const double items = (double)a.tokens * p.groups * a.heads;
    const double per = items / (152.0 * 2048);
    p.per_slice = per < 1 ? 1 : per < a.heads ? (int)per : a.heads;
    if (p.per_slice > 8) p.per_slice = 8;
    if (p.per_slice > kRotaryHeads) p.per_slice = p.per_slice / kRotaryHeads * kRotaryHeads;
    p.slices = (a.heads + p.per_slice - 1) / p.per_slice;
    p.threads = a.tokens * p.slices * p.groups;
    const long long ctas = (p.threads + 255) / 256;
    if (ctas > 0x7fffffffLL) return TR_ERR_NOT_SUPPORTED;
    return launch_row_kernel("rotary kernel", a.halves ? rotary_kernel<E, V, true> : rotary_kernel<E, V, false>, (unsigned)ctas, 256, 0,
                             st, p);
}

// The widest packs on whose boundaries all heads and halves start.
template <typename E>
int type_rotary(const RotaryArgs& a, cudaStream_t st) {
    const int es = sizeof(E);
    unsigned long long at = (uintptr_t)a.x | (uintptr_t)a.out | (unsigned long long)a.dim * es |
                            (unsigned long long)(a.halves ? a.rot / 2 : a.rot / 2 * 2) * es | (unsigned long long)a.rot * es;
    if (a.tokens > 1) at |= (unsigned long long)(a.x_stride * es) | (unsigned long long)(a.out_stride * es);
    auto fits = [&](int V) { return at % (unsigned)(V * es) == 0 && a.rot % (2 * V) == 0; };
    if constexpr (sizeof(E) == 2)
        if (fits(8)) return start_rotary<E, 8>(a, st);
    if (fits(4)) return start_rotary<E, 4>(a, st);
    if (fits(2)) return start_rotary<E, 2>(a, st);
    return start_rotary<E, 1>(a, st);
}

}  // namespace

int launch_rotary(const RotaryArgs& a) {
    cudaStream_t st = static_cast<cudaStream_t>(a.stream);
    if (a.dtype == TR_ELEM_F32) return type_rotary<float>(a, st);
    if (a.dtype == TR_ELEM_F16) return type_rotary<__half>(a, st);
    return type_rotary<__nv_bfloat16>(a, st);
}

}  // namespace trfn
