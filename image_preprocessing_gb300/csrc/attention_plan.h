// How the tensor cores' attention divides its work, in plain arithmetic shared
// by the kernel and a host test.
//
// A tile is 128 rows: `tokens` queries of a sequence times the heads of a key
// head.  An item is two tiles, one after the other, over the keys that its last
// query sees, in blocks of 128; it counts one unit a block and kItemCost for its
// beginning and end (measured: about two blocks' time).  Items
// are numbered by sequence, key head, and place in the sequence, their units in
// that order, and a CTA takes an even share of the units: it may begin and end
// inside an item.  A share's border that is less than a sixteenth of a share from
// an item's border moves there.  Everything is in closed form: a loop over a long
// prompt's items took 60 us before the first product.
#pragma once

#include <math.h>

#ifdef __CUDACC__
#define TRFN_BOTH __host__ __device__ __forceinline__
#else
#define TRFN_BOTH inline
#endif

namespace trfn {
namespace attention {

constexpr int kRows = 128, kKeys = 128;   // of a tile, of a block
constexpr int kItemCost = 2;

// a / b, by the narrow division where that does.
TRFN_BOTH unsigned long long quotient(unsigned long long a, unsigned long long b) {
    return (a | b) >> 32 ? a / b : (unsigned)a / (unsigned)b;
}

// sum over i < n of floor((a i + b) / m), m > 0 (the quotients' whole parts are summed, then rows and
// columns change places: as the greatest common divisor is found).
TRFN_BOTH unsigned long long floor_sum(unsigned long long n, unsigned long long m, unsigned long long a, unsigned long long b) {
    unsigned long long sum = 0;
    for (;;) {
        const unsigned long long qa = quotient(a, m), qb = quotient(b, m);
        sum += (n & 1 ? n * ((n - 1) / 2) : n / 2 * (n - 1)) * qa + n * qb;
        a -= qa * m;
        b -= qb * m;
        const unsigned long long top = a * n + b;
        if (top < m) return sum;
        n = quotient(top, m);
        b = top - n * m;
        const unsigned long long t = m;
        m = a;
        a = t;
    }
}

// Keys that query i of lq sees of lk: the first so many.
TRFN_BOTH int keys_seen(int i, int lq, int lk, bool causal) {
    if (!causal) return lk;
    const long long n = (long long)i + 1 + lk - lq;
    return n < 0 ? 0 : n < lk ? (int)n : lk;
}

struct Sequence {
    int lq, lk;
    int tokens;   // of a tile
    bool causal;

    TRFN_BOTH int items() const { return (int)(((unsigned)lq + 2 * (unsigned)tokens - 1) / (2 * (unsigned)tokens)); }
    // Blocks of tile `half` of item t: what its last query sees; 0 where it has no query.
    TRFN_BOTH int blocks(int t, int half) const {
        const long long first = ((long long)t * 2 + half) * tokens;
        if (first >= lq) return 0;
        const long long end = first + tokens < lq ? first + tokens : lq;
        return (int)(((long long)keys_seen((int)end - 1, lq, lk, causal) + kKeys - 1) / kKeys);
    }
    TRFN_BOTH int item_blocks(int t) const {
        const int a = blocks(t, 0), b = blocks(t, 1);
        return a > b ? a : b;
    }
    TRFN_BOTH int item_units(int t) const { return item_blocks(t) + kItemCost; }
    // Units of the first t items (t <= items()) of a key head.
    TRFN_BOTH long long units_before(int t) const {
        const int n = items(), early = t < n ? t : n - 1;   // of these, all but the sequence's last item
        if (t <= 0) return 0;
        long long sum = (long long)early * kItemCost;
        if (!causal) {
            sum += (long long)early * item_blocks(0);
        } else {
            // item i sees lk - lq + (i + 1) 2 tokens keys, less than lk; from `first` on more than none
            const long long span = 2LL * tokens, ahead = (long long)lk - lq;
            const long long first = ahead >= 0 ? 0 : (long long)quotient((unsigned long long)-ahead, (unsigned long long)span);
            if (first < early)
                sum += (long long)floor_sum((unsigned long long)(early - first), kKeys, (unsigned long long)span,
                                            (unsigned long long)(ahead + (first + 1) * span + kKeys - 1));
        }
        return early < t ? sum + item_units(n - 1) : sum;
    }
    // Units of a key head.
    TRFN_BOTH long long head_units() const { return units_before(items()); }
};

struct Place {
    int head, item, unit;   // unit: within the item, below item_units(item)
};

// Where unit `at` of a sequence (below kv_heads * head_units()) lies.
TRFN_BOTH Place place_of(const Sequence& s, long long at) {
    const long long w = s.head_units();
    Place p;
    p.head = (int)quotient((unsigned long long)at, (unsigned long long)w);
    long long rest = at - p.head * w;
    if (!s.causal) {
        const int u = s.item_units(0);
        p.item = (int)quotient((unsigned long long)rest, (unsigned long long)u);
        p.unit = (int)(rest - (long long)p.item * u);
        return p;
    }
    // a guess, as if an item's units grew evenly, then item by item
    const int n = s.items();
    const float slope = 2.0f * (float)s.tokens / kKeys;
    const float zero = s.lk < s.lq ? (float)((long long)s.lq - s.lk) / (2.0f * (float)s.tokens) : 0.0f;   // items that see nothing
    float guess = (float)rest / (float)kItemCost;
    if (guess > zero) {
        const float b = kItemCost + 0.5f + (s.lk > s.lq ? (float)((long long)s.lk - s.lq) / kKeys : 0.0f) + slope * 0.5f;
        guess = zero + (sqrtf(b * b + 2 * slope * ((float)rest - zero * kItemCost)) - b) / slope;
    }
    p.item = guess < (float)(n - 1) ? (int)guess : n - 1;
    if (p.item < 0) p.item = 0;
    long long before = s.units_before(p.item);
    while (before > rest) before -= s.item_units(--p.item);
    for (int u = s.item_units(p.item); rest - before >= u; u = s.item_units(p.item)) {
        before += u;
        ++p.item;
    }
    p.unit = (int)(rest - before);
    return p;
}

// First unit of share c of `parts`, before and after it is moved to a border of the item that it is in.
TRFN_BOTH long long share_start(long long units, int parts, int c) {
    // (c parts of a quotient and of its remainder: no overflow)
    const long long q = (long long)quotient((unsigned long long)units, (unsigned long long)parts);
    const int r = (int)(units - q * parts);
    return q * c + r * c / parts;
}

// Where a share begins: number of its first unit; sequence, key head, item of the head, unit of the item.
struct Border {
    long long unit;
    int s, head, item, at;
};

// The border at unit `want`, which lies in sequence s, whose units begin at `before`.
TRFN_BOTH Border border_in(const Sequence& q, int s, int kv_heads, long long before, long long want, long long units, int parts) {
    const Place p = place_of(q, want - before);
    Border b{want, s, p.head, p.item, p.unit};
    const long long reach = (long long)quotient((unsigned long long)units, (unsigned long long)parts) / 16 + kItemCost;
    const int n = q.item_units(p.item);
    if (p.unit <= reach) {
        b.unit -= p.unit;
        b.at = 0;
    } else if (n - p.unit <= reach) {   // the next item's start
        b.unit += n - p.unit;
        b.at = 0;
        if (++b.item == q.items()) {
            b.item = 0;
            if (++b.head == kv_heads) {
                b.head = 0;
                ++b.s;   // (an empty sequence is passed over by whoever goes on from here)
            }
        }
    }
    return b;
}

// What a share does of one item: blocks j0 .. j1 of n0 and n1 that its tiles see.
struct Step {
    int head, item, j0, j1, n0, n1;
    bool begins, ends;   // with the item's first unit, with its last
};

// The next step in sequence b.s, of at most `left` units; goes on to the item after it.  (An item's first
// kItemCost units are its cost; shares have their borders elsewhere.)
TRFN_BOTH Step next_step(const Sequence& q, Border& b, long long& left) {
    Step t;
    t.head = b.head;
    t.item = b.item;
    t.n0 = q.blocks(b.item, 0);
    t.n1 = q.blocks(b.item, 1);
    const int n = t.n0 > t.n1 ? t.n0 : t.n1, rest = n + kItemCost - b.at;
    const int take = left < rest ? (int)left : rest, until = b.at + take - kItemCost;
    t.j0 = b.at > kItemCost ? b.at - kItemCost : 0;
    t.j1 = until > 0 ? until : 0;
    t.begins = b.at == 0;
    t.ends = take == rest;
    left -= take;
    b.unit += take;
    b.at = t.ends ? 0 : b.at + take;
    if (t.ends && ++b.item == q.items()) {
        b.item = 0;
        ++b.head;   // the caller goes to the next sequence after the last
    }
    return t;
}

}  // namespace attention
}  // namespace trfn
