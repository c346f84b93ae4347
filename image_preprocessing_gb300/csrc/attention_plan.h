// How the tensor cores' attention divides its work, in plain arithmetic shared
// by the kernel and a host test.
//
// A tile is 128 rows: `tokens` queries of a sequence times the heads of a key
// head.  An item is two tiles, one after the other, over the keys that its last
// query sees, in blocks of 128; it counts one unit a block (one at least).  Items
// are numbered by sequence, key head, and place in the sequence, their units in
// that order, and a CTA takes an even share of the units: it may begin and end
// inside an item.  A share's border that is less than a sixteenth of a share from
// an item's border moves there.
#pragma once

#ifdef __CUDACC__
#define TRFN_BOTH __host__ __device__ __forceinline__
#else
#define TRFN_BOTH inline
#endif

namespace trfn {
namespace attention {

constexpr int kRows = 128, kKeys = 128;   // of a tile, of a block

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

    TRFN_BOTH int items() const { return (int)(((long long)lq + 2 * tokens - 1) / (2 * tokens)); }
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
    TRFN_BOTH int item_units(int t) const {
        const int n = item_blocks(t);
        return n > 0 ? n : 1;
    }
    // Units of a key head.
    TRFN_BOTH long long head_units() const {
        const int n = items();
        if (n == 0) return 0;
        if (!causal) return (long long)n * item_units(0);
        long long sum = 0;
        for (int t = 0; t < n; ++t) sum += item_units(t);
        return sum;
    }
};

struct Place {
    int head, item, unit;   // unit: within the item, below item_units(item)
};

// Where unit `at` of a sequence (below kv_heads * head_units()) lies.
TRFN_BOTH Place place_of(const Sequence& s, long long at) {
    const long long w = s.head_units();
    Place p;
    p.head = (int)(at / w);
    long long rest = at - p.head * w;
    if (!s.causal) {
        const int u = s.item_units(0);
        p.item = (int)(rest / u);
        p.unit = (int)(rest - (long long)p.item * u);
        return p;
    }
    p.item = 0;
    for (int u = s.item_units(0); rest >= u; u = s.item_units(p.item)) {
        rest -= u;
        ++p.item;
    }
    p.unit = (int)rest;
    return p;
}

// First unit of share c of `parts`, before and after it is moved to a border of the item that it is in.
TRFN_BOTH long long share_start(long long units, int parts, int c) {
    // (c parts of a quotient and of its remainder: no overflow)
    const long long q = units / parts, r = units % parts;
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
    const long long reach = units / parts / 16;
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

// The next step in sequence b.s, of at most `left` units; goes on to the item after it.
TRFN_BOTH Step next_step(const Sequence& q, Border& b, long long& left) {
    Step t;
    t.head = b.head;
    t.item = b.item;
    t.n0 = q.blocks(b.item, 0);
    t.n1 = q.blocks(b.item, 1);
    const int n = t.n0 > t.n1 ? t.n0 : t.n1, units = n > 0 ? n : 1, rest = units - b.at;
    const int take = left < rest ? (int)left : rest;
    t.j0 = b.at;
    t.j1 = b.at + take < n ? b.at + take : n;
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
