// The division of attention's work (csrc/attention_plan.h), walked as the kernel
// walks it, against a list of all units: every block of every item is taken once,
// in order, and a share leaves at most one piece of an item that it did not begin
// and one of an item that it did not end.
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>

#include "attention_plan.h"

using namespace trfn::attention;

static void fail(const char* what, long long a, long long b) {
    std::printf("%s: %lld %lld\n", what, a, b);
    std::exit(1);
}

int main() {
    std::mt19937 rng(5);
    auto pick = [&](int lo, int hi) { return (int)(lo + rng() % (unsigned)(hi - lo + 1)); };
    long long splits = 0;
    for (int round = 0; round < 4000; ++round) {
        const int group = pick(1, 64), tokens = kRows / group, kv_heads = pick(1, 12), n = pick(1, 12), ctas = 152;
        const bool causal = rng() & 1;
        const int top = round % 3 == 0 ? 5 : round % 3 == 1 ? 700 : 20000;
        std::vector<Sequence> seq;
        long long units = 0;
        for (int s = 0; s < n; ++s) {
            Sequence q{pick(0, 4) == 0 ? 0 : pick(0, top), pick(0, 4) == 0 ? 0 : pick(0, top), tokens, causal};
            if (pick(0, 2) == 0) q.lq = pick(1, 3);
            seq.push_back(q);
            // the units by hand
            long long w = 0;
            for (int t = 0; (long long)t * 2 * tokens < q.lq; ++t) {
                long long last = (long long)(t + 1) * 2 * tokens < q.lq ? (long long)(t + 1) * 2 * tokens : q.lq;
                long long seen = causal ? last + q.lk - q.lq : q.lk;
                seen = seen < 0 ? 0 : seen > q.lk ? q.lk : seen;
                const long long blocks = (seen + kKeys - 1) / kKeys;
                if (blocks != q.item_blocks(t)) fail("item_blocks", blocks, q.item_blocks(t));
                w += blocks + kItemCost;
                if (w != q.units_before(t + 1)) fail("units_before", w, q.units_before(t + 1));
            }
            if (w != q.head_units()) fail("head_units", w, q.head_units());
            units += w * kv_heads;
        }
        long long parts64 = units / 2 < ctas ? units / 2 : ctas;
        const int parts = parts64 < 1 ? 1 : (int)parts64;
        auto border = [&](int c) {
            const long long want = share_start(units, parts, c < parts ? c : parts);
            long long before = 0;
            for (int s = 0; s < n; ++s) {
                const long long w = seq[s].head_units() * kv_heads;
                if (want >= before && want < before + w) return border_in(seq[s], s, kv_heads, before, want, units, parts);
                before += w;
            }
            return Border{units, n, 0, 0, 0};
        };
        // the place where the next block has to be
        int at_s = 0, at_head = 0, at_item = 0, at_block = 0;
        long long done = 0;
        for (int c = 0; c < ctas; ++c) {
            Border b = border(c);
            const long long start = b.unit, end = border(c + 1).unit;
            if (start != done || end < start) fail("share", start, done);
            long long left = end - start;
            int inside = 0, unfinished = 0;
            while (left > 0) {
                while (b.s < n && seq[b.s].lq == 0) ++b.s;
                if (b.s >= n) fail("past the sequences", b.s, left);
                while (left > 0 && b.head < kv_heads) {
                    const long long before = left;
                    const Step t = next_step(seq[b.s], b, left);
                    done += before - left;
                    while (at_s < n && (seq[at_s].lq == 0 || at_head == kv_heads)) { ++at_s; at_head = 0; }
                    if (t.head != at_head || t.item != at_item || t.j0 != at_block) fail("place", t.item, at_item);
                    if (t.begins != (at_block == 0)) fail("begins", t.j0, at_block);
                    const int blocks = seq[at_s].item_blocks(at_item);
                    if (before - left > t.j1 - t.j0 + (t.begins ? kItemCost : 0)) fail("units and blocks", before - left, t.j1 - t.j0);
                    if (t.j1 > blocks || (t.ends != (t.j1 == blocks))) fail("ends", t.j1, blocks);
                    if (!t.ends && t.j1 <= t.j0) fail("nothing taken", t.j0, t.j1);
                    inside += !t.begins;
                    unfinished += t.begins && !t.ends;
                    at_block = t.j1;
                    if (t.ends) {
                        at_block = 0;
                        if (++at_item == seq[at_s].items()) { at_item = 0; ++at_head; }
                    }
                }
                b.head = 0;
                ++b.s;
            }
            if (inside > 1 || unfinished > 1) fail("pieces", inside, unfinished);
            splits += inside;
        }
        if (done != units) fail("units", done, units);
    }
    if (splits < 1000) fail("hardly any item was split", splits, 0);
    std::printf("ok %lld\n", splits);
    return 0;
}
