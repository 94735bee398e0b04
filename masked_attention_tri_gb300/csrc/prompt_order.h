// prompt_order.h -- the order in which prompt attention's work items are taken, as the kernels count it (prompt_tc.cuh) and as
// a host program can check it.
//
// A tile is up to tq tokens (a power of two) of a group's heads; ng tiles hold the same tokens.  An item is PER neighbouring tiles of one
// (sequence, key head).  Items go by falling level, the key tiles (128 keys) that an item's last tile sees (past 32768 keys as many
// of them together as leave 256 levels); of those of a level by sequence, then place in it, then head.  No table is kept: an index
// is found by counting the items of the sequences, 32 at a time.  Each level that holds items costs two or three passes over the
// sequences and the items of a level one, whatever a block takes of them, levels without items are passed over, and an index past
// the last one ends at once: with 65535 sequences a block needs some million steps of a few hundred clocks at most, a tenth of
// the limit of the waits.
#pragma once

#ifdef __CUDACC__
#define TRIATTN_ORDER_FN __host__ __device__ __forceinline__
#else
#define TRIATTN_ORDER_FN inline
#endif

namespace triattn {
namespace prompt {

// What a sequence gives.
struct Seq {
    int q0, k0;                // first packed rows
    int lq, lk;
    int shift;                 // query j sees the keys up to j + shift
};

// Seqs: the sequences, n() of them, and what 32 lanes do with 32 of them, from s0 on:
//   sum(s0, f), most(s0, f)   of f(sequence); most is -1 at least
//   find(s0, f, place, s)     the sequence s in whose f the place lies, and the place in it; or false, and place less the sum
template <int PER>
struct Order {
    static constexpr int kLevels = 256;
    int tq_bits, ng, heads;    // tq = 1 << tq_bits; key heads
    int step, top;             // key tiles of a level; the highest level
    long long total;           // items
    int level;                 // the level at hand
    long long base, here;      // items of the levels before it, and its own
    int s0, before;            // the sequences looked at last in it, and the places of those before them

    // Tiles of a sequence, its items, and those that end within n levels.
    TRIATTN_ORDER_FN int tiles(const Seq& q) const { return ((q.lq + (1 << tq_bits) - 1) >> tq_bits) * ng; }
    TRIATTN_ORDER_FN int items(const Seq& q) const { return (tiles(q) + PER - 1) / PER; }
    TRIATTN_ORDER_FN int upto(const Seq& q, int n) const {
        if (n < 0) return 0;
        const int keys = 128 * step * n;
        if (q.lk <= keys) return items(q);
        const int x = keys - q.shift;  // tokens (of the sequence) whose last key lies there
        return x <= 0 ? 0 : (int)((long long)(x >> tq_bits) * ng / PER);
    }
    // The level of the last item below level n, or -1.
    TRIATTN_ORDER_FN int next_below(const Seq& q, int n) const {
        const int c = upto(q, n - 1);
        if (c == 0) return -1;
        const int t = (PER * c < tiles(q) ? PER * c : tiles(q)) - 1, end = (t / ng + 1) << tq_bits;
        const int keys = (end < q.lq ? end : q.lq) + q.shift;
        return keys <= 0 ? 0 : ((keys + 127) / 128 + step - 1) / step;
    }
    template <typename Seqs>
    TRIATTN_ORDER_FN long long level_items(const Seqs& seqs, int n) const {
        long long sum = 0;
        for (int s0 = 0; s0 < seqs.n(); s0 += 32) sum += seqs.sum(s0, [&](const Seq& q) { return upto(q, n) - upto(q, n - 1); });
        return sum * heads;
    }
    template <typename Seqs>
    TRIATTN_ORDER_FN void begin(const Seqs& seqs, int tq_bits_, int ng_, int heads_) {
        tq_bits = tq_bits_, ng = ng_, heads = heads_;
        int most = 0;
        total = 0;
        for (int s = 0; s < seqs.n(); s += 32) {
            const int m = seqs.most(s, [&](const Seq& q) { return q.lq > 0 ? (q.lk + 127) / 128 : 0; });
            most = m > most ? m : most;
            total += seqs.sum(s, [&](const Seq& q) { return items(q); });
        }
        total *= heads;
        step = most <= kLevels ? 1 : (most + kLevels - 1) / kLevels;
        top = (most + step - 1) / step;
        restart();
    }
    TRIATTN_ORDER_FN void restart() {
        level = top + 1;
        base = here = 0;
    }
    // The item of an index: its sequence, place in it and key head; false past the last.  Indexes may come in any order (nothing
    // says in which order a block is given others' places): an earlier one than the level at hand begins anew.
    template <typename Seqs>
    TRIATTN_ORDER_FN bool locate(const Seqs& seqs, long long at, int& s, int& item, int& head) {
        if (at >= total) return false;
        if (at < base) restart();
        while (at >= base + here) {
            base += here;
            here = level_items(seqs, --level);
            s0 = before = 0;
            if (here > 0) continue;
            int next = -1;
            for (int i = 0; i < seqs.n(); i += 32) {
                const int m = seqs.most(i, [&](const Seq& q) { return next_below(q, level); });
                next = m > next ? m : next;
            }
            level = next + 1;
        }
        const unsigned rank = (unsigned)(at - base);
        int place = (int)(rank / (unsigned)heads);
        head = (int)(rank - (unsigned)place * (unsigned)heads);
        if (place < before) s0 = before = 0;
        place -= before;
        for (; s0 < seqs.n(); s0 += 32) {
            const int from = place;
            if (seqs.find(s0, [&](const Seq& q) { return upto(q, level) - upto(q, level - 1); }, place, s)) {
                item = upto(seqs.at(s), level - 1) + place;
                return true;
            }
            before += from - place;
        }
        return false;
    }
};

}  // namespace prompt
}  // namespace triattn
