// prompt_order.h -- the order in which prompt attention's work items are taken, as the kernels count it (prompt_tc.cuh) and as
// a host program can check it.
//
// A tile is up to tq tokens (a power of two) of a group's heads; ng tiles hold the same tokens.  An item is PER neighbouring tiles of one
// (sequence, key head).  Items go by falling level, the key tiles (128 keys) that an item's last tile sees; of those of a level by
// sequence, then place in it, then head.  No table is kept: an index is found by counting the items of the sequences, 32 at a time.
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
    int tq_bits, ng, heads;    // tq = 1 << tq_bits; key heads
    int top;                   // the highest level
    int level;                 // the level at hand
    long long base, here;      // items of the levels before it, and its own

    // Tiles of a sequence, and its items that end within n key tiles.
    TRIATTN_ORDER_FN int tiles(const Seq& q) const { return ((q.lq + (1 << tq_bits) - 1) >> tq_bits) * ng; }
    TRIATTN_ORDER_FN int upto(const Seq& q, int n) const {
        if (n < 0) return 0;
        if (q.lk <= 128LL * n) return (tiles(q) + PER - 1) / PER;
        const int x = 128 * n - q.shift;  // tokens (of the sequence) whose last key lies there
        return x <= 0 ? 0 : (int)((long long)(x >> tq_bits) * ng / PER);
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
        top = 0;
        for (int s0 = 0; s0 < seqs.n(); s0 += 32) {
            const int m = seqs.most(s0, [&](const Seq& q) { return q.lq > 0 ? (q.lk + 127) / 128 : 0; });
            top = m > top ? m : top;
        }
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
        if (at < base) restart();
        while (at >= base + here) {
            if (level == 0) return false;
            base += here;
            here = level_items(seqs, --level);
        }
        const unsigned rank = (unsigned)(at - base);
        int place = (int)(rank / (unsigned)heads);
        head = (int)(rank - (unsigned)place * (unsigned)heads);
        for (int s0 = 0; s0 < seqs.n(); s0 += 32) {
            if (!seqs.find(s0, [&](const Seq& q) { return upto(q, level) - upto(q, level - 1); }, place, s)) continue;
            item = upto(seqs.at(s), level - 1) + place;
            return true;
        }
        return false;
    }
};

}  // namespace prompt
}  // namespace triattn
