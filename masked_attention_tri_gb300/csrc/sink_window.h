// sink_window.h -- which blocks TA_MASK_SINK_WINDOW without block lists visits, and how the backward
// shares the first key blocks out over several CTAs.  Plain integer arithmetic, for host and device
// (and for a host program that checks it without the CUDA headers).
#pragma once

#ifdef __CUDACC__
#define TRIATTN_HD __host__ __device__ __forceinline__
#else
#define TRIATTN_HD inline
#endif

namespace triattn {

// The 128-key blocks that hold a kept key for some query of [q0, q1], of a sequence with Lk keys:
// [0, nsink) and [lo, hi].  (A key k is kept for a query of the range when k < sinks and k <= q1, or when
// q0 - window < k <= q1.)
struct SinkBlocks {
    int nsink, lo, hi;
    TRIATTN_HD bool visited(int kb) const { return kb < nsink || (kb >= lo && kb <= hi); }
};
TRIATTN_HD SinkBlocks sink_blocks(int q0, int q1, int Lk, int window, int sinks) {
    SinkBlocks b;
    const int last = q1 < Lk - 1 ? q1 : Lk - 1;  // last key that any query reaches
    const int first = q0 - window + 1 > 0 ? q0 - window + 1 : 0;
    const int ns = sinks < last + 1 ? sinks : last + 1;
    b.nsink = ns > 0 ? (ns + 127) / 128 : 0;
    b.lo = first / 128;
    b.hi = first <= last ? last / 128 : -1;
    return b;
}

// The backward's sharing of the first key blocks.  A q block is far from key block kb when the window of
// its first query starts past the block's 128 columns: it sees the block's sinks alone.  The far q blocks
// of the first nb key blocks go to CTAs of their own, chunk of them each.
struct SinkSharing {
    int nb, chunk, chunks;  // key blocks (0: off), q blocks of a far CTA, far CTAs of a key block
};

// First q block of chunk `far` of those far from key block kb.
TRIATTN_HD long long sink_far_first(int kb, int window, int chunk, int far) {
    return (kb * 128LL + 126 + window) / 128 + 1 + (long long)far * chunk;
}

// The q blocks that a CTA of key block kb looks at, [qb0, qb1): its chunk of the far ones (far >= 0), or all (far < 0).
// Lq queries, Lk keys.
struct QBlocks {
    int qb0, qb1;
    bool all_valid;  // every query has a valid key
};
TRIATTN_HD QBlocks sink_q_blocks(int kb, int Lq, int Lk, int window, int sinks, int chunk, int far) {
    QBlocks r;
    r.qb0 = 0;
    r.qb1 = (Lq + 127) / 128;
    if (far >= 0) {
        const long long first = sink_far_first(kb, window, chunk, far);
        r.qb0 = first < r.qb1 ? (int)first : r.qb1;
        r.qb1 = r.qb1 < r.qb0 + chunk ? r.qb1 : r.qb0 + chunk;
    }
    r.all_valid = sinks > 0 || (long long)Lq - Lk < window;
    if (r.all_valid && r.qb0 < kb) r.qb0 = kb;  // (earlier q blocks see no key of this block)
    return r;
}

// What the CTA does with q block qb of those: 1 it is visited, 0 only if a row of it has no valid key (the weights of such
// a row are 1 / Lk at every key), -1 left out (by this CTA).  shared: the key block is one of the first nb.
TRIATTN_HD int sink_q_state(int qb, int kb, int Lq, int Lk, int window, int sinks, bool all_valid, bool shared, int far) {
    const int q1 = qb * 128 + 128 < Lq ? qb * 128 + 127 : Lq - 1;
    const SinkBlocks sb = sink_blocks(qb * 128, q1, Lk, window, sinks);
    const int st = sb.visited(kb) ? 1 : 0;
    if (st == 0 && all_valid) return -1;
    if (!shared) return st;
    // (by the rule that the far CTAs start by, whatever the number of keys: a window that starts past the last key
    // but within the block's columns is not far)
    const bool is_far = st == 1 && qb >= sink_far_first(kb, window, 0, 0);
    return is_far == (far >= 0) ? st : -1;
}

// The sharing of a problem.  sinks: the number for every sequence, or -1 where the device knows it for each.
TRIATTN_HD SinkSharing sink_sharing(int num_seqs, int total_q, int H, int max_q, int max_k, int window, int sinks) {
    SinkSharing s;
    s.nb = s.chunk = s.chunks = 0;
    if (sinks == 0) return s;
    const int chunk = 8;
    // q blocks of the longest sequence past the reach of its first key block
    const long long nqb = ((long long)max_q + 127) / 128, far = nqb - ((126LL + window) / 128 + 1);
    if (far <= chunk) return s;
    // The first key block's CTA is issued first and walks nqb q blocks; the others, window / 128 + 2 each,
    // keep 152 SMs busy for total_q / 128 * H * (window / 128 + 2) / 152 of them.  Shared where the one
    // is longer than the other.  (8 heads of 64; q blocks of the longest against that number, the backward
    // unshared and shared: 8 sequences of 256 to 2048 tokens, window 512: 16 to 22, 95 and 104 us; 4 of 4096,
    // window 512: 32 to 40, 173 and 179; 8192 + 4484 + 777, window 1024: 64 to 55, 216 and 204; 2 of 8192,
    // window 256: 64 to 27, 220 and 154.)
    const double rest = (double)total_q / 128 * H * ((double)window / 128 + 2) / 152;
    if ((double)nqb < rest) return s;
    // (with a number of sinks for each sequence, the host knows none of them: the first block is shared)
    const long long nb = sinks < 0 ? 1 : ((long long)sinks + 127) / 128, nkb = ((long long)max_k + 127) / 128;
    if (nb > 4) return s;  // (many key blocks see everything: they balance one another)
    // (many short sequences beside a long one: an accumulator larger than dQ's would cost more than it saves)
    if (num_seqs * nb * 2 * 128 > (long long)total_q) return s;
    s.nb = (int)(nb < nkb ? nb : nkb);
    s.chunk = chunk;
    s.chunks = (int)((far + chunk - 1) / chunk);
    return s;
}

}  // namespace triattn
