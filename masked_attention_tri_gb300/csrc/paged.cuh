// paged.cuh -- attention over a paged cache: the parameter block, the split of the
// work over the CTAs and the joining of split rows, shared by the kernels of
// paged_simt.cu and paged_mma.cu.
//
// O[i, h] = softmax_k(scale q_i . K[k]) V over the keys that token i sees.  The n
// new tokens of a sequence are the last of its `len` slots; token i at position
// p = len - n + i sees slot k when k <= p and, with a window, k > p - window or
// k < sinks.
//
// A unit is up to RT rows of one (sequence, kv head): its n tokens x G grouped query
// heads, row r = token * G + head.  A unit visits the tiles (of p.tile slots) that hold a key one of
// its rows sees: all up to the last row's position, or those of the first `sinks` slots
// and those from the first row's window on.  The units' tiles, in the order
// (sequence, kv head, row tile), form one axis that is cut into equal shares, one
// for each CTA, whatever the sequences' lengths: one long sequence is spread over
// the GPU and a ragged batch is balanced, from lengths that only the device knows.
// A unit that lies in one share is finished by its CTA.  One that is cut leaves for each
// share its unnormalised O with the running maximum m and sum l (base 2), which a
// second kernel joins in the order of the shares: the same result every time.
//
// Scales of 8-bit pages.  Keys: a factor on the logit.  Values: 2^log2(vs) joins the
// exponent, x' = x + log2 vs, so the weights 2^(x' - m') multiply the bare codes and
// their maximum m' is the largest weighted page's; the sum takes 2^(x' - m') / vs.  That wants vs in the range that
// kv_append.cu writes, 2^-56 to 2^56: then no sum passes fp32, and what a weight loses below 2^-126 is less than
// 2^-126 of the ratio of the row's largest and smallest vs (2^-14 of the largest weight at worst).
#pragma once

#include <cuda_fp8.h>

#include "internal.h"
#include "rotary.cuh"

namespace triattn {
namespace paged {

constexpr int kGrid = 152;     // shares (one CTA per SM)
constexpr int kMaxRT = 32;     // rows of a unit, at most

// Workspace: partial O [2 kGrid][RT][D] and (m, l) [2 kGrid][RT] (slot 2c: the unit that reaches
// into share c; 2c + 1: the one that starts in it and goes on), then the join records.
struct Join {
    int parts;                 // shares of the unit that starts in this share and is cut; 0: none
    int seq_row0, h;           // the sequence's first packed row, the kv head
    int row0, rows;            // the unit's first row and how many exist
};
struct Workspace {
    float* o;
    float2* ml;
    Join* join;
};
__host__ __device__ inline size_t workspace_bytes(int RT, int D) {
    return (size_t)2 * kGrid * RT * (D + 2) * 4 + (size_t)kGrid * sizeof(Join);
}
__host__ __device__ inline Workspace workspace(void* ws, int RT, int D) {
    Workspace w;
    w.o = static_cast<float*>(ws);
    w.ml = reinterpret_cast<float2*>(w.o + (size_t)2 * kGrid * RT * D);
    w.join = reinterpret_cast<Join*>(w.ml + (size_t)2 * kGrid * RT);
    return w;
}

// What a sequence gives: n new tokens from packed row row0, len slots.
struct Seq {
    int row0, n, len;
};
__device__ __forceinline__ Seq load_seq(const PagedParams& p, int s, bool tell) {
    Seq q;
    q.row0 = p.cu ? p.cu[s] : s;
    const int row1 = p.cu ? p.cu[s + 1] : s + 1;
    q.len = p.kv_len[s];
    q.n = row1 - q.row0;
    bool bad = false;
    if (q.row0 < 0 || row1 < q.row0 || row1 > p.total_q || q.n > p.max_q) {
        bad = true;
        q.n = 0;
    }
    if (q.len < 0 || q.len > (long long)p.max_pages * p.page) {  // read as holding nothing
        bad = true;
        q.len = 0;
    }
    if (bad && tell) atomicCAS(p.status, 0, kStatusDevice);
    return q;
}

// The tiles of a unit: `nt` of them, tile(j) = j below sink_t, else lo_t + j - sink_t.
struct Tiles {
    int nt, sink_t, lo_t;
    int p0, p1;                // positions of the unit's first and last row
    __device__ __forceinline__ int tile(int j) const { return j < sink_t ? j : lo_t + (j - sink_t); }
};
__device__ __forceinline__ Tiles unit_tiles(const PagedParams& p, const Seq& q, int rt) {
    Tiles t;
    const int r0 = rt * p.RT, r1 = min(q.n * p.G, r0 + p.RT) - 1;
    t.p0 = q.len - q.n + r0 / p.G;
    t.p1 = q.len - q.n + r1 / p.G;
    t.sink_t = t.lo_t = 0;
    t.nt = t.p1 < 0 ? 0 : t.p1 / p.tile + 1;
    if (p.window > 0 && t.p1 >= 0) {
        const long long lo = (long long)t.p0 - p.window + 1;
        const int lo_t = lo > 0 ? (int)(lo / p.tile) : 0;
        const int sink_t = (min(p.sinks, t.p1 + 1) + p.tile - 1) / p.tile;
        if (lo_t > sink_t) {
            t.lo_t = lo_t;
            t.sink_t = sink_t;
            t.nt = sink_t + t.nt - lo_t;
        }
    }
    return t;
}
__device__ __forceinline__ int row_tiles(const PagedParams& p, const Seq& q) { return (q.n * p.G + p.RT - 1) / p.RT; }
// (These walk the row tiles one by one: made for sequences with few new rows.  8192 new tokens in one call are 2048 row
// tiles of 16 rows, 4 heads a group, and every CTA walks them before its first load.)
// Tiles of one kv head of a sequence (a unit without keys counts one: its rows are written too).
__device__ __forceinline__ long long head_tiles(const PagedParams& p, const Seq& q) {
    long long t = 0;
    for (int rt = 0; rt < row_tiles(p, q); ++rt) t += max(1, unit_tiles(p, q, rt).nt);
    return t;
}

// A token at position pos sees slot key.
__device__ __forceinline__ bool sees(const PagedParams& p, int pos, int key) {
    return key <= pos && (p.window <= 0 || pos - key < p.window || key < p.sinks);
}
// Some row of the unit sees the slot (positions p0 to p1).
__device__ __forceinline__ bool unit_sees(const PagedParams& p, const Tiles& t, int key) {
    return key <= t.p1 && (p.window <= 0 || (long long)t.p0 - key < p.window || key < p.sinks);
}

// A value scale that the kernels take (a NaN is none).
__device__ __forceinline__ bool v_scale_ok(float vs) { return vs >= 0x1p-56f && vs <= 0x1p56f; }

// The CTA's share: tiles [begin, end) of the axis and the unit that begin falls in.  Every
// thread of the block calls it; scan is shared scratch of one long long a warp.
struct Share {
    long long begin, end, per;
    int seq;                   // sequence of tile `begin`
    long long in_seq;          // its place among the sequence's tiles
};
template <int THREADS>
__device__ Share find_share(const PagedParams& p, int min_tiles, long long* scan, long long* found) {
    constexpr int kW = THREADS / 32;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    auto block_sum = [&](long long v, long long& before) -> long long {  // exclusive prefix and total
        long long x = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        __syncthreads();
        if (lane == 31) scan[warp] = x;
        __syncthreads();
        long long base = 0, total = 0;
#pragma unroll
        for (int w = 0; w < kW; ++w) {
            if (w < warp) base += scan[w];
            total += scan[w];
        }
        before = base + x - v;
        return total;
    };
    Share sh;
    long long total = 0, before, w0 = 0;
    for (int s0 = 0; s0 < p.num_seqs; s0 += THREADS) {
        const int s = s0 + threadIdx.x;
        long long w = 0;
        if (s < p.num_seqs) w = head_tiles(p, load_seq(p, s, blockIdx.x == 0)) * p.Hk;
        if (s0 == 0) w0 = w;
        total += block_sum(w, before);
    }
    sh.per = (total + kGrid - 1) / kGrid;
    if (sh.per < min_tiles) sh.per = min_tiles;
    sh.begin = (long long)blockIdx.x * sh.per;
    sh.end = min(sh.begin + sh.per, total);
    if (threadIdx.x == 0) found[0] = -1;
    long long at = 0;
    for (int s0 = 0; s0 < p.num_seqs && at <= sh.begin; s0 += THREADS) {
        const int s = s0 + threadIdx.x;
        long long w = 0;
        if (s < p.num_seqs) w = s0 == 0 ? w0 : head_tiles(p, load_seq(p, s, false)) * p.Hk;
        const long long n = block_sum(w, before);
        if (w > 0 && at + before <= sh.begin && sh.begin < at + before + w) {
            found[0] = s;
            found[1] = sh.begin - at - before;
        }
        at += n;
    }
    __syncthreads();
    sh.seq = (int)found[0];
    sh.in_seq = found[1];
    if (sh.begin >= sh.end) sh.seq = -1;
    return sh;
}

// The walk over the share's units, the same in every thread.
struct Unit {
    Seq q;
    Tiles t;
    int seq, h, rt;
    int j0, j1;                // its tiles in this share: [j0, j1)
    bool starts, ends;         // the unit's first / last tile is in this share
    int rows;                  // rows that exist
};
struct Walk {
    long long left;            // tiles of the share still to go
    long long skip;            // tiles of the current sequence before the next unit's first tile
    int seq, h, rt;
    bool fresh;
    Seq q;
};
__device__ __forceinline__ Walk walk_begin(const PagedParams& p, const Share& sh) {
    Walk w;
    w.left = sh.seq < 0 ? 0 : sh.end - sh.begin;
    w.seq = sh.seq;
    w.skip = sh.in_seq;
    w.h = w.rt = 0;
    w.fresh = true;
    return w;
}
__device__ __forceinline__ bool walk_next(const PagedParams& p, Walk& w, Unit& u) {
    if (w.left <= 0) return false;
    if (w.fresh) {
        w.fresh = false;
        w.q = load_seq(p, w.seq, false);
        const long long ht = head_tiles(p, w.q);
        w.h = (int)(w.skip / ht);
        w.skip -= w.h * ht;
    }
    for (;;) {
        if (w.rt >= row_tiles(p, w.q)) {
            w.rt = 0;
            if (w.q.n == 0 || ++w.h >= p.Hk) {
                w.h = 0;
                if (++w.seq >= p.num_seqs) return false;
                w.q = load_seq(p, w.seq, false);
                continue;
            }
        }
        u.t = unit_tiles(p, w.q, w.rt);
        const int nt = max(1, u.t.nt);
        if (w.skip >= nt) {
            w.skip -= nt;
            ++w.rt;
            continue;
        }
        u.q = w.q;
        u.seq = w.seq;
        u.h = w.h;
        u.rt = w.rt;
        u.j0 = (int)w.skip;
        u.j1 = (int)min((long long)nt, u.j0 + w.left);
        u.starts = u.j0 == 0;
        u.ends = u.j1 == nt;
        u.rows = min(p.RT, w.q.n * p.G - w.rt * p.RT);
        w.left -= u.j1 - u.j0;
        w.skip = 0;
        ++w.rt;
        return true;
    }
}

// The shares that unit u reaches over, from the one that it starts in (this one).
__device__ __forceinline__ int unit_parts(const Share& sh, const Unit& u, long long u_begin) {
    const long long last = u_begin + max(1, u.t.nt) - 1;
    return (int)(last / sh.per - blockIdx.x) + 1;
}

__device__ __forceinline__ void store_out(const PagedParams& p, long long i, float v) {
    if (p.dtype == TA_F32) static_cast<float*>(p.out)[i] = v;
    else if (p.dtype == TA_F16) static_cast<__half*>(p.out)[i] = __float2half_rn(v);
    else static_cast<__nv_bfloat16*>(p.out)[i] = __float2bfloat16_rn(v);
}

// A row (or a part of it) that has seen no key.  (A maximum passes over NaN, so a row
// of NaN logits has m = -inf too; its sum is NaN and not 0.)
__device__ __forceinline__ bool no_key(float m, float l) { return m == -INFINITY && l == 0.f; }

// log-sum-exp of a row (natural units) from base-2 m and l; no key: -inf.
__device__ __forceinline__ float row_lse(float m, float l) {
    return no_key(m, l) ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

// Joins the split units (paged_simt.cu), after the kernel that left their parts.
cudaError_t launch_join(const PagedParams& p, cudaStream_t stream);
cudaError_t launch_simt(const PagedParams& p, cudaStream_t stream);
// 16-bit queries on tensor cores (paged_mma*.cu).
cudaError_t launch_mma(const PagedParams& p, cudaStream_t stream);

}  // namespace paged
}  // namespace triattn
