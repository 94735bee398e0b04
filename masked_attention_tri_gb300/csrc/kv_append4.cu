// kv_append4.cu -- new keys and values of packed sequences into the pages of a 4-bit cache (cache4.cuh), with the rotation of k
// and of q on the way.
//
// Bound: memory, with the arithmetic of the codes close behind: eight prompts of 256 to 2048 tokens, 8 heads of 128, 16.4 us (2.9
// TB/s; 18.6 called from Python; 27 by kv_append.cu's threads of half groups with two divisions an element).  One CTA takes some rows of one page of one
// sequence and one job: some heads of k, of v or of q.  A thread takes a group of 16 elements, or, where the halves of a head
// turn together, a group and its partner half a turn away; so no lane waits for another, a row is read and written once, and
// no two threads write the same byte. cos and sin of the rows' pairs lie in a table in shared memory, computed once for the
// job's heads.

#include "cache4.cuh"
#include "internal.h"
#include "rotary.cuh"
#include "tc_kernel.cuh"

namespace triattn {
namespace {

constexpr int kThreads = 256;    // of a CTA, at most
constexpr int kRows = 16;        // rows of a CTA, at most
constexpr int kMaxHeads = 32;    // heads of a CTA, at most

struct Append4Args {
    KvAppendParams p;
    int runs;                    // pages a sequence can touch
    int both;                    // units that hold two groups, 16 elements from u * 16 and dim / 2 further on
    int units;                   // units of a head
    tc::FastDiv fu, fh[3];       // units; heads of a CTA (k, v, q)
    int heads[3], jobs[3];       // heads of a CTA, CTAs of a page's rows
};

template <typename T>
struct Group {                   // 16 elements as they are in memory
    static constexpr int n = sizeof(T);
    uint4 v[n];
    __device__ __forceinline__ void load(const T* p) {
#pragma unroll
        for (int i = 0; i < n; ++i) v[i] = reinterpret_cast<const uint4*>(p)[i];
    }
    __device__ __forceinline__ void floats(float (&f)[16]) const {
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if constexpr (n == 4) {
                    f[4 * i + j] = __uint_as_float(w[j]);
                } else {
                    const float2 x = rot_unpack(T(), w[j]);
                    f[8 * i + 2 * j] = x.x, f[8 * i + 2 * j + 1] = x.y;
                }
            }
        }
    }
};
template <typename T>
__device__ __forceinline__ void store_group(T* p, const float (&f)[16]) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T); ++i) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if constexpr (sizeof(T) == 4) w[j] = __float_as_uint(f[4 * i + j]);
            else w[j] = rot_pack(T(), make_float2(f[8 * i + 2 * j], f[8 * i + 2 * j + 1]));
        }
        reinterpret_cast<uint4*>(p)[i] = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

template <typename T>
__device__ __forceinline__ void store_codes(uint8_t* codes, uint8_t* scale, const float (&f)[16], float inv) {
    float most = 0.f;  // (a NaN stays)
#pragma unroll
    for (int i = 0; i < 16; i += 2) asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(most) : "f"(most), "f"(fabsf(f[i])), "f"(fabsf(f[i + 1])));
    const uint32_t sc = cache4::scale_code(__float_as_uint(most), inv);
    const cache4::Scale s(cache4::scale_value(sc));
    uint2 w;
    if constexpr (sizeof(T) == 2) {
        w = cache4::codes16(f, inv, s, !(most * inv < 7.484375f * s.s));
    } else {
        uint32_t u[2][8];
#pragma unroll
        for (int i = 0; i < 16; ++i) u[i / 8][i % 8] = cache4::code(f[i] * inv, s) & 15u;
        w = make_uint2(cache4::pack8(u[0]), cache4::pack8(u[1]));
    }
    *reinterpret_cast<uint2*>(codes) = w;
    *scale = (uint8_t)sc;
}

// BOTH: units of two groups (the halves of a head turn together); else each is one.
template <typename T, bool BOTH, int THREADS>
__global__ void __launch_bounds__(THREADS) kv_append4_kernel(const Append4Args a) {
    constexpr int kAhead = (BOTH ? 4 : 8) / (int)sizeof(T);    // units in flight a thread
    extern __shared__ float2 table[];          // cos and sin of (row, pair)
    __shared__ float inv_s[kMaxHeads];         // reciprocals of the heads' factors
    const KvAppendParams& p = a.p;
    const int seq = blockIdx.x / a.runs, run = blockIdx.x % a.runs;
    const int row0 = p.cu ? p.cu[seq] : seq, row1 = p.cu ? p.cu[seq + 1] : seq + 1;
    const int len = p.kv_len[seq];
    if (row1 == row0) return;
    if (row0 < 0 || row1 < row0 || row1 > p.total || row1 - row0 > p.max_n || len < row1 - row0 ||
        len > (long long)p.max_pages * p.page) {
        if (run == 0 && blockIdx.y == 0 && blockIdx.z == 0 && threadIdx.x == 0) atomicCAS(p.status, 0, kStatusDevice);
        return;
    }
    const int start = len - (row1 - row0);
    const int lp = start / p.page + run;                       // logical page of the sequence
    const long long slot0 = (long long)lp * p.page;
    const int s0 = (int)max((long long)start, min(slot0, (long long)len)) + (int)blockIdx.z * kRows;
    const int s1 = (int)min(min(slot0 + p.page, (long long)len), (long long)s0 + kRows);
    if (s0 >= s1) return;
    const int cnt = s1 - s0, off0 = (int)(s0 - slot0);
    const long long tok0 = (long long)row0 + (s0 - start);
    int job = blockIdx.y, kind = 0;                            // 0 k, 1 v, 2 q
    while (job >= a.jobs[kind]) job -= a.jobs[kind++];
    const int nh = a.heads[kind], h0 = job * nh;
    uint8_t *codes0 = nullptr, *scale0 = nullptr;              // of the page's first head of the job
    long long codes_h = 0, scale_h = 0;
    bool bad = false;
    if (kind != 2) {
        const long long page = p.table[(long long)seq * p.max_pages + lp];
        if (page < 0 || page >= p.num_pages) {
            if (threadIdx.x == 0) atomicCAS(p.status, 0, kStatusDevice);
            return;
        }
        codes_h = p.c4.cs[kind][1];
        scale_h = p.c4.ss[kind][1];
        codes0 = p.c4.codes[kind] + page * p.c4.cs[kind][0] + h0 * codes_h;
        scale0 = p.c4.scale[kind] + page * p.c4.ss[kind][0] + h0 * scale_h;
        if (threadIdx.x < nh) {
            const float f = p.c4.factor[kind] ? p.c4.factor[kind][h0 + threadIdx.x] : 1.f;
            bad = !(f >= cache4::kLeastFactor && f <= cache4::kMostFactor);
            inv_s[threadIdx.x] = 1.f / f;
        }
    }
    const bool turn = kind != 1 && p.dim > 0;
    const int np = p.dim / 2;
    if (turn) {
        for (int e = threadIdx.x; e < cnt * np; e += THREADS) {
            const int t = e / np, i = e - t * np;
            const int pos = p.positions ? rotary_position(p.positions, p.axes, p.num_axes, i, p.total, tok0 + t) : s0 + t;
            const float2 cs = rotary_cos_sin(pos, p.turns[i]);
            table[e] = make_float2(cs.x * p.mscale, cs.y * p.mscale);
        }
    }
    if (bad) atomicCAS(p.status, 0, kStatusDevice);
    if (__syncthreads_or(bad)) return;  // a factor out of range: its heads' rows are not written
    const T* src = static_cast<const T*>(kind == 0 ? p.k : kind == 1 ? p.v : p.q) + (long long)h0 * p.D;
    const long long rs = kind == 0 ? p.k_rs : kind == 1 ? p.v_rs : p.q_rs;
    const int items = cnt * nh * a.units;
    struct Place {
        int row, head, at;                                     // the first group's first element
        bool two;
    };
    auto place = [&](int e) {
        Place x;
        const int rh = (int)a.fu.div((uint32_t)e), u = e - rh * a.units;
        x.row = (int)a.fh[kind].div((uint32_t)rh);
        x.head = rh - x.row * nh;
        x.two = BOTH && u < a.both;
        x.at = !BOTH || x.two ? 16 * u : 16 * (u + a.both);
        return x;
    };
    for (int e0 = threadIdx.x; e0 < items; e0 += kAhead * THREADS) {
        Group<T> x[kAhead], y[BOTH ? kAhead : 1];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            if (e0 + j * THREADS >= items) break;
            const Place b = place(e0 + j * THREADS);
            const T* from = src + (tok0 + b.row) * rs + (long long)b.head * p.D + b.at;
            x[j].load(from);
            if (BOTH && b.two) y[BOTH ? j : 0].load(from + np);
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            if (e0 + j * THREADS >= items) break;
            const Place b = place(e0 + j * THREADS);
            float f[16], g[16];
            x[j].floats(f);
            if (BOTH && b.two) y[BOTH ? j : 0].floats(g);
            if (BOTH && turn && b.two) {
                const float2* cs = table + b.row * np + b.at;
#pragma unroll
                for (int i = 0; i < 16; i += 2) {
                    const float2 c0 = cs[i], c1 = cs[i + 1];
                    float2 u = make_float2(f[i], f[i + 1]), w = make_float2(g[i], g[i + 1]);
                    rot_turn2(u, w, make_float4(c0.x, c1.x, c0.y, c1.y), false);
                    f[i] = u.x, f[i + 1] = u.y, g[i] = w.x, g[i + 1] = w.y;
                }
            } else if (!BOTH && turn && b.at < p.dim) {        // interleaved pairs
                const float2* cs = table + b.row * np + b.at / 2;
#pragma unroll
                for (int i = 0; i < 16; i += 4) {
                    const float2 c0 = cs[i / 2], c1 = cs[i / 2 + 1];
                    float2 u = make_float2(f[i], f[i + 1]), w = make_float2(f[i + 2], f[i + 3]);
                    rot_turn2(u, w, make_float4(c0.x, c1.x, c0.y, c1.y), true);
                    f[i] = u.x, f[i + 1] = u.y, f[i + 2] = w.x, f[i + 3] = w.y;
                }
            }
            if (kind == 2) {
                T* to = static_cast<T*>(p.q_out) + (tok0 + b.row) * p.qo_rs + (long long)(h0 + b.head) * p.D + b.at;
                store_group<T>(to, f);
                if (BOTH && b.two) store_group<T>(to + np, g);
                continue;
            }
            const int slot = off0 + b.row;
            uint8_t* codes = codes0 + b.head * codes_h + slot * (p.D / 2) + b.at / 2;
            uint8_t* scale = scale0 + b.head * scale_h + slot * (p.D / 16) + b.at / 16;
            const float inv = inv_s[b.head];
            store_codes<T>(codes, scale, f, inv);
            if (BOTH && b.two) store_codes<T>(codes + np / 2, scale + np / 16, g, inv);
        }
    }
}

// The largest divisor of H that is at most `most`.
int divisor(int H, int most) {
    for (int h = most < H ? most : H; h > 1; --h)
        if (H % h == 0) return h;
    return 1;
}

template <typename T>
cudaError_t launch(const KvAppendParams& p, cudaStream_t stream) {
    Append4Args a;
    a.p = p;
    a.runs = p.max_n == 1 ? 1 : (p.max_n + p.page - 1) / p.page + 1;
    a.both = p.interleaved ? 0 : p.dim / 32;
    a.units = p.D / 16 - a.both;
    a.fu = tc::make_fastdiv((uint32_t)a.units);
    a.heads[0] = divisor(p.Hk, 8);
    a.heads[1] = divisor(p.Hk, 8);
    a.heads[2] = p.q ? divisor(p.Hq, kMaxHeads) : 1;
    for (int i = 0; i < 3; ++i) a.fh[i] = tc::make_fastdiv((uint32_t)a.heads[i]);
    a.jobs[0] = p.Hk / a.heads[0];
    a.jobs[1] = p.Hk / a.heads[1];
    a.jobs[2] = p.q ? p.Hq / a.heads[2] : 0;
    const int most = p.page < p.max_n ? p.page : p.max_n, parts = (most + kRows - 1) / kRows, rows = most < kRows ? most : kRows;
    const long long gx = (long long)p.num_seqs * a.runs, gy = (long long)a.jobs[0] + a.jobs[1] + a.jobs[2];
    if (gx > 0x7fffffffLL || gy > 65535) return cudaErrorInvalidConfiguration;
    const size_t smem = (size_t)rows * (p.dim / 2) * sizeof(float2);  // at most 16 KB
    const dim3 grid((unsigned)gx, (unsigned)gy, (unsigned)parts);
    // Half as many threads where nothing turns and no table is shared (the prompts above: 16.6 us for 18.6; with k and 32
    // heads of q turned 62 for 61).
    if (a.both > 0) kv_append4_kernel<T, true, kThreads><<<grid, kThreads, smem, stream>>>(a);
    else if (p.dim > 0) kv_append4_kernel<T, false, kThreads><<<grid, kThreads, smem, stream>>>(a);
    else kv_append4_kernel<T, false, kThreads / 2><<<grid, kThreads / 2, smem, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_append4(const KvAppendParams& p, cudaStream_t stream) {
    switch (p.dtype) {
    case TA_F32: return launch<float>(p, stream);
    case TA_F16: return launch<__half>(p, stream);
    default: return launch<__nv_bfloat16>(p, stream);
    }
}

}  // namespace triattn
