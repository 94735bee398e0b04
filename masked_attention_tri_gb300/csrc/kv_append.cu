// kv_append.cu -- new keys and values of packed sequences into the pages of a
// cache, with the rotation of k (and of q) on the way, and to 8 bits with one
// power-of-two scale for each (page, head) where the cache is e4m3.
//
// 8-bit pages.  A page of one head stands for code * scale, scale = 2^e the smallest
// power of two with max |x| <= 448 scale over the page (-56 <= e <= 56).  A power of
// two costs e4m3 no precision (it only moves the exponent) and makes the change of a
// scale exact: when new rows need a larger scale than the page has, the rows that are
// there are re-coded by a shift of their exponents, which rounds only those that fall below
// the least normal code.  The first row of a page starts a new scale, whatever the
// page held before.
//
// Bound: memory.  One CTA takes one page of one sequence (the rows of this call in
// it) and one job: some heads of q, or some of k, or some of v.  As in rotary.cu a thread
// keeps one unit (two vectors) of a row, and cos and sin of the rows' pairs lie in a table in
// shared memory, computed once for the job's heads.  Codes need the largest |x| of a page's rows
// before the first is written: as many rows as 512 units hold stay in registers between the
// two (64 rows of D = 128: a page of the usual size is read once); larger pages are read twice.
// No two CTAs write the same (page, head), so nothing is ordered by atomics (the largest |x| is a maximum
// of bit patterns: the same in any order).
//   Eight prompts of 256 to 2048 tokens, 32 + 8 heads of 128, pages of 64 in 8 bits: 54 us.

#include <cuda_fp8.h>

#include "internal.h"
#include "rotary.cuh"
#include "tc_kernel.cuh"

namespace triattn {
namespace {

constexpr int kThreads = 256;
constexpr int kHold = 2;         // units a thread holds (codes) or has in flight
constexpr int kMaxHeads = 32;    // heads of one CTA, at most

struct AppendArgs {
    KvAppendParams p;
    int units, lanes;            // units per head; rows (or heads) that the CTA's threads take at once
    int runs;                    // pages a sequence can touch
    int table_rows;              // rows of the table of cos and sin
    int row_part;                // rows of a CTA where no maxima are needed
    // k, v, q: heads of a CTA (they divide Hk and Hq), parts of a page's rows, CTAs of a page
    int heads[3], parts[3], jobs[3];
    tc::FastDiv fd[3];           // heads
};

__device__ __forceinline__ uint32_t to_e4m3x2(float a, float b) {
    // An infinity has no code: it becomes NaN, like NaN itself, and stays in its own element.
    a = fabsf(a) <= 3.402823466e38f ? a : __int_as_float(0x7fffffff);
    b = fabsf(b) <= 3.402823466e38f ? b : __int_as_float(0x7fffffff);
    return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

// log2 of the scale for rows of largest magnitude `most` (bits of a finite fp32 >= 0):
// 448 = 1.75 * 2^8, so 2^(E - 8) for a significand up to 1.75, else 2^(E - 7).
__device__ __forceinline__ int scale_exp(uint32_t most) {
    const int e = (int)(most >> 23) - 127 - 8 + ((most & 0x7fffffu) > 0x600000u ? 1 : 0);
    return e < -56 ? -56 : (e > 56 ? 56 : e);
}
__device__ __forceinline__ float exp2i(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// A unit as codes: its first vector at p, its second o1 further on.
template <int V>
__device__ __forceinline__ void store_codes(uint8_t* p, int o1, const float2 (&f)[V], float inv) {
    if constexpr (V == 1) {
        const uint32_t w = to_e4m3x2(f[0].x * inv, f[0].y * inv);
        p[0] = (uint8_t)w;
        if (o1 >= 0) p[o1] = (uint8_t)(w >> 8);
    } else {
        uint32_t w[V / 2];
#pragma unroll
        for (int i = 0; i < V / 2; ++i)
            w[i] = to_e4m3x2(f[2 * i].x * inv, f[2 * i].y * inv) |
                   (to_e4m3x2(f[2 * i + 1].x * inv, f[2 * i + 1].y * inv) << 16);
        if constexpr (V == 8) {
            *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
            if (o1 >= 0) *reinterpret_cast<uint2*>(p + o1) = make_uint2(w[2], w[3]);
        } else {
            *reinterpret_cast<uint32_t*>(p) = w[0];
            if (o1 >= 0) *reinterpret_cast<uint32_t*>(p + o1) = w[1];
        }
    }
}

// The bits of the largest finite magnitude of a unit.
template <int V>
__device__ __forceinline__ uint32_t largest(const float2 (&f)[V]) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const uint32_t a = __float_as_uint(f[i].x) & 0x7fffffffu, b = __float_as_uint(f[i].y) & 0x7fffffffu;
        if (a < 0x7f800000u) m = max(m, a);
        if (b < 0x7f800000u) m = max(m, b);
    }
    return m;
}

// C: the cache's element type (T itself, or uint8_t for e4m3 codes).
template <typename T, typename C, int V>
__global__ void __launch_bounds__(kThreads, 4) kv_append_kernel(const AppendArgs a) {
    constexpr bool kCodes = sizeof(C) == 1;
    extern __shared__ float4 table4[];
    float* table = reinterpret_cast<float*>(table4);
    __shared__ uint32_t most[kMaxHeads];
    __shared__ float before[kMaxHeads];
    const KvAppendParams& p = a.p;
    const int seq = blockIdx.x / a.runs, run = blockIdx.x % a.runs;
    const int row0 = p.cu ? p.cu[seq] : seq, row1 = p.cu ? p.cu[seq + 1] : seq + 1;
    const int len = p.kv_len[seq];
    if (row1 == row0) return;
    if (row0 < 0 || row1 < row0 || row1 > p.total || row1 - row0 > p.max_n || len < row1 - row0 ||
        len > (long long)p.max_pages * p.page) {
        if (run == 0 && blockIdx.y == 0 && threadIdx.x == 0) atomicCAS(p.status, 0, kStatusDevice);
        return;
    }
    const int start = len - (row1 - row0);
    const int lp = start / p.page + run;                       // logical page of the sequence
    const long long slot0 = (long long)lp * p.page;
    const int s0 = (int)max((long long)start, min(slot0, (long long)len));
    const int s1 = (int)min(slot0 + p.page, (long long)len);
    if (s0 >= s1) return;
    const int cnt = s1 - s0, off0 = (int)(s0 - slot0);         // rows of this call; first slot in the page
    const long long tok0 = (long long)row0 + (s0 - start);

    // The job: kind 0 k, 1 v, 2 q (the longest CTAs, whole pages of codes, are issued first), and its heads.
    int job = blockIdx.y, kind = 0;
    while (job >= a.jobs[kind]) job -= a.jobs[kind++];
    const int part = job % a.parts[kind], nh = a.heads[kind], h0 = job / a.parts[kind] * nh;
    long long page = 0;
    if (kind != 2) {
        page = p.table[(long long)seq * p.max_pages + lp];
        if (page < 0 || page >= p.num_pages) {
            if (threadIdx.x == 0) atomicCAS(p.status, 0, kStatusDevice);
            return;
        }
    }
    const T* src = static_cast<const T*>(kind == 0 ? p.k : kind == 1 ? p.v : p.q);
    const long long rs = kind == 0 ? p.k_rs : kind == 1 ? p.v_rs : p.q_rs;
    const long long* cst = kind == 0 ? p.ks : p.vs;
    C* cache = static_cast<C*>(kind == 0 ? p.k_cache : p.v_cache) + page * cst[0];

    // This thread's unit, and the rows' table.
    const int hl = threadIdx.x / a.units, u = threadIdx.x - hl * a.units;
    const bool in = hl < a.lanes;
    const RotUnit r = rot_unit<V>(u, p.D, p.dim, p.interleaved);
    const int np = p.dim / 2, nr = np / V;
    const bool turn = kind != 1 && p.dim > 0, turned = turn && r.turned;
    const int hold = a.lanes * kHold;                          // rows that the CTA's registers hold
    src += tok0 * rs + (long long)h0 * p.D + r.o0;
    auto fill = [&](int c0, int rows) {
        if (!turn) return;
        __syncthreads();
        for (int e = threadIdx.x; e < rows * np; e += kThreads) {
            const int t = e / np, i = e - t * np;
            const int pos = p.positions ? rotary_position(p.positions, p.axes, p.num_axes, i, p.total, tok0 + c0 + t)
                                        : s0 + c0 + t;
            const float2 cs = rotary_cos_sin(pos, p.turns[i]);
            rot_table_put<V>(table, t, i, nr, cs.x * p.mscale, cs.y * p.mscale);
        }
        __syncthreads();
    };
    auto turned_floats = [&](const RotRaw<T, V>& w, int row, float2 (&f)[V]) {
        rot_floats<T, V>(w, f);
        if (turned) rot_turn<V>(f, rot_table_at<V>(table, row, u, nr), nr, p.interleaved);
    };

    if (!kCodes || kind == 2) {
        // ---- q, and caches of the inputs' type: some rows of the page, rows and heads in the order of memory.
        const int c0 = part * a.row_part;
        if (c0 < cnt) {
            const int rows = min(a.row_part, cnt - c0);
            fill(c0, rows);
            if (!in) return;
            for (int n0 = hl; n0 < rows * nh; n0 += hold) {
                RotRaw<T, V> w[kHold];
                int row[kHold], head[kHold];
#pragma unroll
                for (int j = 0; j < kHold; ++j) {
                    const int n = n0 + j * a.lanes;
                    if (n >= rows * nh) break;
                    row[j] = (int)a.fd[kind].div((uint32_t)n);
                    head[j] = n - row[j] * nh;
                    w[j].load(src + (c0 + row[j]) * rs + head[j] * p.D, r.o1);
                }
#pragma unroll
                for (int j = 0; j < kHold; ++j) {
                    if (n0 + j * a.lanes >= rows * nh) break;
                    if (turned) {
                        float2 f[V];
                        turned_floats(w[j], row[j], f);
                        w[j] = rot_raw<T, V>(f);
                    }
                    if (kind == 2) {
                        w[j].store(static_cast<T*>(p.q_out) + (tok0 + c0 + row[j]) * p.qo_rs +
                                       (long long)(h0 + head[j]) * p.D + r.o0, r.o1);
                    } else if constexpr (!kCodes) {
                        w[j].store(cache + (h0 + head[j]) * cst[1] + (off0 + c0 + row[j]) * cst[2] + r.o0, r.o1);
                    }
                }
            }
        }
        return;
    }

    // ---- Codes.  The heads go in groups that fit the registers, n = head * cnt + row; a page with more rows than
    // that goes head by head, twice over its rows.
    if constexpr (kCodes) {
        float* scale = (kind == 0 ? p.k_scale : p.v_scale) + page * p.Hk + h0;
        if (threadIdx.x < nh) {
            most[threadIdx.x] = 0;
            before[threadIdx.x] = off0 > 0 ? scale[threadIdx.x] : 0.f;
        }
        const bool whole = cnt <= hold;             // the rows stay in registers
        const bool once = cnt <= a.table_rows;      // the table holds them all
        if (once) fill(0, cnt);
        __syncthreads();
        const int group = whole ? min(nh, hold / cnt) : 1;
        for (int g0 = 0; g0 < nh; g0 += group) {
            const int items = min(group, nh - g0) * min(cnt, hold);
            RotRaw<T, V> w[kHold];
            auto split = [&](int j, int& head, int& row) -> bool {
                const int n = hl + j * a.lanes;
                head = group == 1 ? 0 : n / cnt;
                row = n - head * cnt;
                return in && n < items;
            };
            auto load = [&](int c0) {
#pragma unroll
                for (int j = 0; j < kHold; ++j) {
                    int head, row;
                    if (split(j, head, row) && c0 + row < cnt) w[j].load(src + (c0 + row) * rs + (g0 + head) * p.D, r.o1);
                }
            };
            auto maxima = [&](int c0) {
#pragma unroll
                for (int j = 0; j < kHold; ++j) {
                    int head, row;
                    const bool on = split(j, head, row) && c0 + row < cnt;
                    const int t0 = once ? c0 : 0;
                    uint32_t m = 0;
                    if (on) {
                        float2 f[V];
                        turned_floats(w[j], t0 + row, f);
                        m = largest<V>(f);
                    }
                    if (group == 1) {
                        m = __reduce_max_sync(0xffffffffu, m);
                        if (threadIdx.x % 32 == 0) atomicMax(&most[g0], m);
                    } else if (on) {
                        atomicMax(&most[g0 + head], m);
                    }
                }
            };
            // A head's scale: its reciprocal, and the factor on the codes that are there (1: unchanged).
            auto scales = [&](int head, float& inv, float& down, float& need) {
                const int e = scale_exp(most[g0 + head]);
                const float b = before[g0 + head];
                need = exp2i(e);
                const bool keep = b >= need;  // the page's scale covers the new rows
                inv = keep ? 1.f / b : exp2i(-e);
                down = keep ? 1.f : b * exp2i(-e);
            };
            auto write = [&](int c0) {
#pragma unroll
                for (int j = 0; j < kHold; ++j) {
                    int head, row;
                    if (!split(j, head, row) || c0 + row >= cnt) continue;
                    const int t0 = once ? c0 : 0;
                    float2 f[V];
                    turned_floats(w[j], t0 + row, f);
                    float inv, down, need;
                    scales(head, inv, down, need);
                    store_codes<V>(cache + (h0 + g0 + head) * cst[1] + (off0 + c0 + row) * cst[2] + r.o0, r.o1, f, inv);
                }
            };
            for (int c0 = 0; c0 < cnt; c0 += hold) {
                if (!once) fill(c0, min(hold, cnt - c0));
                load(c0);
                maxima(c0);
            }
            __syncthreads();
            // The new scale, and the codes that were there where it has grown.
            for (int i = 0; i < min(group, nh - g0); ++i) {
                float inv, down, need;
                scales(i, inv, down, need);
                if (down == 1.f) continue;
                if (threadIdx.x == 0) scale[g0 + i] = need;
                const int words = p.D / 4;
                C* rows = cache + (h0 + g0 + i) * cst[1];
                for (int j = threadIdx.x; j < off0 * words; j += kThreads) {
                    const int row = j / words, d = (j - row * words) * 4;
                    uint32_t* at = reinterpret_cast<uint32_t*>(rows + row * cst[2] + d);
                    const uint32_t x = *at;
                    const __half2 lo(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(x & 0xffffu), __NV_E4M3));
                    const __half2 hi(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(x >> 16), __NV_E4M3));
                    const float2 fl = __half22float2(lo), fh = __half22float2(hi);
                    *at = to_e4m3x2(fl.x * down, fl.y * down) | (to_e4m3x2(fh.x * down, fh.y * down) << 16);
                }
            }
            if (whole) {
                write(0);
            } else {
                for (int c0 = 0; c0 < cnt; c0 += hold) {
                    if (!once) fill(c0, min(hold, cnt - c0));
                    load(c0);
                    write(c0);
                }
            }
        }
    }
}

// The largest divisor of H that is at most `most`.
int heads_of_job(int H, int most) {
    for (int h = most < H ? most : H; h > 1; --h)
        if (H % h == 0) return h;
    return 1;
}

template <typename T, typename C, int V>
cudaError_t launch(const KvAppendParams& p, cudaStream_t stream) {
    AppendArgs a;
    a.p = p;
    a.units = rot_units<V>(p.D, p.dim);
    a.lanes = kThreads / a.units;  // (a head has at most 128 units)
    a.runs = p.max_n == 1 ? 1 : (p.max_n + p.page - 1) / p.page + 1;
    // Heads of a CTA: the table serves them all (16 rows of a page are work enough); but few for codes of
    // whole pages, which go one after the other.
    const bool few = p.max_n <= 8;
    const bool codes = sizeof(C) == 1;
    a.heads[0] = heads_of_job(p.Hk, codes && !few ? 4 : 16);
    a.heads[1] = heads_of_job(p.Hk, codes && !few ? 2 : 16);
    a.heads[2] = p.q ? heads_of_job(p.Hq, 32) : 1;
    for (int i = 0; i < 3; ++i) a.fd[i] = tc::make_fastdiv((uint32_t)a.heads[i]);
    // The table: a page's rows of this call, or 64 KB of them (twice what the registers hold, at least).
    const int row_bytes = (p.dim / 2) * (int)sizeof(float2);
    int rows = p.page < p.max_n ? p.page : p.max_n;
    if (row_bytes > 0 && rows > (64 << 10) / row_bytes) rows = (64 << 10) / row_bytes;
    a.table_rows = rows;
    a.row_part = rows < 16 ? rows : 16;
    const int parts = ((p.page < p.max_n ? p.page : p.max_n) + a.row_part - 1) / a.row_part;
    for (int i = 0; i < 3; ++i) a.parts[i] = i == 2 || !codes ? parts : 1;
    a.jobs[0] = p.Hk / a.heads[0] * a.parts[0];
    a.jobs[1] = p.Hk / a.heads[1] * a.parts[1];
    a.jobs[2] = p.q ? p.Hq / a.heads[2] * a.parts[2] : 0;
    const long long gx = (long long)p.num_seqs * a.runs, gy = (long long)a.jobs[0] + a.jobs[1] + a.jobs[2];
    if (gx > 0x7fffffffLL || gy > 65535) return cudaErrorInvalidConfiguration;
    const size_t smem = (size_t)rows * row_bytes;
    if (smem > (47 << 10)) {  // (48 KB without the attribute, the maxima and scales of the heads among them)
        const cudaError_t e = cudaFuncSetAttribute(kv_append_kernel<T, C, V>, cudaFuncAttributeMaxDynamicSharedMemorySize, 64 << 10);
        if (e != cudaSuccess) return e;
    }
    kv_append_kernel<T, C, V><<<dim3((unsigned)gx, (unsigned)gy), kThreads, smem, stream>>>(a);
    return cudaGetLastError();
}

template <typename T, int V>
cudaError_t launch_t(const KvAppendParams& p, cudaStream_t stream) {
    const bool codes = p.cache_dtype == TA_E4M3;
    if (p.dim % (2 * V) == 0) return codes ? launch<T, uint8_t, V>(p, stream) : launch<T, T, V>(p, stream);
    return codes ? launch<T, uint8_t, 1>(p, stream) : launch<T, T, 1>(p, stream);
}

}  // namespace

cudaError_t launch_kv_append4(const KvAppendParams& p, cudaStream_t stream);  // kv_append4.cu

cudaError_t launch_kv_append(const KvAppendParams& p, cudaStream_t stream) {
    if (p.cache_dtype == TA_INT4) return launch_kv_append4(p, stream);
    switch (p.dtype) {
    case TA_F32: return launch_t<float, 4>(p, stream);
    case TA_F16: return launch_t<__half, 8>(p, stream);
    default: return launch_t<__nv_bfloat16, 8>(p, stream);
    }
}

}  // namespace triattn
