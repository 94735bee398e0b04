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
// it) and one job: some heads of q, or some of k, or some of v.  A thread keeps one
// unit of one row (rotary.cuh: two vectors, V pairs) with its cos and sin in registers
// and walks the heads.  For an 8-bit cache it walks them twice: first for the
// largest |x| of each head, then to write the codes; the second reading comes from
// L1 / L2.  No two CTAs write the same (page, head), so nothing is ordered by atomics
// (the largest |x| is a maximum of bit patterns: the same in any order).

#include <cuda_fp8.h>

#include "internal.h"
#include "rotary.cuh"

namespace triattn {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxJobHeads = 8;  // heads of one CTA

struct AppendArgs {
    KvAppendParams p;
    int units, runs;        // units per head; pages a sequence can touch
    int job_heads, q_jobs, kv_jobs;  // heads per CTA; CTAs per run for q, and for each of k and v
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

// C: the cache's element type (T itself, or uint8_t for e4m3 codes).
template <typename T, typename C, int V>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const AppendArgs a) {
    constexpr bool kCodes = sizeof(C) == 1;
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

    // The job: kind 0 q, 1 k, 2 v, and its heads.
    int job = blockIdx.y, kind = 0;
    if (job >= a.q_jobs) {
        job -= a.q_jobs;
        kind = 1 + job / a.kv_jobs;
        job -= (kind - 1) * a.kv_jobs;
    }
    const int H = kind == 0 ? p.Hq : p.Hk, h0 = job * a.job_heads, nh = min(a.job_heads, H - h0);
    const bool turn = kind != 2 && p.dim > 0;
    long long page = 0;
    if (kind != 0) {
        page = p.table[(long long)seq * p.max_pages + lp];
        if (page < 0 || page >= p.num_pages) {
            if (threadIdx.x == 0) atomicCAS(p.status, 0, kStatusDevice);
            return;
        }
    }
    const T* src = static_cast<const T*>(kind == 0 ? p.q : kind == 1 ? p.k : p.v);
    const long long rs = kind == 0 ? p.q_rs : kind == 1 ? p.k_rs : p.v_rs;
    const long long* cst = kind == 1 ? p.ks : p.vs;
    C* cache = static_cast<C*>(kind == 1 ? p.k_cache : p.v_cache) + page * cst[0];
    float* scale = kind == 1 ? p.k_scale : p.v_scale;

    // items = rows x units; threads beyond the items take further heads
    const int items = cnt * a.units;
    const int hs = items >= kThreads ? 1 : kThreads / items;
    const int hsub = items >= kThreads ? 0 : threadIdx.x / items;
    const int item0 = items >= kThreads ? threadIdx.x : threadIdx.x - hsub * items;

    __shared__ uint32_t most[kMaxJobHeads];
    __shared__ float inv[kMaxJobHeads], down[kMaxJobHeads];
    if constexpr (kCodes) {
        if (kind != 0) {
            if (threadIdx.x < kMaxJobHeads) most[threadIdx.x] = 0;
            __syncthreads();
        }
    }
    // pass 0: the largest finite |x| of each head; pass 1: write
    for (int pass = (kCodes && kind != 0) ? 0 : 1; pass < 2; ++pass) {
        if (kCodes && kind != 0 && pass == 1) {
            __syncthreads();
            if (threadIdx.x < nh) {
                float* sp = scale + page * p.Hk + h0 + threadIdx.x;
                const int e = scale_exp(most[threadIdx.x]);
                const float need = exp2i(e), before = off0 > 0 ? *sp : 0.f;
                const bool keep = before >= need;  // the page's scale covers the new rows
                inv[threadIdx.x] = keep ? 1.f / before : exp2i(-e);
                down[threadIdx.x] = keep ? 1.f : before * exp2i(-e);
                if (!keep) *sp = need;
            }
            __syncthreads();
            if (off0 > 0) {  // re-code the rows that were there, where a scale has grown
                const int words = p.D / 4;
                for (int i = 0; i < nh; ++i) {
                    if (down[i] == 1.f) continue;
                    C* rows = cache + (long long)(h0 + i) * cst[1];
                    for (int j = threadIdx.x; j < off0 * words; j += kThreads) {
                        const int r = j / words, d = (j - r * words) * 4;
                        uint32_t* w = reinterpret_cast<uint32_t*>(rows + (long long)r * cst[2] + d);
                        const uint32_t x = *w;
                        const __half2 lo(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(x & 0xffffu), __NV_E4M3));
                        const __half2 hi(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(x >> 16), __NV_E4M3));
                        const float2 fl = __half22float2(lo), fh = __half22float2(hi);
                        *w = to_e4m3x2(fl.x * down[i], fl.y * down[i]) |
                             (to_e4m3x2(fh.x * down[i], fh.y * down[i]) << 16);
                    }
                }
            }
        }
        // (every lane of a warp makes the same number of turns: the maxima are reduced over it)
        for (int base = 0; base < items; base += kThreads) {
            const bool on = hsub < hs && base + item0 < items;
            const int item = on ? base + item0 : 0;
            const int row = item / a.units, u = item - row * a.units;
            const RotUnit r = rot_unit<V>(u, p.D, p.dim, p.interleaved);
            const bool rot = turn && r.pair0 >= 0;
            float cs[V], sn[V];
            if (rot) {
                const int pos = p.positions ? p.positions[tok0 + row] : s0 + row;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float2 t = rotary_cos_sin(pos, p.turns[r.pair0 + i]);
                    cs[i] = t.x * p.mscale;
                    sn[i] = t.y * p.mscale;
                }
            }
            const T* srow = src + (tok0 + row) * rs + (long long)h0 * p.D;
            for (int i = hs == 1 ? 0 : hsub; i < nh; i += hs) {
                if (hs > 1 && !on) break;
                float x0[V], x1[V];
                rot_load<T, V>(srow + (long long)i * p.D + r.o0, x0);
                if (r.o1 >= 0) rot_load<T, V>(srow + (long long)i * p.D + r.o1, x1);
                if (rot) rot_turn<V>(x0, x1, cs, sn, p.interleaved);
                if (kind == 0) {
                    if (!on) continue;
                    T* dst = static_cast<T*>(p.q_out) + (tok0 + row) * p.qo_rs + (long long)(h0 + i) * p.D;
                    rot_store<T, V>(dst + r.o0, x0);
                    if (r.o1 >= 0) rot_store<T, V>(dst + r.o1, x1);
                    continue;
                }
                C* dst = cache + (long long)(h0 + i) * cst[1] + (long long)(off0 + row) * cst[2];
                if constexpr (!kCodes) {
                    if (!on) continue;
                    rot_store<C, V>(dst + r.o0, x0);
                    if (r.o1 >= 0) rot_store<C, V>(dst + r.o1, x1);
                } else if (pass == 0) {
                    uint32_t m = 0;
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        const uint32_t b0 = __float_as_uint(x0[j]) & 0x7fffffffu;
                        const uint32_t b1 = r.o1 >= 0 ? __float_as_uint(x1[j]) & 0x7fffffffu : 0u;
                        if (b0 < 0x7f800000u) m = max(m, b0);
                        if (b1 < 0x7f800000u) m = max(m, b1);
                    }
                    if (hs == 1) {  // every lane of the warp is here, with the same head
                        m = __reduce_max_sync(0xffffffffu, on ? m : 0u);
                        if ((threadIdx.x & 31) == 0) atomicMax(&most[i], m);
                    } else {
                        atomicMax(&most[i], m);
                    }
                } else if (on) {
                    const float iv = inv[i];
                    RotVec<C, V> c0, c1;
                    if constexpr (V == 1) {
                        c0.e[0] = (C)to_e4m3x2(x0[0] * iv, 0.f);
                        c1.e[0] = (C)to_e4m3x2(x1[0] * iv, 0.f);
                    } else {
#pragma unroll
                        for (int j = 0; j < V; j += 2) {
                            const uint32_t w0 = to_e4m3x2(x0[j] * iv, x0[j + 1] * iv);
                            c0.e[j] = (C)w0;
                            c0.e[j + 1] = (C)(w0 >> 8);
                            const uint32_t w1 = to_e4m3x2(x1[j] * iv, x1[j + 1] * iv);
                            c1.e[j] = (C)w1;
                            c1.e[j + 1] = (C)(w1 >> 8);
                        }
                    }
                    *reinterpret_cast<RotVec<C, V>*>(dst + r.o0) = c0;
                    if (r.o1 >= 0) *reinterpret_cast<RotVec<C, V>*>(dst + r.o1) = c1;
                }
            }
        }
    }
}

template <typename T, typename C, int V>
cudaError_t launch(const KvAppendParams& p, cudaStream_t stream) {
    AppendArgs a;
    a.p = p;
    a.units = rot_units<V>(p.D, p.dim);
    a.runs = (p.max_n + p.page - 1) / p.page + 1;
    if (p.max_n == 1) a.runs = 1;
    a.job_heads = kMaxJobHeads;
    a.q_jobs = p.q ? (p.Hq + a.job_heads - 1) / a.job_heads : 0;
    a.kv_jobs = (p.Hk + a.job_heads - 1) / a.job_heads;
    const long long gx = (long long)p.num_seqs * a.runs, gy = a.q_jobs + 2LL * a.kv_jobs;
    if (gx > 0x7fffffffLL || gy > 65535) return cudaErrorInvalidConfiguration;
    kv_append_kernel<T, C, V><<<dim3((unsigned)gx, (unsigned)gy), kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

template <typename T, int V>
cudaError_t launch_t(const KvAppendParams& p, cudaStream_t stream) {
    const bool codes = p.cache_dtype == TA_E4M3;
    if (p.dim % (2 * V) == 0) return codes ? launch<T, uint8_t, V>(p, stream) : launch<T, T, V>(p, stream);
    return codes ? launch<T, uint8_t, 1>(p, stream) : launch<T, T, 1>(p, stream);
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendParams& p, cudaStream_t stream) {
    switch (p.dtype) {
    case TA_F32: return launch_t<float, 4>(p, stream);
    case TA_F16: return launch_t<__half, 8>(p, stream);
    default: return launch_t<__nv_bfloat16, 8>(p, stream);
    }
}

}  // namespace triattn
