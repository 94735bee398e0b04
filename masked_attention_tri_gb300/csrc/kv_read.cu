// kv_read.cu -- rows of a paged cache back into packed k and v: of the inputs' type as they are, of 8-bit codes times
// their page's scale, of 4-bit codes times their group's scale and their head's factor (cache4.cuh), rounded once.
//
// Bound: memory.  One CTA takes one page of one sequence (the rows of this call in it) and some heads; a thread takes 16
// codes (or 16 bytes) at a time, with four such pieces in flight.  Neighbouring threads hold a row's pieces and then the
// next slot's, so that a page's codes are read in the order of memory and every row of a head is written whole.  16 contexts of
// 2k to 16k slots, 8 heads of 128: 127 us from 4 bits to bf16 (774 MB, 6.1 TB/s; 164 with conversions one element at a time).

#include <type_traits>

#include "cache4.cuh"
#include "internal.h"
#include "rotary.cuh"
#include "tc_kernel.cuh"

namespace triattn {
namespace {

constexpr int kThreads = 256;
constexpr int kAhead = 4;        // pieces in flight a thread

struct ReadArgs {
    KvReadParams p;
    int runs;                    // pages a sequence can touch
    int heads;                   // heads of a CTA
    int units;                   // pieces of a row
    tc::FastDiv fu;              // units
};

struct Raw {};                   // a cache of the output's own type

// Sixteen 4-bit codes as n * x in 16 bits, for a scale times a factor x (four significant bits) within `reads_fast`: a code put
// into the low bits of a power of two makes 128 + u (bf16) or 16 + u (fp16), u = n + 8, and one fused multiplication and a
// sum give (128 + u) x - 136 x or (16 + u) x - 24 x exactly: 136 x = 17 * 8 x has eight significant bits at most, 24 x six.
__device__ __forceinline__ void fast_values(__nv_bfloat16, uint32_t w, float x, uint32_t (&y)[4]) {
    const __nv_bfloat162 s = __float2bfloat162_rn(x), c = __float2bfloat162_rn(-136.f * x);
    uint32_t v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // codes i and i + 4
        uint32_t t;
        asm("lop3.b32 %0, %1, 0x000f000f, 0x43004300, 0xEA;" : "=r"(t) : "r"(w >> (4 * i)));
        const __nv_bfloat162 z = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&t), s, c);
        v[i] = *reinterpret_cast<const uint32_t*>(&z);
    }
    y[0] = __byte_perm(v[0], v[1], 0x5410), y[1] = __byte_perm(v[2], v[3], 0x5410);
    y[2] = __byte_perm(v[0], v[1], 0x7632), y[3] = __byte_perm(v[2], v[3], 0x7632);
}
__device__ __forceinline__ void fast_values(__half, uint32_t w, float x, uint32_t (&y)[4]) {
    const __half2 s = __float2half2_rn(x), c = __float2half2_rn(-24.f * x);
    uint32_t v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t t;
        asm("lop3.b32 %0, %1, 0x03c003c0, 0x4c004c00, 0xEA;" : "=r"(t) : "r"(i < 2 ? w << (6 - 4 * i) : w >> (4 * i - 6)));
        const __half2 z = __hfma2(*reinterpret_cast<const __half2*>(&t), s, c);
        v[i] = *reinterpret_cast<const uint32_t*>(&z);
    }
    y[0] = __byte_perm(v[0], v[1], 0x5410), y[1] = __byte_perm(v[2], v[3], 0x5410);
    y[2] = __byte_perm(v[0], v[1], 0x7632), y[3] = __byte_perm(v[2], v[3], 0x7632);
}
// A factor that is a power of two, and far enough from what the type holds (scales are 2^-9 to 448).
__device__ __forceinline__ bool reads_fast(__nv_bfloat16, float f) {
    return (__float_as_uint(f) & 0x007fffffu) == 0 && f >= 0x1p-100f && f <= 0x1p100f;
}
__device__ __forceinline__ bool reads_fast(__half, float f) {
    return (__float_as_uint(f) & 0x007fffffu) == 0 && f >= 0x1p-15f && f <= 4.f;
}
__device__ __forceinline__ bool reads_fast(float, float) { return false; }
__device__ __forceinline__ void fast_values(float, uint32_t, float, uint32_t (&)[4]) {}

// The numbers of N floats as T, 16 bytes at a time.
template <typename T, int N>
__device__ __forceinline__ void store_row(T* p, const float (&f)[N]) {
    constexpr int kV = 16 / sizeof(T);
#pragma unroll
    for (int i = 0; i < N; i += kV) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if constexpr (sizeof(T) == 4) w[j] = __float_as_uint(f[i + j]);
            else w[j] = rot_pack(T(), make_float2(f[i + 2 * j], f[i + 2 * j + 1]));
        }
        *reinterpret_cast<uint4*>(p + i) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// S: Raw, uint8_t (e4m3) or cache4::Code.
template <typename T, typename S>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(const ReadArgs a) {
    constexpr bool kRaw = std::is_same<S, Raw>::value, kFour = std::is_same<S, cache4::Code>::value;
    const KvReadParams& p = a.p;
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
    const int lp = start / p.page + run;
    const long long slot0 = (long long)lp * p.page;
    const int s0 = (int)max((long long)start, min(slot0, (long long)len));
    const int s1 = (int)min(slot0 + p.page, (long long)len);
    if (s0 >= s1) return;
    const long long page = p.table[(long long)seq * p.max_pages + lp];
    if (page < 0 || page >= p.num_pages) {
        if (threadIdx.x == 0) atomicCAS(p.status, 0, kStatusDevice);
        return;
    }
    const int cnt = s1 - s0, off0 = (int)(s0 - slot0);
    const long long tok0 = (long long)row0 + (s0 - start);
    const int h0 = blockIdx.y * a.heads, nh = min(a.heads, p.Hk - h0);

    // (16-bit outputs whose rows are 32-byte multiples: a piece is one store)
    const bool wide = sizeof(T) == 2 && ((reinterpret_cast<uintptr_t>(p.out[0]) | reinterpret_cast<uintptr_t>(p.out[1])) & 31) == 0 &&
                      p.rs[0] % 16 == 0 && p.rs[1] % 16 == 0;
    // A warp takes the rows of a head's k or v (or, where there are fewer of those than warps, every `share`th piece of them).
    struct Piece {
        int kind, h, row, u;
    };
    constexpr int kWarps = kThreads / 32;
    const int share = 2 * nh < kWarps ? kWarps / (2 * nh) : 1, warp = threadIdx.x / 32, items = cnt * a.units;
    for (int hh = warp / share; hh < 2 * nh; hh += kWarps)
    for (int e0 = warp % share * 32 + threadIdx.x % 32; e0 < items; e0 += kAhead * 32 * share) {
        auto piece = [&](int e) {
            Piece x;
            x.row = (int)a.fu.div((uint32_t)e);
            x.u = e - x.row * a.units;
            x.kind = hh >= nh;
            x.h = h0 + (x.kind ? hh - nh : hh);
            return x;
        };
        uint4 w[kAhead];
        uint32_t sc[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int e = e0 + j * 32 * share;
            if (e >= items) break;
            const Piece x = piece(e);
            const int slot = off0 + x.row;
            if constexpr (kFour) {
                const uint8_t* c = p.c4.codes[x.kind] + page * p.c4.cs[x.kind][0] + x.h * p.c4.cs[x.kind][1];
                const uint2 y = *reinterpret_cast<const uint2*>(c + (long long)slot * (p.D / 2) + x.u * 8);
                w[j] = make_uint4(y.x, y.y, 0u, 0u);
                sc[j] = p.c4.scale[x.kind][page * p.c4.ss[x.kind][0] + x.h * p.c4.ss[x.kind][1] +
                                           (long long)slot * (p.D / 16) + x.u];
            } else {
                const long long at = page * p.st[x.kind][0] + x.h * p.st[x.kind][1] + slot * p.st[x.kind][2];
                if constexpr (kRaw) w[j] = *reinterpret_cast<const uint4*>(static_cast<const T*>(p.cache[x.kind]) + at + x.u * (16 / (int)sizeof(T)));
                else w[j] = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.cache[x.kind]) + at + x.u * 16);
                if constexpr (!kRaw) sc[j] = __float_as_uint(p.scale[x.kind][page * p.Hk + x.h]);
            }
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int e = e0 + j * 32 * share;
            if (e >= items) break;
            const Piece x = piece(e);
            T* out = static_cast<T*>(p.out[x.kind]) + (tok0 + x.row) * p.rs[x.kind] + (long long)x.h * p.D;
            if constexpr (kRaw) {
                *reinterpret_cast<uint4*>(out + x.u * (16 / (int)sizeof(T))) = w[j];
            } else {
                float f[16];
                const uint32_t ws[4] = {w[j].x, w[j].y, w[j].z, w[j].w};
                if constexpr (kFour) {
                    const float s = cache4::scale_value(sc[j]);
                    const float fac = p.c4.factor[x.kind] ? p.c4.factor[x.kind][x.h] : 1.f;
                    if (reads_fast(T(), fac)) {
                        uint32_t y[2][4];
                        fast_values(T(), ws[0], s * fac, y[0]);
                        fast_values(T(), ws[1], s * fac, y[1]);
                        T* at = out + x.u * 16;
                        if (wide) {
                            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(at), "r"(y[0][0]), "r"(y[0][1]),
                                         "r"(y[0][2]), "r"(y[0][3]), "r"(y[1][0]), "r"(y[1][1]), "r"(y[1][2]), "r"(y[1][3])
                                         : "memory");
                        } else {
                            reinterpret_cast<uint4*>(at)[0] = make_uint4(y[0][0], y[0][1], y[0][2], y[0][3]);
                            reinterpret_cast<uint4*>(at)[1] = make_uint4(y[1][0], y[1][1], y[1][2], y[1][3]);
                        }
                        continue;
                    }
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float v[8];
                        cache4::values8(ws[i], s, v);
#pragma unroll
                        for (int k = 0; k < 8; ++k) f[8 * i + k] = v[k] * fac;
                    }
                } else {
                    const float s = __uint_as_float(sc[j]);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const __half2 h(__nv_cvt_fp8x2_to_halfraw2(
                            (__nv_fp8x2_storage_t)(ws[i / 2] >> (16 * (i % 2)) & 0xffffu), __NV_E4M3));
                        const float2 v = __half22float2(h);
                        f[2 * i] = v.x * s;
                        f[2 * i + 1] = v.y * s;
                    }
                }
                store_row<T, 16>(out + x.u * 16, f);
            }
        }
    }
}

template <typename T, typename S>
cudaError_t launch(const KvReadParams& p, cudaStream_t stream) {
    ReadArgs a;
    a.p = p;
    a.runs = p.max_n == 1 ? 1 : (p.max_n + p.page - 1) / p.page + 1;
    a.units = std::is_same<S, Raw>::value ? p.D * (int)sizeof(T) / 16 : p.D / 16;
    a.fu = tc::make_fastdiv((uint32_t)a.units);
    // As many heads a CTA as leave four CTAs for each of 152 SMs; a CTA's pieces are counted in 31 bits.
    const long long pages = (long long)p.num_seqs * a.runs;
    int heads = p.Hk < 64 ? p.Hk : 64;
    while (heads > 1 && pages * ((p.Hk + heads - 1) / heads) < 152 * 4) heads = (heads + 1) / 2;
    a.heads = heads;
    const long long gy = (p.Hk + heads - 1) / heads;
    if (pages > 0x7fffffffLL || gy > 65535) return cudaErrorInvalidConfiguration;
    kv_read_kernel<T, S><<<dim3((unsigned)pages, (unsigned)gy), kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_t(const KvReadParams& p, cudaStream_t stream) {
    if (p.cache_dtype == TA_INT4) return launch<T, cache4::Code>(p, stream);
    return p.cache_dtype == TA_E4M3 ? launch<T, uint8_t>(p, stream) : launch<T, Raw>(p, stream);
}

}  // namespace

cudaError_t launch_kv_read(const KvReadParams& p, cudaStream_t stream) {
    switch (p.dtype) {
    case TA_F32: return launch_t<float>(p, stream);
    case TA_F16: return launch_t<__half>(p, stream);
    default: return launch_t<__nv_bfloat16>(p, stream);
    }
}

}  // namespace triattn
