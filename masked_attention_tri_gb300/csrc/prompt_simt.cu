// prompt_simt.cu -- causal attention of packed prompts with grouped heads, forward and backward, on CUDA cores in exact
// fp32: fp32 inputs, and 16-bit ones with D > 128.
//
// Tiles of BM rows (tokens x grouped heads, prompt.cuh) and 64 keys in shared memory as fp32, 256 threads.  A thread forms
// a BM / 16 x 4 piece of the logits from vectors of four columns (16 FMAs for two shared loads) and holds as many rows of
// the result by D / 16 columns.  Bound: shared-memory loads beside the FMAs.  The backward runs two kernels, one for each
// tile of keys (dK, dV) and one for each tile of rows (dQ): both form P and dP, no sum is left to atomics, and the order of
// every sum is fixed.

#include <type_traits>

#include "prompt.cuh"
#include "tc_kernel.cuh"

namespace triattn {
namespace prompt {
namespace {

constexpr int kThreads = 256, kKeys = 64, kLP = kKeys + 4;  // (rows of P are kLP floats apart)

template <typename T>
struct Vec;
template <>
struct Vec<float> {
    static constexpr int n = 4;
    static __device__ __forceinline__ void load(const float* p, float (&f)[4]) {
        const float4 v = *reinterpret_cast<const float4*>(p);
        f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
    }
};
template <typename T>
struct Vec {
    static constexpr int n = 8;
    static __device__ __forceinline__ void load(const T* p, float (&f)[8]) {
        const uint4 v = *reinterpret_cast<const uint4*>(p);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 x = rot_unpack(T(), w[i]);
            f[2 * i] = x.x, f[2 * i + 1] = x.y;
        }
    }
};

// ROWS rows of D columns as fp32, rows LD floats apart; at(r): the row's address, or NULL (zeros).
template <typename T, int ROWS, int LD, typename At>
__device__ __forceinline__ void load_tile(float* dst, int D, At at) {
    constexpr int kV = Vec<T>::n, kPer = (LD - 4) / kV;
    for (int e = threadIdx.x; e < ROWS * kPer; e += kThreads) {
        const int r = e / kPer, d = (e - r * kPer) * kV;
        const T* p = d < D ? at(r) : nullptr;
        float f[kV];
        if (p) {
            Vec<T>::load(p + d, f);
        } else {
#pragma unroll
            for (int i = 0; i < kV; ++i) f[i] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < kV; i += 4)
            *reinterpret_cast<float4*>(dst + r * LD + d + i) = make_float4(f[i], f[i + 1], f[i + 2], f[i + 3]);
    }
}

// s[i][j] = a[ty RM + i] . b[tx + 16 j]
template <int RM, int LD>
__device__ __forceinline__ void products(const float* a, const float* b, int D, float (&s)[RM][4]) {
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
#pragma unroll
    for (int i = 0; i < RM; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll 4
    for (int d = 0; d < D; d += 4) {
        float4 x[RM], y[4];
#pragma unroll
        for (int i = 0; i < RM; ++i) x[i] = *reinterpret_cast<const float4*>(a + (ty * RM + i) * LD + d);
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = *reinterpret_cast<const float4*>(b + (tx + 16 * j) * LD + d);
#pragma unroll
        for (int i = 0; i < RM; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s[i][j] = fmaf(x[i].x, y[j].x, s[i][j]);
                s[i][j] = fmaf(x[i].y, y[j].y, s[i][j]);
                s[i][j] = fmaf(x[i].z, y[j].z, s[i][j]);
                s[i][j] = fmaf(x[i].w, y[j].w, s[i][j]);
            }
    }
}

// o[i][c] += sum_k p[row i][k] b[k][64 c + 4 tx ...]: rows of p in shared memory (by row), 64 of k.
template <int RM, int NC, int LD>
__device__ __forceinline__ void add_rows(const float* p, const float* b, float4 (&o)[RM][NC]) {
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
#pragma unroll 2
    for (int k = 0; k < kKeys; k += 4) {
        float4 w[RM];
#pragma unroll
        for (int i = 0; i < RM; ++i) w[i] = *reinterpret_cast<const float4*>(p + (ty * RM + i) * kLP + k);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                const float4 y = *reinterpret_cast<const float4*>(b + (k + kk) * LD + 64 * c + 4 * tx);
#pragma unroll
                for (int i = 0; i < RM; ++i) {
                    const float x = kk == 0 ? w[i].x : kk == 1 ? w[i].y : kk == 2 ? w[i].z : w[i].w;
                    o[i][c].x = fmaf(x, y.x, o[i][c].x);
                    o[i][c].y = fmaf(x, y.y, o[i][c].y);
                    o[i][c].z = fmaf(x, y.z, o[i][c].z);
                    o[i][c].w = fmaf(x, y.w, o[i][c].w);
                }
            }
    }
}

// o[i][c] += sum_r p[r][key 4 ty + i] b[r][64 c + 4 tx ...]: BM rows.
template <int BM, int NC, int LD>
__device__ __forceinline__ void add_cols(const float* p, const float* b, float4 (&o)[4][NC]) {
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
#pragma unroll 4
    for (int r = 0; r < BM; ++r) {
        const float4 w = *reinterpret_cast<const float4*>(p + r * kLP + 4 * ty);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const float4 y = *reinterpret_cast<const float4*>(b + r * LD + 64 * c + 4 * tx);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float x = i == 0 ? w.x : i == 1 ? w.y : i == 2 ? w.z : w.w;
                o[i][c].x = fmaf(x, y.x, o[i][c].x);
                o[i][c].y = fmaf(x, y.y, o[i][c].y);
                o[i][c].z = fmaf(x, y.z, o[i][c].z);
                o[i][c].w = fmaf(x, y.w, o[i][c].w);
            }
        }
    }
}

template <typename T>
__device__ __forceinline__ void store4(T* p, float4 v, float by) {
    if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<float4*>(p) = make_float4(v.x * by, v.y * by, v.z * by, v.w * by);
    } else {
        *reinterpret_cast<uint2*>(p) = make_uint2(rot_pack(T(), make_float2(v.x * by, v.y * by)),
                                                  rot_pack(T(), make_float2(v.z * by, v.w * by)));
    }
}

// The tile of the block: the longest rows first.  (sequence, key head, tile of rows or keys)
struct Place {
    int tile, h, seq;
};
__device__ __forceinline__ Place place(const PromptParams& p, int tiles, bool last_first) {
    Place x;
    const unsigned per = (unsigned)p.num_seqs * (unsigned)p.Hk;
    x.tile = (int)(blockIdx.x / per);
    const unsigned rest = blockIdx.x % per;
    if (last_first) x.tile = tiles - 1 - x.tile;
    x.seq = (int)(rest / (unsigned)p.Hk);
    x.h = (int)(rest % (unsigned)p.Hk);
    return x;
}

// Row r of the tile at row0: its address in a (total, Hq, D) tensor of rows rs apart.
template <typename T>
__device__ __forceinline__ const T* row_at(const PromptParams& p, const Seq& q, int h, int r, const void* base, long long rs) {
    if (r >= q.lq * p.G) return nullptr;
    return static_cast<const T*>(base) + (long long)(q.q0 + r / p.G) * rs + (long long)(h * p.G + r % p.G) * p.D;
}
template <typename T>
__device__ __forceinline__ const T* key_at(const PromptParams& p, const Seq& q, int h, int k, const void* base, long long rs) {
    return k < q.lk ? static_cast<const T*>(base) + (long long)(q.k0 + k) * rs + (long long)h * p.D : nullptr;
}

template <typename T, int NC>
__global__ void __launch_bounds__(kThreads) prompt_fwd_simt(const PromptParams p, int tiles) {
    constexpr int BM = 64, RM = 4, LD = 64 * NC + 4;
    extern __shared__ float smem[];
    float *sq = smem, *sk = sq + BM * LD, *sv = sk + kKeys * LD, *sp = sk;  // (P over K, which is read by then)
    const Place x = place(p, tiles, true);
    const Seq q = load_seq(p, x.seq, threadIdx.x == 0 && x.tile == 0 && x.h == 0);
    const int rows = q.lq * p.G, r0 = x.tile * BM, ty = threadIdx.x / 16, tx = threadIdx.x % 16;
    if (r0 >= rows) return;
    load_tile<T, BM, LD>(sq, p.D, [&](int r) { return row_at<T>(p, q, x.h, r0 + r, p.q, p.q_rs); });
    int limit[RM];             // the last key that a row sees
    float m[RM], l[RM];
    float4 o[RM][NC];
#pragma unroll
    for (int i = 0; i < RM; ++i) {
        const int r = r0 + ty * RM + i;
        limit[i] = r < rows ? r / p.G + q.shift : -1;
        m[i] = -INFINITY, l[i] = 0.f;
#pragma unroll
        for (int c = 0; c < NC; ++c) o[i][c] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    const int last = min(r0 + BM, rows) - 1, keys = last / p.G + q.shift + 1;  // keys that some row sees
    const float f = p.scale * kToLog2;
    for (int k0 = 0; k0 < keys; k0 += kKeys) {
        __syncthreads();
        load_tile<T, kKeys, LD>(sk, p.D, [&](int k) { return k0 + k < keys ? key_at<T>(p, q, x.h, k0 + k, p.k, p.k_rs) : nullptr; });
        load_tile<T, kKeys, LD>(sv, p.D, [&](int k) { return k0 + k < keys ? key_at<T>(p, q, x.h, k0 + k, p.v, p.v_rs) : nullptr; });
        __syncthreads();
        float s[RM][4];
        products<RM, LD>(sq, sk, p.D, s);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < RM; ++i) {
            float mt = m[i];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s[i][j] = k0 + tx + 16 * j <= limit[i] ? s[i][j] * f : -INFINITY;
                mt = fmaxf(mt, s[i][j]);
            }
#pragma unroll
            for (int w = 1; w < 16; w <<= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, w));
            // (a row that has seen no key, or NaN alone, keeps -inf)
            const float ref = mt == -INFINITY ? 0.f : mt, alpha = exp2f(m[i] - ref);
            m[i] = mt;
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float pr = exp2f(s[i][j] - ref);
                sp[(ty * RM + i) * kLP + tx + 16 * j] = pr;
                sum += pr;
            }
            l[i] = fmaf(l[i], alpha, sum);
#pragma unroll
            for (int c = 0; c < NC; ++c) o[i][c].x *= alpha, o[i][c].y *= alpha, o[i][c].z *= alpha, o[i][c].w *= alpha;
        }
        __syncthreads();
        add_rows<RM, NC, LD>(sp, sv, o);
    }
#pragma unroll
    for (int i = 0; i < RM; ++i) {
        const int r = r0 + ty * RM + i;
#pragma unroll
        for (int w = 1; w < 16; w <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], w);
        if (r >= rows) continue;
        const int tok = q.q0 + r / p.G, h = x.h * p.G + r % p.G;
        const bool none = m[i] == -INFINITY && l[i] == 0.f;
        const float inv = none ? 0.f : 1.f / l[i];
        T* out = static_cast<T*>(p.out) + ((long long)tok * p.Hq + h) * p.D;
#pragma unroll
        for (int c = 0; c < NC; ++c)
            if (64 * c + 4 * tx < p.D) store4<T>(out + 64 * c + 4 * tx, o[i][c], inv);
        if (tx == 0 && p.lse) p.lse[(long long)h * p.total_q + tok] = none ? -INFINITY : (m[i] + log2f(l[i])) * kLn2;
    }
}

// P and dS of a tile of BM rows (at r0) and the keys from k0 on, from the four tiles in shared memory, into sp and sd.
template <int RM, int LD>
__device__ __forceinline__ void weights(const PromptParams& p, const Seq& q, int h, int r0, int k0, const float* sq,
                                        const float* sg, const float* sk, const float* sv, float* sp, float* sd) {
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16, rows = q.lq * p.G;
    float s[RM][4], g[RM][4];
    products<RM, LD>(sq, sk, p.D, s);
    products<RM, LD>(sg, sv, p.D, g);
    const float f = p.scale * kToLog2;
#pragma unroll
    for (int i = 0; i < RM; ++i) {
        const int r = r0 + ty * RM + i;
        const long long at = (long long)(h * p.G + r % p.G) * p.total_q + q.q0 + r / p.G;
        const int limit = r < rows ? r / p.G + q.shift : -1;
        const float lse = r < rows ? p.lse[at] * kToLog2 : 0.f, delta = r < rows ? p.delta[at] : 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const bool sees = k0 + tx + 16 * j <= limit;
            const float pr = sees ? exp2f(fmaf(s[i][j], f, -lse)) : 0.f;
            if (sp) sp[(ty * RM + i) * kLP + tx + 16 * j] = pr;
            sd[(ty * RM + i) * kLP + tx + 16 * j] = sees ? pr * (g[i][j] - delta) : 0.f;
        }
    }
}

template <typename T, int NC, int BM>
__global__ void __launch_bounds__(kThreads) prompt_dkv_simt(const PromptParams p, int tiles) {
    constexpr int RM = BM / 16, LD = 64 * NC + 4;
    extern __shared__ float smem[];
    float *sk = smem, *sv = sk + kKeys * LD, *sq = sv + kKeys * LD, *sg = sq + BM * LD, *sp = sg + BM * LD, *sd = sp + BM * kLP;
    const Place x = place(p, tiles, false);
    const Seq q = load_seq(p, x.seq, threadIdx.x == 0 && x.tile == 0 && x.h == 0);
    const int k0 = x.tile * kKeys, rows = q.lq * p.G, ty = threadIdx.x / 16, tx = threadIdx.x % 16;
    if (k0 >= q.lk) return;
    load_tile<T, kKeys, LD>(sk, p.D, [&](int k) { return key_at<T>(p, q, x.h, k0 + k, p.k, p.k_rs); });
    load_tile<T, kKeys, LD>(sv, p.D, [&](int k) { return key_at<T>(p, q, x.h, k0 + k, p.v, p.v_rs); });
    float4 dk[4][NC], dv[4][NC];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int c = 0; c < NC; ++c) dk[i][c] = dv[i][c] = make_float4(0.f, 0.f, 0.f, 0.f);
    // the first row that sees a key of the tile
    const long long first = (long long)max(0, k0 - q.shift) * p.G;
    for (long long r = first / BM * BM; r < rows; r += BM) {
        const int r0 = (int)r;
        __syncthreads();
        load_tile<T, BM, LD>(sq, p.D, [&](int i) { return row_at<T>(p, q, x.h, r0 + i, p.q, p.q_rs); });
        load_tile<T, BM, LD>(sg, p.D, [&](int i) { return row_at<T>(p, q, x.h, r0 + i, p.d_out, (long long)p.Hq * p.D); });
        __syncthreads();
        weights<RM, LD>(p, q, x.h, r0, k0, sq, sg, sk, sv, sp, sd);
        __syncthreads();
        add_cols<BM, NC, LD>(sp, sg, dv);
        add_cols<BM, NC, LD>(sd, sq, dk);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int k = k0 + 4 * ty + i;
        if (k >= q.lk) continue;
        const long long at = ((long long)(q.k0 + k) * p.Hk + x.h) * p.D;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int d = 64 * c + 4 * tx;
            if (d >= p.D) continue;
            store4<T>(static_cast<T*>(p.dk) + at + d, dk[i][c], p.scale);
            store4<T>(static_cast<T*>(p.dv) + at + d, dv[i][c], 1.f);
        }
    }
}

template <typename T, int NC, int BM>
__global__ void __launch_bounds__(kThreads) prompt_dq_simt(const PromptParams p, int tiles) {
    constexpr int RM = BM / 16, LD = 64 * NC + 4;
    extern __shared__ float smem[];
    float *sk = smem, *sv = sk + kKeys * LD, *sq = sv + kKeys * LD, *sg = sq + BM * LD, *sd = sg + BM * LD;
    const Place x = place(p, tiles, true);
    const Seq q = load_seq(p, x.seq, threadIdx.x == 0 && x.tile == 0 && x.h == 0);
    const int rows = q.lq * p.G, r0 = x.tile * BM, ty = threadIdx.x / 16, tx = threadIdx.x % 16;
    if (r0 >= rows) return;
    load_tile<T, BM, LD>(sq, p.D, [&](int i) { return row_at<T>(p, q, x.h, r0 + i, p.q, p.q_rs); });
    load_tile<T, BM, LD>(sg, p.D, [&](int i) { return row_at<T>(p, q, x.h, r0 + i, p.d_out, (long long)p.Hq * p.D); });
    float4 dq[RM][NC];
#pragma unroll
    for (int i = 0; i < RM; ++i)
#pragma unroll
        for (int c = 0; c < NC; ++c) dq[i][c] = make_float4(0.f, 0.f, 0.f, 0.f);
    const int last = min(r0 + BM, rows) - 1, keys = last / p.G + q.shift + 1;
    for (int k0 = 0; k0 < keys; k0 += kKeys) {
        __syncthreads();
        load_tile<T, kKeys, LD>(sk, p.D, [&](int k) { return k0 + k < keys ? key_at<T>(p, q, x.h, k0 + k, p.k, p.k_rs) : nullptr; });
        load_tile<T, kKeys, LD>(sv, p.D, [&](int k) { return k0 + k < keys ? key_at<T>(p, q, x.h, k0 + k, p.v, p.v_rs) : nullptr; });
        __syncthreads();
        weights<RM, LD>(p, q, x.h, r0, k0, sq, sg, sk, sv, nullptr, sd);
        __syncthreads();
        add_rows<RM, NC, LD>(sd, sk, dq);
    }
#pragma unroll
    for (int i = 0; i < RM; ++i) {
        const int r = r0 + ty * RM + i;
        if (r >= rows) continue;
        T* at = static_cast<T*>(p.dq) + ((long long)(q.q0 + r / p.G) * p.Hq + x.h * p.G + r % p.G) * p.D;
#pragma unroll
        for (int c = 0; c < NC; ++c)
            if (64 * c + 4 * tx < p.D) store4<T>(at + 64 * c + 4 * tx, dq[i][c], p.scale);
    }
}

// Sixteen lanes a row of (t, h): delta, and in fp16 on tensor cores |dO|.
template <typename T>
__global__ void __launch_bounds__(kThreads) prompt_delta_kernel(const PromptParams p) {
    constexpr int kV = Vec<T>::n;
    const long long r = ((long long)blockIdx.x * kThreads + threadIdx.x) / 16;
    const int lane = threadIdx.x % 16;
    const bool in = r < (long long)p.total_q * p.Hq;
    float sum = 0.f, square = 0.f;
    for (int d = lane * kV; in && d < p.D; d += 16 * kV) {
        float a[kV], b[kV];
        Vec<T>::load(static_cast<const T*>(p.out) + r * p.D + d, a);
        Vec<T>::load(static_cast<const T*>(p.d_out) + r * p.D + d, b);
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            sum = fmaf(a[i], b[i], sum);
            if constexpr (std::is_same<T, __half>::value) square = fmaf(b[i], b[i], square);
        }
    }
    float* to = p.delta;
    if constexpr (std::is_same<T, __half>::value) {  // (even lanes go on with the sum, odd ones with the square)
        const float other = __shfl_xor_sync(0xffffffffu, lane & 1 ? sum : square, 1);
        sum = (lane & 1 ? square : sum) + other;
        if (lane & 1) to = p.norm;
    } else {
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
    }
#pragma unroll
    for (int o = 2; o < 16; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (in && lane < (std::is_same<T, __half>::value ? 2 : 1) && to) to[(r % p.Hq) * p.total_q + r / p.Hq] = lane ? sqrtf(sum) : sum;
    if constexpr (std::is_same<T, __half>::value) {
        if (!p.norm) return;
        for (long long e = (long long)blockIdx.x * kThreads + threadIdx.x; e < (long long)p.num_seqs * p.Hk * 3; e += (long long)gridDim.x * kThreads)
            p.most[e] = 0.f;  // (for prompt_most_kernel)
    }
}

// p.most (zeroed before) of the block's (sequence, key head): the largest |V| of its keys (D <= 128), |dO| and |delta| of its
// rows; blocks along y share them out.  An infinity or NaN does not count (what is multiplied with one is no number anyway).
__global__ void __launch_bounds__(kThreads) prompt_most_kernel(const PromptParams p) {
    const Seq q = load_seq(p, (int)(blockIdx.x / (unsigned)p.Hk), false);
    const int h = (int)(blockIdx.x % (unsigned)p.Hk), lane = threadIdx.x % 16;
    auto finite = [](float x) { return x <= 3.4e38f ? x : 0.f; };
    float most[3] = {0.f, 0.f, 0.f};
    constexpr int kAhead = 4, kPer = kThreads / 16 * kAhead;  // keys a thread has in flight, keys of a block at a time
    for (int k0 = (int)blockIdx.y * kPer; k0 < q.lk; k0 += (int)gridDim.y * kPer) {
        float square[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int k = k0 + j * (kThreads / 16) + threadIdx.x / 16;
            float a[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            if (k < q.lk && lane * 8 < p.D) Vec<__half>::load(key_at<__half>(p, q, h, k, p.v, p.v_rs) + lane * 8, a);
            square[j] = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) square[j] = fmaf(a[i], a[i], square[j]);
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
#pragma unroll
            for (int o = 1; o < 16; o <<= 1) square[j] += __shfl_xor_sync(0xffffffffu, square[j], o);
            most[0] = fmaxf(most[0], finite(sqrtf(square[j])));
        }
    }
    for (int g = 0; g < p.G; ++g) {
        const long long row = (long long)(h * p.G + g) * p.total_q + q.q0;
#pragma unroll 4
        for (int t = (int)blockIdx.y * kThreads + threadIdx.x; t < q.lq; t += (int)gridDim.y * kThreads) {
            most[1] = fmaxf(most[1], finite(p.norm[row + t]));
            most[2] = fmaxf(most[2], finite(fabsf(p.delta[row + t])));
        }
    }
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        const unsigned m = __reduce_max_sync(0xffffffffu, __float_as_uint(most[i]));  // (not negative: ordered as its bits)
        if (threadIdx.x % 32 == 0 && m) atomicMax(reinterpret_cast<unsigned*>(p.most) + blockIdx.x * 3 + i, m);
    }
}

cudaError_t grid_of(const PromptParams& p, long long tiles, unsigned& grid) {
    const long long n = tiles * p.num_seqs * p.Hk;
    if (n > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    grid = (unsigned)n;
    return cudaSuccess;
}

template <typename K>
cudaError_t start(K kern, const PromptParams& p, long long tiles, size_t floats, cudaStream_t stream) {
    unsigned grid = 0;
    cudaError_t e = grid_of(p, tiles, grid);
    if (e != cudaSuccess || grid == 0) return e;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxDynamicSmem);
    if (e != cudaSuccess) return e;
    kern<<<grid, kThreads, floats * sizeof(float), stream>>>(p, (int)tiles);
    return cudaGetLastError();
}

template <typename T, int NC>
cudaError_t forward(const PromptParams& p, cudaStream_t stream) {
    const long long tiles = ((long long)p.max_q * p.G + 63) / 64;
    return start(prompt_fwd_simt<T, NC>, p, tiles, (size_t)3 * 64 * (64 * NC + 4), stream);
}

}  // namespace

cudaError_t launch_delta(const PromptParams& p, cudaStream_t stream) {
    const long long n = ((long long)p.total_q * p.Hq + 15) / 16;
    if (n > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    switch (p.dtype) {
    case TA_F32: prompt_delta_kernel<float><<<(unsigned)n, kThreads, 0, stream>>>(p); break;
    case TA_F16: prompt_delta_kernel<__half><<<(unsigned)n, kThreads, 0, stream>>>(p); break;
    default: prompt_delta_kernel<__nv_bfloat16><<<(unsigned)n, kThreads, 0, stream>>>(p); break;
    }
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !p.norm) return e;
    const long long pairs = (long long)p.num_seqs * p.Hk;
    if (pairs > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    // Blocks of a pair: one for 64 keys or rows of the longest, up to 64, but not many more in all than the GPU has places.
    const long long longest = p.max_q > p.max_k ? p.max_q : p.max_k, room = 16384 / pairs;
    long long shares = (longest + 63) / 64 < 64 ? (longest + 63) / 64 : 64;
    if (shares > room) shares = room;
    prompt_most_kernel<<<dim3((unsigned)pairs, (unsigned)(shares > 1 ? shares : 1)), kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

namespace {

template <typename T, int NC>
cudaError_t backward(const PromptParams& p, cudaStream_t stream) {
    constexpr int BM = NC == 4 ? 32 : 64, LD = 64 * NC + 4;
    cudaError_t e = p.total_q > 0 ? launch_delta(p, stream) : cudaSuccess;
    if (e != cudaSuccess) return e;
    const size_t tile = (size_t)2 * (kKeys + BM) * LD;
    e = start(prompt_dkv_simt<T, NC, BM>, p, (p.max_k + kKeys - 1) / kKeys, tile + 2 * BM * kLP, stream);
    if (e != cudaSuccess) return e;
    return start(prompt_dq_simt<T, NC, BM>, p, ((long long)p.max_q * p.G + BM - 1) / BM, tile + BM * kLP, stream);
}

template <typename T>
cudaError_t launch(const PromptParams& p, bool back, cudaStream_t stream) {
    if constexpr (sizeof(T) == 4) {  // (16-bit rows of these widths run on tensor cores)
        if (p.D <= 64) return back ? backward<T, 1>(p, stream) : forward<T, 1>(p, stream);
        if (p.D <= 128) return back ? backward<T, 2>(p, stream) : forward<T, 2>(p, stream);
    }
    return back ? backward<T, 4>(p, stream) : forward<T, 4>(p, stream);
}

cudaError_t launch_any(const PromptParams& p, bool back, cudaStream_t stream) {
    switch (p.dtype) {
    case TA_F32: return launch<float>(p, back, stream);
    case TA_F16: return launch<__half>(p, back, stream);
    default: return launch<__nv_bfloat16>(p, back, stream);
    }
}

}  // namespace
}  // namespace prompt

cudaError_t launch_prompt_simt_fwd(const PromptParams& p, cudaStream_t stream) { return prompt::launch_any(p, false, stream); }
cudaError_t launch_prompt_simt_bwd(const PromptParams& p, cudaStream_t stream) { return prompt::launch_any(p, true, stream); }

}  // namespace triattn
