// rotary.cu -- rotary positions of packed queries and keys, forward and inverse
// (the inverse is the backward: the turn is orthogonal up to mscale).  The
// mathematics stands in rotary.cuh.
//
// Bound: memory, 2 bytes moved per byte of q and k.  A CTA takes a few tokens: first it
// fills a table of their cos and sin in shared memory, each pair once for all heads, then its
// threads walk the tokens' units (V pairs, two vectors of 16 bytes each) in the order of memory,
// so that a warp's loads cover whole kilobytes of one token's row.  The 16-bit values stay packed
// until they are turned, two at a time: at 48 registers a thread five CTAs share an SM, which
// does more for the loads in flight than longer queues of a thread (at 120 registers: 187 us).
// 16384 tokens x 40 heads of 128 in bf16, both ways: 110 us, 6.1 TB/s.

#include "internal.h"
#include "rotary.cuh"
#include "tc_kernel.cuh"

namespace triattn {
namespace {

constexpr int kThreads = 256;
constexpr int kAhead = 2;        // units in flight a thread
constexpr int kMaxTokens = 4;    // tokens of a CTA (16: 116 us, 8: 112, 4: 110 in the case above)

struct RotaryArgs {
    RotaryParams p;
    int tokens;                  // of a CTA
    int units;                   // units per head
    int lanes;                   // heads that the CTA's threads take at once (each thread keeps its unit)
    tc::FastDiv fd_heads;        // Hq + Hk
};

template <typename T, int V, bool INTER>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const RotaryArgs a) {
    extern __shared__ float4 table4[];
    float* table = reinterpret_cast<float*>(table4);
    const RotaryParams& p = a.p;
    const int tok0 = blockIdx.x * a.tokens, nt = min(a.tokens, p.total - tok0);
    const int np = p.dim / 2, nr = np / V, H = p.Hq + p.Hk;
    for (int e = threadIdx.x; e < nt * np; e += kThreads) {
        const int t = e / np, i = e - t * np;
        const float2 cs = rotary_cos_sin(p.positions[tok0 + t], p.turns[i]);
        rot_table_put<V>(table, t, i, nr, cs.x * p.mscale, (p.inverse ? -cs.y : cs.y) * p.mscale);
    }
    __syncthreads();

    // This thread's unit; its heads are hl, hl + lanes, ... of the CTA's tokens' in a row.
    const int hl = threadIdx.x / a.units, u = threadIdx.x - hl * a.units;
    if (hl >= a.lanes) return;
    const RotUnit r = rot_unit<V>(u, p.D, p.dim, INTER);
    auto place = [&](int n, const T*& src, T*& dst) -> int {
        const int t = (int)a.fd_heads.div((uint32_t)n), h = n - t * H;
        const long long tok = tok0 + t;
        if (h < p.Hq) {
            src = static_cast<const T*>(p.q) + tok * p.q_rs + h * p.D + r.o0;
            dst = static_cast<T*>(p.q_out) + tok * p.qo_rs + h * p.D + r.o0;
        } else {
            src = static_cast<const T*>(p.k) + tok * p.k_rs + (h - p.Hq) * p.D + r.o0;
            dst = static_cast<T*>(p.k_out) + tok * p.ko_rs + (h - p.Hq) * p.D + r.o0;
        }
        return t;
    };
    for (int n0 = hl; n0 < nt * H; n0 += kAhead * a.lanes) {
        RotRaw<T, V> w[kAhead];
        T* dst[kAhead];
        int tok[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int n = n0 + j * a.lanes;
            if (n >= nt * H) break;
            const T* src;
            tok[j] = place(n, src, dst[j]);
            w[j].load(src, r.o1);
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            if (n0 + j * a.lanes >= nt * H) break;
            if (r.turned) {
                float2 f[V];
                rot_floats<T, V>(w[j], f);
                rot_turn<V>(f, rot_table_at<V>(table, tok[j], u, nr), nr, INTER);
                w[j] = rot_raw<T, V>(f);
            }
            w[j].store(dst[j], r.o1);
        }
    }
}

template <typename T, int V>
cudaError_t launch(const RotaryParams& p, cudaStream_t stream) {
    RotaryArgs a;
    a.p = p;
    a.units = rot_units<V>(p.D, p.dim);
    const long long H = (long long)p.Hq + p.Hk;
    if (H * kMaxTokens > 0x3fffffffLL || H * p.D > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    // As many tokens a CTA as leave eight CTAs for each of 152 SMs: few, and latency is what counts; many, and
    // a table serves longer.
    const int t = p.total / (152 * 8);
    a.tokens = t < 1 ? 1 : (t > kMaxTokens ? kMaxTokens : t);
    a.lanes = kThreads / a.units;  // (a head has at most 128 units)
    a.fd_heads = tc::make_fastdiv((uint32_t)H);
    const unsigned grid = (unsigned)(((long long)p.total + a.tokens - 1) / a.tokens);
    const size_t smem = (size_t)a.tokens * (p.dim / 2) * sizeof(float2);  // at most 4 KB
    if (p.interleaved) rotary_kernel<T, V, true><<<grid, kThreads, smem, stream>>>(a);
    else rotary_kernel<T, V, false><<<grid, kThreads, smem, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rotary(const RotaryParams& p, cudaStream_t stream) {
    // 16-byte vectors where they cover whole groups of pairs, else one pair at a time.
    const int V = p.dtype == TA_F32 ? 4 : 8;
    const bool vec = p.dim % (2 * V) == 0;
    switch (p.dtype) {
    case TA_F32: return vec ? launch<float, 4>(p, stream) : launch<float, 1>(p, stream);
    case TA_F16: return vec ? launch<__half, 8>(p, stream) : launch<__half, 1>(p, stream);
    default: return vec ? launch<__nv_bfloat16, 8>(p, stream) : launch<__nv_bfloat16, 1>(p, stream);
    }
}

}  // namespace triattn
