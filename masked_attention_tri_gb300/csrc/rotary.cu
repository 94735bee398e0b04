// rotary.cu -- rotary positions of packed queries and keys, forward and inverse
// (the inverse is the backward: the turn is orthogonal up to mscale).  The
// mathematics stands in rotary.cuh.
//
// Bound: memory, 2 bytes moved per byte of q and k.  One thread takes one unit
// (V pairs) of one token and walks the token's heads with that unit's cos and sin
// in registers, so their 40-odd instructions a pair are paid once for all heads; four
// heads are loaded before the first is stored, which keeps 128 bytes a thread
// in flight.  With few tokens the heads are dealt over more threads instead
// (each computing cos and sin again) until the grid fills the GPU: there latency
// counts and not instructions.

#include "internal.h"
#include "rotary.cuh"

namespace triattn {
namespace {

constexpr int kThreads = 256;
constexpr int kAhead = 4;  // heads in flight a thread

struct RotaryArgs {
    RotaryParams p;
    int units;        // units per head
    int splits;       // threads that share one (token, unit)'s heads
    long long threads;
};

template <typename T, int V>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const RotaryArgs a) {
    const RotaryParams& p = a.p;
    const long long id = (long long)blockIdx.x * kThreads + threadIdx.x;
    if (id >= a.threads) return;
    const int u = (int)(id % a.units);
    const long long rest = id / a.units;
    const long long tok = rest / a.splits;
    const int split = (int)(rest - tok * a.splits);
    const RotUnit r = rot_unit<V>(u, p.D, p.dim, p.interleaved);
    float cs[V], sn[V];
    if (r.pair0 >= 0) {
        const int pos = p.positions[tok];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float2 t = rotary_cos_sin(pos, p.turns[r.pair0 + i]);
            cs[i] = t.x * p.mscale;
            sn[i] = (p.inverse ? -t.y : t.y) * p.mscale;
        }
    }
    const int H = p.Hq + p.Hk;
    const T* q = static_cast<const T*>(p.q) + tok * p.q_rs;
    const T* k = static_cast<const T*>(p.k) + tok * p.k_rs;
    T* qo = static_cast<T*>(p.q_out) + tok * p.qo_rs;
    T* ko = static_cast<T*>(p.k_out) + tok * p.ko_rs;
    for (int h0 = split; h0 < H; h0 += kAhead * a.splits) {
        float x0[kAhead][V], x1[kAhead][V];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int h = h0 + j * a.splits;
            if (h >= H) break;
            const T* src = h < p.Hq ? q + (long long)h * p.D : k + (long long)(h - p.Hq) * p.D;
            rot_load<T, V>(src + r.o0, x0[j]);
            if (r.o1 >= 0) rot_load<T, V>(src + r.o1, x1[j]);
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int h = h0 + j * a.splits;
            if (h >= H) break;
            T* dst = h < p.Hq ? qo + (long long)h * p.D : ko + (long long)(h - p.Hq) * p.D;
            if (r.pair0 >= 0) rot_turn<V>(x0[j], x1[j], cs, sn, p.interleaved);
            rot_store<T, V>(dst + r.o0, x0[j]);
            if (r.o1 >= 0) rot_store<T, V>(dst + r.o1, x1[j]);
        }
    }
}

template <typename T, int V>
cudaError_t launch(const RotaryParams& p, cudaStream_t stream) {
    RotaryArgs a;
    a.p = p;
    a.units = rot_units<V>(p.D, p.dim);
    const int H = p.Hq + p.Hk;
    // Threads that fill the GPU once (152 SMs of 2048): below that the heads are dealt over
    // more threads.
    const long long fill = 152LL * 2048, base = (long long)p.total * a.units;
    long long s = (fill + base - 1) / base;
    a.splits = (int)(s < 1 ? 1 : (s > H ? H : s));
    a.threads = base * a.splits;
    const long long grid = (a.threads + kThreads - 1) / kThreads;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    rotary_kernel<T, V><<<(unsigned)grid, kThreads, 0, stream>>>(a);
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
