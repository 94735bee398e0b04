// rotary.cuh -- rotary positions on pairs of a head's leading elements, shared by
// the rotary kernel (rotary.cu) and the cache append (kv_append.cu).
//
// Pair i of a head at position p turns by the angle 2 pi p f_i (f_i in turns per
// position, f_i = theta_i / 2 pi):
//     (a, b) -> mscale * (a cos - b sin, a sin + b cos),
// the inverse (which is the transpose up to mscale, so the gradient) by the
// opposite angle.  Only the angle's part of a whole turn matters, so f_i is held
// as a 64-bit fixed-point fraction of a turn and the product p * f_i wraps to it
// exactly (two's complement: negative positions too).  A position of 2^31 is thus
// as exact as position 1, where p * theta_i in fp32 is off by a radian at p = 2^24.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

namespace triattn {

// cos and sin of `pos` positions at `turns` (2^-64 turns per position).  The top 32 bits of
// the phase are reduced to an eighth of a turn either side of a quadrant in integers, so the
// fp32 argument is off by at most 2^-27 half-turns.
__device__ __forceinline__ float2 rotary_cos_sin(int pos, unsigned long long turns) {
    const unsigned long long ph = (unsigned long long)(long long)pos * turns;
    const uint32_t p = (uint32_t)((ph + (1ull << 31)) >> 32);  // 2^-32 turns, to nearest
    const uint32_t quad = (p + (1u << 29)) >> 30;              // nearest quarter turn
    const int r = (int)(p - (quad << 30));                     // [-2^29, 2^29): within an eighth of a turn
    float s, c;
    sincospif((float)r * 4.656612873077393e-10f /* 2^-31: half-turns */, &s, &c);
    const float cq = (quad & 1u) ? s : c, sq = (quad & 1u) ? c : s;
    return make_float2((quad + 1u) & 2u ? -cq : cq, quad & 2u ? -sq : sq);
}

// V elements of T as fp32, moved as one access (16 bytes for fp32 V = 4 and 16-bit V = 8).
template <typename T>
__device__ __forceinline__ float rot_to_f(T x) {
    return (float)x;
}
template <typename T>
__device__ __forceinline__ T rot_from_f(float x);
template <>
__device__ __forceinline__ float rot_from_f<float>(float x) {
    return x;
}
template <>
__device__ __forceinline__ __half rot_from_f<__half>(float x) {
    return __float2half_rn(x);
}
template <>
__device__ __forceinline__ __nv_bfloat16 rot_from_f<__nv_bfloat16>(float x) {
    return __float2bfloat16_rn(x);
}

template <typename T, int V>
struct alignas(sizeof(T) * V) RotVec {
    T e[V];
};

template <typename T, int V>
__device__ __forceinline__ void rot_load(const T* p, float (&x)[V]) {
    const RotVec<T, V> v = *reinterpret_cast<const RotVec<T, V>*>(p);
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = rot_to_f(v.e[i]);
}
template <typename T, int V>
__device__ __forceinline__ void rot_store(T* p, const float (&x)[V]) {
    RotVec<T, V> v;
#pragma unroll
    for (int i = 0; i < V; ++i) v.e[i] = rot_from_f<T>(x[i]);
    *reinterpret_cast<RotVec<T, V>*>(p) = v;
}

// The work of one head is cut into units of two vectors of V elements: first the
// rotated pairs (V pairs a unit), then the elements past rotary_dim.
//   half layout   elements [uV, uV + V) and rotary_dim / 2 further on
//   interleaved   elements [2uV, 2uV + 2V)
//   past          elements [rotary_dim + 2uV, ...): the second vector may be missing
struct RotUnit {
    int o0, o1;   // element offsets of the two vectors; o1 < 0: none
    int pair0;    // first rotated pair, or -1 past rotary_dim
};
template <int V>
__host__ __device__ __forceinline__ int rot_units(int D, int dim) {
    return dim / (2 * V) + (D - dim + 2 * V - 1) / (2 * V);
}
template <int V>
__device__ __forceinline__ RotUnit rot_unit(int u, int D, int dim, int interleaved) {
    RotUnit r;
    const int nr = dim / (2 * V);
    if (u < nr) {
        r.pair0 = u * V;
        r.o0 = interleaved ? 2 * u * V : u * V;
        r.o1 = interleaved ? r.o0 + V : r.o0 + dim / 2;
    } else {
        r.pair0 = -1;
        r.o0 = dim + 2 * (u - nr) * V;
        r.o1 = r.o0 + V < D ? r.o0 + V : -1;
    }
    return r;
}

// Turns the unit's V pairs in place: cs holds cos, sn sin (sign and mscale applied).
template <int V>
__device__ __forceinline__ void rot_turn(float (&x0)[V], float (&x1)[V], const float (&cs)[V], const float (&sn)[V],
                                         int interleaved) {
    if (V > 1 && interleaved) {
        // pairs (0, 1), (2, 3), ...: the first half of them in x0, the rest in x1
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            const float a = x0[2 * i], b = x0[2 * i + 1], c = x1[2 * i], d = x1[2 * i + 1];
            x0[2 * i] = a * cs[i] - b * sn[i];
            x0[2 * i + 1] = a * sn[i] + b * cs[i];
            x1[2 * i] = c * cs[i + V / 2] - d * sn[i + V / 2];
            x1[2 * i + 1] = c * sn[i + V / 2] + d * cs[i + V / 2];
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float a = x0[i], b = x1[i];
            x0[i] = a * cs[i] - b * sn[i];
            x1[i] = a * sn[i] + b * cs[i];
        }
    }
}

}  // namespace triattn
