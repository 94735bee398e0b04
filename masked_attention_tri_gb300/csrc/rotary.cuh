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
// as exact as position 1, where p * theta_i in fp32 is off by a radian at p = 2^24.  Several axes change only which
// position a pair is multiplied with.
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

// The position by which pair i of row `row` turns: with several axes (time, height, width: positions (num_axes, total))
// each pair has an axis of its own.  (A number that names no axis is read as axis 0.)
__device__ __forceinline__ int rotary_position(const int32_t* positions, const int32_t* axes, int num_axes, int i,
                                               int total, long long row) {
    if (!axes) return positions[row];
    const uint32_t a = (uint32_t)axes[i];
    return positions[(a < (uint32_t)num_axes ? (long long)a * total : 0LL) + row];
}

// One value of T to and from fp32.
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

// The work of one head is cut into units of two vectors of V elements (16 bytes; V = 1 where
// rotary_dim is no multiple of 2 V): first the rotated pairs (V pairs a unit), then the elements
// past rotary_dim.
//   half layout   elements [uV, uV + V) and rotary_dim / 2 further on
//   interleaved   elements [2uV, 2uV + 2V)
//   past          elements [rotary_dim + 2uV, ...): the second vector may be missing
struct RotUnit {
    int o0, o1;   // element offset of the first vector, and of the second from it; o1 < 0: none
    bool turned;
};
template <int V>
__host__ __device__ __forceinline__ int rot_units(int D, int dim) {
    return dim / (2 * V) + (D - dim + 2 * V - 1) / (2 * V);
}
template <int V>
__device__ __forceinline__ RotUnit rot_unit(int u, int D, int dim, bool interleaved) {
    RotUnit r;
    const int nr = dim / (2 * V);
    r.turned = u < nr;
    if (r.turned) {
        r.o0 = interleaved ? 2 * u * V : u * V;
        r.o1 = interleaved ? V : dim / 2;
    } else {
        r.o0 = dim + 2 * (u - nr) * V;
        r.o1 = r.o0 + V < D ? V : -1;
    }
    return r;
}

// Tables of cos and sin in shared memory: for the rotated unit u (of nr) of row r and the pairs 2j, 2j + 1
// of its V, (cos, cos, sin, sin) at [r][j][u], so that the lanes of a warp, which hold neighbouring
// units, read neighbouring 16 bytes.  One pair a unit (V = 1): (cos, sin) at [r][u].
template <int V>
__device__ __forceinline__ void rot_table_put(float* table, int row, int pair, int nr, float c, float s) {
    if (V == 1) {
        table[(row * nr + pair) * 2] = c;
        table[(row * nr + pair) * 2 + 1] = s;
    } else {
        const int u = pair / V, w = pair % V;
        float* at = table + ((row * (V / 2) + w / 2) * nr + u) * 4 + (w & 1);
        at[0] = c;
        at[2] = s;
    }
}
template <int V>
__device__ __forceinline__ const float* rot_table_at(const float* table, int row, int u, int nr) {
    return V == 1 ? table + (row * nr + u) * 2 : table + ((row * (V / 2)) * nr + u) * 4;
}

// A unit in registers as it is in memory.
template <typename T, int V>
struct RotRaw {
    uint4 v0, v1;  // 16 bytes each: V = 8 of 16 bits, 4 of fp32
    __device__ __forceinline__ void load(const T* p, int o1) {
        v0 = *reinterpret_cast<const uint4*>(p);
        v1 = o1 >= 0 ? *reinterpret_cast<const uint4*>(p + o1) : make_uint4(0u, 0u, 0u, 0u);
    }
    __device__ __forceinline__ void store(T* p, int o1) const {
        *reinterpret_cast<uint4*>(p) = v0;
        if (o1 >= 0) *reinterpret_cast<uint4*>(p + o1) = v1;
    }
};
template <typename T>
struct RotRaw<T, 1> {
    T v0, v1;
    __device__ __forceinline__ void load(const T* p, int o1) {
        v0 = p[0];
        v1 = o1 >= 0 ? p[o1] : rot_from_f<T>(0.f);
    }
    __device__ __forceinline__ void store(T* p, int o1) const {
        p[0] = v0;
        if (o1 >= 0) p[o1] = v1;
    }
};
__device__ __forceinline__ float2 rot_unpack(__nv_bfloat16, uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ float2 rot_unpack(__half, uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
__device__ __forceinline__ uint32_t rot_pack(__nv_bfloat16, float2 x) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(x.x, x.y);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t rot_pack(__half, float2 x) {
    const __half2 v = __floats2half2_rn(x.x, x.y);
    return *reinterpret_cast<const uint32_t*>(&v);
}
// ... and as fp32: f[0, V / 2) the first vector, f[V / 2, V) the second (V = 1: both in f[0]).
template <typename T, int V>
__device__ __forceinline__ void rot_floats(const RotRaw<T, V>& r, float2 (&f)[V]) {
    if constexpr (V == 1) {
        f[0] = make_float2(rot_to_f(r.v0), rot_to_f(r.v1));
    } else {
        const uint32_t a[8] = {r.v0.x, r.v0.y, r.v0.z, r.v0.w, r.v1.x, r.v1.y, r.v1.z, r.v1.w};
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if constexpr (sizeof(T) == 2) f[i] = rot_unpack(T(), a[i]);
            else f[i] = make_float2(__uint_as_float(a[2 * i]), __uint_as_float(a[2 * i + 1]));
        }
    }
}
template <typename T, int V>
__device__ __forceinline__ RotRaw<T, V> rot_raw(const float2 (&f)[V]) {
    RotRaw<T, V> r;
    if constexpr (V == 1) {
        r.v0 = rot_from_f<T>(f[0].x);
        r.v1 = rot_from_f<T>(f[0].y);
    } else {
        uint32_t a[8];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if constexpr (sizeof(T) == 2) a[i] = rot_pack(T(), f[i]);
            else a[2 * i] = __float_as_uint(f[i].x), a[2 * i + 1] = __float_as_uint(f[i].y);
        }
        r.v0 = make_uint4(a[0], a[1], a[2], a[3]);
        r.v1 = make_uint4(a[4], a[5], a[6], a[7]);
    }
    return r;
}

// Two neighbouring pairs turned by (cos, cos, sin, sin): of the half layout (a.x, b.x) and (a.y, b.y), of the
// interleaved one (a.x, a.y) and (b.x, b.y).
__device__ __forceinline__ void rot_turn2(float2& a, float2& b, float4 cs, bool interleaved) {
    const float2 c = make_float2(cs.x, cs.y), s = make_float2(cs.z, cs.w), x = a, y = b;
    if (interleaved) {
        a = make_float2(x.x * c.x - x.y * s.x, x.x * s.x + x.y * c.x);
        b = make_float2(y.x * c.y - y.y * s.y, y.x * s.y + y.y * c.y);
    } else {
        a = __ffma2_rn(x, c, __fmul2_rn(y, make_float2(-s.x, -s.y)));
        b = __ffma2_rn(x, s, __fmul2_rn(y, c));
    }
}
template <int V>
__device__ __forceinline__ void rot_turn(float2 (&f)[V], const float* table, int nr, bool interleaved) {
    if constexpr (V == 1) {
        const float c = table[0], s = table[1];
        f[0] = make_float2(f[0].x * c - f[0].y * s, f[0].x * s + f[0].y * c);
    } else {
        const float4* t4 = reinterpret_cast<const float4*>(table);
#pragma unroll
        for (int j = 0; j < V / 2; ++j) {
            if (interleaved) rot_turn2(f[2 * j], f[2 * j + 1], t4[j * nr], true);
            else rot_turn2(f[j], f[V / 2 + j], t4[j * nr], false);
        }
    }
}

}  // namespace triattn
