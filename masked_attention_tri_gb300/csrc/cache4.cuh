// cache4.cuh -- the 4-bit codes of a paged cache, shared by the kernels that write them (kv_append4.cu), read them back
// (kv_read.cu) and attend to them (paged_simt.cu, paged_mma.cuh).
//
// 16 neighbouring elements of a row share a scale.  An element of head h stands for n * s * f_h: n a whole number from
// -7 to 7, s an e4m3 number, f_h the head's factor (fixed by the caller; 1 without).  With a = max |x| / f_h of the 16,
//     s = e4m3(a / 7), from 2^-9 to 448,    n = x / (f_h s) rounded to the nearest whole number, ties to even.
// A row keeps its codes for good: nothing that is appended later re-codes it, as a scale belongs to 16 elements of one
// row and not to a page.  (Whole numbers and not the 4-bit floating type: n and s multiply exactly in 16-bit floating
// point, and a code becomes a number by one logical operation and one fused multiplication, where e2m1's sign and
// exponent need three or four on the half-rate pipe; with 16 to a scale both are off by about as much.)
// An infinity or NaN makes its 16 elements NaN: s is e4m3's NaN.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <stdint.h>

namespace triattn {
namespace cache4 {

// Factors: within these 1 / f, and times 1 / s, are fp32 numbers of full precision.
constexpr float kLeastFactor = 0x1p-100f, kMostFactor = 0x1p100f;

// Tag of a 4-bit cache's elements.
struct Code {
    uint8_t two;
};

// The scale's code from the bits of the group's largest |x|.
__device__ __forceinline__ uint32_t scale_code(uint32_t most, float inv_factor) {
    if (most >= 0x7f800000u) return 0x7fu;
    const float a = __fdiv_rn(__uint_as_float(most) * inv_factor, 7.f);
    return __nv_cvt_float_to_fp8(fminf(fmaxf(a, 0x1p-9f), 448.f), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ float scale_value(uint32_t code) {
    return __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)code, __NV_E4M3)));
}
// 1 / x to within 2^-23 of it.
__device__ __forceinline__ float about_inverse(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// A scale s with what the codes of its elements take.
struct Scale {
    float s, inv, half, most;
    __device__ __forceinline__ explicit Scale(float v) : s(v), inv(about_inverse(v)), half(0.5f * v), most(7.f * v) {}
};
// n + 8 in the low four bits (the others are not zero) of y = x / f_h: y / s to the nearest whole number, ties to even, 7 at
// most. y times 1 / s may fall on the wrong side of a border, so the remainder y - n s decides (fp32 holds it exactly: n s has
// eight significant bits, and y is at most 7 s and n s not far from it).  (A NaN's scale says what it is.)
__device__ __forceinline__ uint32_t code(float y, const Scale& c) {
    y = fminf(fmaxf(y, -c.most), c.most);
    const float t = fmaf(y, c.inv, 12582920.f);  // 1.5 * 2^23 + 8: whole numbers, n + 8 in the low bits
    const float d = fmaf(12582920.f - t, c.s, y), a = fabsf(d);
    const uint32_t n = __float_as_uint(t);
    const bool off = a > c.half || (a == c.half && (n & 1u));
    return off ? (d > 0.f ? n + 1u : n - 1u) : n;
}

// Eight codes (n + 8 from 0 to 15, whole bytes zero above) of the low bytes of u as a word.
__device__ __forceinline__ uint32_t pack8(const uint32_t (&u)[8]) {
    uint32_t x[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t y = __byte_perm(__byte_perm(u[4 * i], u[4 * i + 1], 0x0040), __byte_perm(u[4 * i + 2], u[4 * i + 3], 0x0040), 0x5410);
        x[i] = y | (y >> 4);
    }
    return __byte_perm(x[0], x[1], 0x6420);
}
// Sixteen elements x of 16 bits as codes, two words.  x / (f_h s) is rounded to 2^-16 first, which takes the product's error
// off a border, and then to whole numbers.  This is the nearest for elements of at most eleven significant bits and a factor
// that is a power of two: with m of s = m 2^k from 8 to 15, x / (f_h s) is a / (m 2^j), a < 2^11 and 2^j < 2^12; if it is no
// border, it is at least 2^-13 from one.  (Turned elements and other factors: within 2^-16 of a border a code may fall on
// either side.)
__device__ __forceinline__ uint2 codes16(const float (&x)[16], float inv, const Scale& c, bool clamp) {
    const float r = c.inv * inv;
    uint32_t u[2][8];
#pragma unroll
    for (int i = 0; i < 16; ++i) u[i / 8][i % 8] = __float_as_uint(fmaf(x[i], r, 192.f) + 12582728.f);  // 1.5 * 2^7; 1.5 * 2^23 + 8 - 192
    if (clamp) {  // a scale at an end of e4m3's range: some element is more than 7 of it
#pragma unroll
        for (int i = 0; i < 16; ++i)
            u[i / 8][i % 8] = __float_as_uint(fmaf(fminf(fmaxf(x[i] * inv, -c.most), c.most), c.inv, 192.f) + 12582728.f);
    }
    return make_uint2(pack8(u[0]), pack8(u[1]));
}

// Eight codes of a word as eight numbers times s.
__device__ __forceinline__ void values8(uint32_t w, float s, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (float)((int)((w >> (4 * i)) & 15u) - 8) * s;
}

}  // namespace cache4
}  // namespace triattn
