// cache4.cuh -- the 4-bit codes of a paged cache, shared by the kernels that write them (kv_append.cu), read them back
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
// n + 8 of y = x / f_h.  (A NaN gives 8: its scale says what it is.)
__device__ __forceinline__ uint32_t nibble(float y, float s) {
    const int n = __float2int_rn(__fdiv_rn(y, s));
    return (uint32_t)(min(7, max(-7, n)) + 8);
}

// Eight codes of a word as eight numbers times s.
__device__ __forceinline__ void values8(uint32_t w, float s, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (float)((int)((w >> (4 * i)) & 15u) - 8) * s;
}

}  // namespace cache4
}  // namespace triattn
