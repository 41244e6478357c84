// kv4.cuh -- the 4-bit cache row: layout, block scale, codes and values.
//
// One cache row (one slot, all KV heads) holds
//     Hkv * dh / 2   bytes of codes, head after head: two e2m1 codes a byte,
//                    the lower element in the lower half
//     Hkv * dh / 16  bytes of scales: one e4m3 for 16 consecutive elements
//     padding up to a multiple of 16 bytes
// A block of 16 elements x is stored as s = e4m3 nearest to max|x| / 6 (ties
// to the even mantissa, at most 448) and c = e2m1 nearest to x / s (ties to
// the even mantissa, at most 6); it stands for c * s.  s has at most four
// significant bits and c two, so c * s has at most six and lies in
// [2^-10, 2688] or is 0: exact in bf16, in fp16 and in fp32.  A block that
// holds an infinity or a NaN gets the NaN scale and stands for 16 NaNs.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include "common.cuh"

namespace medusa {

__host__ __device__ constexpr int kv4_code_bytes(int Hkv, int dh) { return Hkv * dh / 2; }
__host__ __device__ constexpr int kv4_row_bytes(int Hkv, int dh) {
    return (Hkv * dh / 2 + Hkv * dh / 16 + 15) / 16 * 16;
}

constexpr uint32_t kE4m3Nan = 0x7f;

// value of a non-negative finite e4m3 byte (exact)
__device__ __forceinline__ float e4m3_value(uint32_t byte) {
    const __half_raw h = __nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)byte, __NV_E4M3);
    return __half2float(__half(h));
}

// two e2m1 codes (one byte) -> two halves (exact)
__device__ __forceinline__ __half2 e2m1x2_half2(uint32_t byte) {
    const __half2_raw h =
        __nv_cvt_fp4x2_to_halfraw2((__nv_fp4x2_storage_t)(byte & 0xffu), __NV_E2M1);
    return __half2(h);
}

// Scale byte of a block whose largest magnitude is `amax` (finite): the e4m3
// nearest to amax / 6.  The conversion of the rounded quotient can be off by
// one step next to a midpoint m; comparing amax with 6 m, which is exact
// (m has five significant bits), puts it right.
__device__ __forceinline__ uint32_t kv4_scale_byte(float amax) {
    uint32_t c = __nv_cvt_float_to_fp8(amax / 6.f, __NV_SATFINITE, __NV_E4M3);
    const float v = e4m3_value(c);
    if (c > 0) {
        const float lo6 = 3.f * (e4m3_value(c - 1) + v);  // six times the midpoint below
        if (amax < lo6 || (amax == lo6 && (c & 1))) return c - 1;
    }
    if (c < 0x7e) {
        const float hi6 = 3.f * (v + e4m3_value(c + 1));
        if (amax > hi6 || (amax == hi6 && (c & 1))) return c + 1;
    }
    return c;
}

// Code (0..15) of x in a block of scale s > 0.  The midpoints between the
// e2m1 magnitudes have at most three significant bits, so their products
// with s are exact and so are the comparisons; a tie goes to the even code.
__device__ __forceinline__ uint32_t kv4_code(float x, float s) {
    const float a = fabsf(x);
    uint32_t c = (a > 0.25f * s) + (a >= 0.75f * s) + (a > 1.25f * s) + (a >= 1.75f * s) +
                 (a > 2.5f * s) + (a >= 3.5f * s) + (a > 5.f * s);
    return c | (x < 0.f ? 8u : 0u);
}

}  // namespace medusa
