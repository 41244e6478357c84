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

// the eight codes of a word as four fp16 pairs, times s (exact)
__device__ __forceinline__ uint4 kv4_widen(uint32_t w, __half2 s) {
    uint32_t h[4];
    asm("{\n.reg .b8 b0, b1, b2, b3;\n"
        "mov.b32 {b0, b1, b2, b3}, %4;\n"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n}\n"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 v = __hmul2(*reinterpret_cast<const __half2 *>(&h[i]), s);
        h[i] = *reinterpret_cast<const uint32_t *>(&v);
    }
    return make_uint4(h[0], h[1], h[2], h[3]);
}

// the eight values of a word in fp32
__device__ __forceinline__ void kv4_widen(uint32_t w, __half s, float (&x)[8]) {
    const uint4 v = kv4_widen(w, __half2half2(s));
    const uint32_t h[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h[i]));
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}

__device__ __forceinline__ __half e4m3_half(uint32_t byte) {
    return __half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)byte, __NV_E4M3));
}

// Scale byte of a block whose largest magnitude is `amax` (finite): the e4m3
// nearest to amax / 6.  The conversion of the rounded product can be off by
// one step next to a midpoint m; comparing amax with 6 m, which is exact
// (m has five significant bits), puts it right.
__device__ __forceinline__ uint32_t kv4_scale_byte(float amax) {
    uint32_t c = __nv_cvt_float_to_fp8(amax * (1.f / 6.f), __NV_SATFINITE, __NV_E4M3);
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

// The codes of eight elements.  For bf16 elements the hardware's conversion of
// y = x * (1/s) serves: a bf16 x (eight bits) is either exactly a midpoint
// times s (seven bits at most) or off it by a relative 2^-8, at least 2^-10 of y
// as the midpoints begin at 1/4; y, off by a relative 2^-22, is rounded to a
// multiple of 2^-13 first (by adding and taking away 3 * 2^9), which puts the exact
// ties back on the midpoints and moves nothing across one.  The sign is kept, so
// that a negative x near 0 gives -0; a -0 itself became +0 in the first product.
// fp32 elements can lie closer to a midpoint, so they are compared (14
// instructions each against 3).
__device__ __forceinline__ uint32_t kv4_codes(const float *x, float s, float) {
    uint32_t w = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) w |= kv4_code(x[j], s) << (4 * j);
    return w;
}
__device__ __forceinline__ uint32_t kv4_codes(const float *x, float s, bf16) {
    float inv;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));  // within one unit in the last place
    const float2 i2 = make_float2(inv, inv), zero = make_float2(0.f, 0.f), big = make_float2(1536.f, 1536.f),
                 less = make_float2(-1536.f, -1536.f);
    float y[8];
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        const float2 q = __ffma2_rn(make_float2(x[j], x[j + 1]), i2, zero);
        const float2 r = __fadd2_rn(__fadd2_rn(q, big), less);
        y[j] = copysignf(r.x, q.x);
        y[j + 1] = copysignf(r.y, q.y);
    }
    uint32_t w;
    asm("{\n.reg .b8 b0, b1, b2, b3;\n"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n"
        "mov.b32 %0, {b0, b1, b2, b3};\n}\n"
        : "=r"(w)
        : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
    return w;
}

}  // namespace medusa
