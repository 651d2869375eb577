// fp4.cuh -- the formats of a cache held in 4 bits: codes of 4 bits (sign, 2
// bits of exponent, 1 of mantissa: 0, 1/2, 1, 3/2, 2, 3, 4, 6) and scales of 8
// (4 bits of exponent, 3 of mantissa).  The GPU converts both to fp16 exactly;
// a code times a scale has 6 significant bits and lies between 2^-10 and 2688, so
// the product is exact in fp16 too.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

namespace dspark {
namespace fp4 {

constexpr int kGroup = 16;               // entries that share a scale

// The 8 codes of a word as 4 fp16 pairs, lower entries first.
__device__ __forceinline__ void unpack(uint32_t w, uint32_t (&h)[4]) {
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3]) : "r"(w));
}

// Two scales (the low 16 bits of w) as an fp16 pair.
__device__ __forceinline__ uint32_t scale_pair(uint32_t w) {
    uint32_t h;
    asm("{\n\t.reg .b16 s;\n\tcvt.u16.u32 s, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, s;\n\t}" : "=r"(h) : "r"(w));
    return h;
}
__device__ __forceinline__ float scale_value(uint32_t byte) {
    const uint32_t h = scale_pair(byte);
    return __half2float(__ushort_as_half((unsigned short)(h & 0xffffu)));
}

__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ float2 floats(uint32_t h) {
    __half2 x;
    *reinterpret_cast<uint32_t*>(&x) = h;
    return __half22float2(x);
}

// The scale nearest to x >= 0 (ties to even), at most 448; NaN stays NaN.
__device__ __forceinline__ uint32_t scale_code(float x) {
    uint32_t r;
    asm("{\n\t.reg .b16 s;\n\tcvt.rn.satfinite.e4m3x2.f32 s, %1, %1;\n\tcvt.u32.u16 %0, s;\n\t}" : "=r"(r) : "f"(x));
    return r & 0xffu;
}

// The levels nearest to 8 numbers (ties to the even code, at most 6), as a word.
__device__ __forceinline__ uint32_t pack(const float (&x)[8]) {
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r) : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
    return r;
}

}  // namespace fp4
}  // namespace dspark
