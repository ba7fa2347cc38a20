// kda_latent_q8.cuh -- a row of the 8-bit latent cache: e4m3 numbers y and one power of two 2^e, values y 2^e.
//
//     e = the smallest integer with max |x| <= 448 2^e, within kLeastPower .. kMostPower,   y = e4m3(x 2^-e).
//
// e4m3 is a floating format: a power of two costs it no precision, only range (the largest number of a row lies above
// 224), the scaling is exact, so that y is rounded once, and a value has four significant bits and is exact in bf16.
// The bounds keep 2^e and 2^-e normal fp32 numbers, and sums of 2^-e over 2^31 rows finite.  A row of zeros takes the
// lowest e: it never sets the range of the softmax weights of the rows beside it.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace kda {
namespace latent {

constexpr int kLeastPower = -64, kMostPower = 120;

// 2^e for -126 <= e <= 127.
__device__ __forceinline__ float two_to(int e) { return __int_as_float((e + 127) << 23); }

// e for the largest magnitude of a row, given by its bits (which order as magnitudes do, NaN above infinity).
// 448 = 1.75 * 2^8.
__device__ __forceinline__ int power_for(uint32_t bits) {
    const int e = (int)(bits >> 23) - 127 - ((bits & 0x7fffffu) <= 0x600000u ? 8 : 7);
    return bits == 0 || e < kLeastPower ? kLeastPower : (e > kMostPower ? kMostPower : e);
}

// The scale byte of a row (e8m0: e + 127), and e of a byte; bytes outside the format's range count as its nearest.
__device__ __forceinline__ uint8_t power_byte(int e) { return (uint8_t)(e + 127); }
__device__ __forceinline__ int power_of(uint8_t byte) {
    const int e = (int)byte - 127;
    return e < kLeastPower ? kLeastPower : (e > kMostPower ? kMostPower : e);
}

// Four numbers to e4m3, a in the low byte: to nearest even, beyond 448 to 448.
__device__ __forceinline__ uint32_t to_e4m3x4(float a, float b, float c, float d) {
    uint32_t r;
    asm("{\n\t.reg .b16 l, u;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 u, %4, %3;\n\t"
        "mov.b32 %0, {l, u};\n\t}"
        : "=r"(r)
        : "f"(a), "f"(b), "f"(c), "f"(d));
    return r;
}
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
// The same from and to fp16, two numbers a word.
__device__ __forceinline__ uint32_t to_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t sub_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t add_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t fma_f16x2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t r;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}
constexpr uint32_t k128 = 0x58005800u;        // (2^7, 2^7)
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t f16_to_e4m3x4(uint32_t lo, uint32_t hi) {
    uint32_t r;
    asm("{\n\t.reg .b16 l, u;\n\t"
        "cvt.rn.satfinite.e4m3x2.f16x2 l, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f16x2 u, %2;\n\t"
        "mov.b32 %0, {l, u};\n\t}"
        : "=r"(r)
        : "r"(lo), "r"(hi));
    return r;
}
__device__ __forceinline__ uint32_t f16_to_e5m2x4(uint32_t lo, uint32_t hi) {
    uint32_t r;
    asm("{\n\t.reg .b16 l, u;\n\t"
        "cvt.rn.satfinite.e5m2x2.f16x2 l, %1;\n\t"
        "cvt.rn.satfinite.e5m2x2.f16x2 u, %2;\n\t"
        "mov.b32 %0, {l, u};\n\t}"
        : "=r"(r)
        : "r"(lo), "r"(hi));
    return r;
}
// Four e4m3 numbers, exactly.
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t x, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 l, u;\n\t"
        "mov.b32 {l, u}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, u;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(x));
}
__device__ __forceinline__ void e5m2x4_to_f16(uint32_t x, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 l, u;\n\t"
        "mov.b32 {l, u}, %2;\n\t"
        "cvt.rn.f16x2.e5m2x2 %0, l;\n\t"
        "cvt.rn.f16x2.e5m2x2 %1, u;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(x));
}
__device__ __forceinline__ float2 f16x2_to_floats(uint32_t x) {
    float2 f;
    asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, u;\n\t}"
        : "=f"(f.x), "=f"(f.y)
        : "r"(x));
    return f;
}

}  // namespace latent
}  // namespace kda
