// kv4.cuh -- the 4-bit cache format, shared by the kernels that write and read it.
//
// 16 consecutive channels of one token's head are a group.  A group holds 16 e2m1 codes (values
// 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives, two a byte, the lower channel in the low half)
// and one e4m3 scale s; code c stands for e2m1(c) * s * u, with u a power of two given for all
// keys or all values of the cache.  e2m1 has two significant bits and e4m3 four, so e2m1 * s is
// exact in fp16 (at most 6 * 448, at least 0.5 * 2^-9).  A scale that is NaN marks a group that
// held an infinity or a NaN.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace bsattn {

constexpr int kGroup4 = 16;
constexpr uint32_t kNanScale4 = 0x7fu;

// The four code pairs (bytes) of a word as fp16 pairs, low half = low code.
__device__ __forceinline__ void e2m1_word_to_f16(uint32_t w, uint32_t& r0, uint32_t& r1, uint32_t& r2,
                                                 uint32_t& r3) {
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
        : "r"(w));
}

// Two e4m3 scales (low 16 bits) as an fp16 pair.
__device__ __forceinline__ uint32_t e4m3x2_to_f16(uint32_t two) {
    uint32_t r;
    asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(r) : "r"(two));
    return r;
}

// Eight values to eight codes in a word, rounded to nearest (ties to even), saturated at 6.
__device__ __forceinline__ uint32_t f32x8_to_e2m1(const float (&x)[8]) {
    uint32_t w;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(w)
        : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
    return w;
}

// One value to e4m3, rounded to nearest (ties to even), saturated at 448.
__device__ __forceinline__ uint32_t f32_to_e4m3(float x) {
    uint32_t r;
    asm("{\n\t.reg .b16 t;\n\tcvt.rn.satfinite.e4m3x2.f32 t, %1, %2;\n\tcvt.u32.u16 %0, t;\n\t}"
        : "=r"(r)
        : "f"(0.f), "f"(x));
    return r & 0xffu;
}

__device__ __forceinline__ uint32_t hmul2_u32(uint32_t a, uint32_t b) {
    __half2 r = __hmul2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
    return *reinterpret_cast<uint32_t*>(&r);
}

// A scale the cache can be held in units of: a power of two in [2^-16, 2^16].
inline bool unit_ok4(float u) {
    uint32_t b;
    static_assert(sizeof(b) == sizeof(u), "32-bit float");
    __builtin_memcpy(&b, &u, sizeof(b));
    const int e = static_cast<int>(b >> 23) - 127;
    return (b & 0x807fffffu) == 0 && e >= -16 && e <= 16;
}

}  // namespace bsattn
