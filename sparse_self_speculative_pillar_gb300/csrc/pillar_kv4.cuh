// pillar_kv4.cuh -- the 4-bit cache's number formats.
//
// A value is e2m1(code) * scale.  Codes: sign, two exponent bits of bias 1, one
// fraction bit (magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6).  A scale byte holds five
// exponent bits of bias 15 and three fraction bits: it is an f16 value without
// its sign and its low seven fraction bits.  Every product of the two has at most
// six significant bits and lies between 2^-18 and 61440, so it is exact in f16 and
// in bf16.
#pragma once

#include "pillar_device.cuh"

namespace pillar {

constexpr int kGroup4 = PILLAR_KV4_GROUP;  // values of a row that share a scale byte
constexpr int kTopScale = 226;             // the byte of 1.25 * 2^13: six times that is the last one f16 holds

// Eight codes (the word's nibbles from the lowest on) as four f16 pairs.
__device__ __forceinline__ void f16_of_e2m1(uint32_t w, uint32_t (&h)[4]) {
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
}

// Byte i of a word of scale bytes as an f16 pair of that scale.
__device__ __forceinline__ uint32_t scale_pair(uint32_t bytes, int i) {
    return __byte_perm(bytes, 0, 0x0404 | (i << 4) | (i << 12)) >> 1;  // byte << 8, halved in place: byte << 7
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

}  // namespace pillar
