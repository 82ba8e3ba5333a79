// mx4.cuh -- the 4-bit numbers of the cache (dflash_mx4_cache.h has format and layout).
//
// E2M1 codes, 32 to a power of two 2^(s - 127) that one byte s holds. FP16 holds every code exactly, and
// its product with a power of two as long as that stays inside FP16's range: what the tensor core
// multiplies is exact.
#pragma once

#include <stdint.h>

#include "common.cuh"

namespace dflash {
namespace mx4 {

constexpr int kTokens = 16;        // tokens of a chunk
constexpr int kBlock = 32;         // elements of a scale
constexpr int kBlocks = kHeadDim / kBlock;
constexpr int kCodeBytes = kTokens * kHeadDim / 2;
constexpr int kChunkBytes = kCodeBytes + kTokens * kBlocks;  // 2176
constexpr int kNanScale = 255;

// Two codes (low half of the byte = first element) -> FP16x2 (low half = first element), exact. Byte kByte
// of a word.
template <int kByte>
__device__ __forceinline__ uint32_t codes_to_f16x2(uint32_t w) {
    uint32_t r;
    if constexpr (kByte == 0)
        asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %1;\n\t"
            "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t}" : "=r"(r) : "r"(w));
    else if constexpr (kByte == 1)
        asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %1;\n\t"
            "cvt.rn.f16x2.e2m1x2 %0, b1;\n\t}" : "=r"(r) : "r"(w));
    else if constexpr (kByte == 2)
        asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %1;\n\t"
            "cvt.rn.f16x2.e2m1x2 %0, b2;\n\t}" : "=r"(r) : "r"(w));
    else
        asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %1;\n\t"
            "cvt.rn.f16x2.e2m1x2 %0, b3;\n\t}" : "=r"(r) : "r"(w));
    return r;
}

// Eight numbers -> their codes, the first in the lowest half byte: round to nearest, ties to the even
// code, sizes above 6 to 6.
__device__ __forceinline__ uint32_t codes_of(const float (&x)[8]) {
    uint32_t r;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(r)
        : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
    return r;
}

// The scale byte of a block from the bits of its largest size (as an integer a NaN's are above an
// infinity's, and those above every number's): the smallest e with max <= 7 2^e = 1.75 2^(e + 2).
__device__ __forceinline__ int scale_of_max(uint32_t bits) {
    if (bits >= 0x7F800000u) return kNanScale;
    // (the exponent field of a subnormal is 0, and e = -127 is the least there is)
    const int s = (int)(bits >> 23) - 2 + ((bits & 0x007FFFFFu) > 0x00600000u ? 1 : 0);
    return s < 0 ? 0 : s;
}

// 2^-e of a scale byte that scale_of_max gives (at most 253: a normal number); 0 for a NaN block,
// whose codes are 0.
__device__ __forceinline__ float inverse_of_scale(int s) {
    return s == kNanScale ? 0.f : __int_as_float((254 - s) << 23);
}

// 2^(s - 127) as FP32 (byte 0 too: a subnormal number), NaN of byte 255.
__device__ __forceinline__ float power_of_scale(int s) {
    if (s == kNanScale) return __int_as_float(0x7FC00000);
    return s == 0 ? __int_as_float(0x00400000) : __int_as_float(s << 23);
}

// Where token t's code bytes and scales start in its chunk, and a chunk's place in its pool.
__device__ __forceinline__ int64_t chunk_offset(int64_t slot, int num_kv_heads, int h) {
    return ((slot / kTokens) * num_kv_heads + h) * kChunkBytes;
}

}  // namespace mx4
}  // namespace dflash
