// The 8-bit format (include/bi.h, "8-bit matrices") on the device: the scale
// byte of a block, the codes of its values, and where a scale byte lies.
#pragma once
#include <cstdint>

#include "bi_internal.h"
#include "bi_ptx.cuh"

namespace bi_fp8 {

constexpr int kBlock = BI_FP8_BLOCK;          // values that share a scale
constexpr int kSpan = 4 * BI_FP8_BLOCK;       // values of a row in one scale tile
constexpr int kTileBytes = BI_FP8_TILE_BYTES; // 128 rows x 4 blocks of scale bytes

// Scale byte of a block whose largest magnitude has these fp32 bits: the least
// b >= 8 with max|x| <= 448 * 2^(b - 127).  448 = 1.75 * 2^8, so the exponent
// less 8, and one more where the mantissa is above 1.75 (the add carries).  Bits
// from 0x7F800000 up (an infinity or a NaN in the block; integer order puts
// them last) give 255, for which the block stands for NaN.  From 8 up the
// scale's reciprocal is a normal fp32 number; magnitudes below 2^-129 become 0.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax_bits) {
    if (amax_bits >= 0x7F800000u) return 255u;
    return max((amax_bits + 0x1FFFFFu) >> 23, 16u) - 8u;
}

// max(|a|, |b|, |c|), NaN if one is: one instruction.
__device__ __forceinline__ float max3_abs(float a, float b, float c) {
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// {a * b, c * d}, each rounded to nearest, in one instruction.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "mul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}

// 2^(127 - b), by which a block's values are multiplied (exactly, but for
// results below 2^-126, which become the code 0 either way); NaN for b = 255,
// which makes every code of the block NaN.
__device__ __forceinline__ float inverse_scale(uint32_t b) {
    return b == 255u ? __uint_as_float(0x7FC00000u) : __uint_as_float((254u - b) << 23);
}

// Two e4m3 codes, lo in the low byte: the one rounding (to nearest even).
__device__ __forceinline__ uint32_t codes2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
    return codes2(a, b) | (codes2(c, d) << 16);
}

// Offset of the scale bytes of row `row`, blocks 4 * span .. 4 * span + 3, in
// tiles [ceil(rows / 128)][spans][512].
__device__ __forceinline__ int64_t scale_word(int64_t row, int span, int spans) {
    return ((row >> 7) * spans + span) * kTileBytes + (row & 31) * 16 + ((row >> 5) & 3) * 4;
}

inline int spans_of(int64_t K) { return static_cast<int>((K + kSpan - 1) / kSpan); }

}  // namespace bi_fp8
