// The 4-bit KV-cache format: quantising a group, placing codes, reading them
// back.  Shared by the append, read-back and decode-attention kernels.
//
// A group is 32 consecutive dims of one token and kv-head (4 groups per row):
//     s = RN4(max|x| / 7)                  4 significant bits, nearest even
//     n = rne(x / s),   code = n + 8;      x^ = n * s
// RN4 moves s by at most a factor 1 +- 1/17, so max|x| / s < 7.5: n is within
// -7 .. 7 and no value is off by more than s / 2.  n has 3 significant bits and s 4, so n * s is a
// bf16 number: reading back rounds nothing, and attention over the codes can
// use the very operands that attention over a read-back bf16 cache would.  A
// scale with all 8 bits of a bf16 would cost a rounding per element (and the
// equality of the two), and its quantisation error is the same to 1 %: s
// wanders by 3 % rms around max|x| / 7, to either side.
// A group whose magnitudes are all below 2^-120 gets s = 0 and reads back as
// zeros (so s and 1 / s stay normal numbers); one with a NaN, an infinity or a
// magnitude of 2^123 and more gets s = NaN and reads back as NaN (soon after,
// 136 s of kv4_pair would leave bf16's range).
//
// One (page, kv-head) block of K or of V, kBlockBytes = 1152: 1024 bytes of
// codes, then bf16 scales [16 tokens][4 groups].  Codes lie in 32-bit words of
// 8 (code i at bits 4i .. 4i + 3), in the order in which a lane of mma.sync
// m16n8k16 holds them as its A operand:
//     K (rows = tokens, k = dims): dim 32j + 8p + 2t + e of token r is code
//       p + 4e of word 16r + 4t + j: lane (r % 8, t) finds its 32 dims of
//       token r in one 16-byte load, and word j holds group j alone;
//     V (rows = dims, k = tokens): dim 64w + 32h + 8p + g of token
//       8a + 2b + c is code 4h + p of word 128a + 16g + 4b + 2c + w: lane
//       (g, b) finds its 16 dims of tokens 2b and 2b + 1 in one 16-byte load.
#pragma once
#include <cuda_bf16.h>

#include <cstdint>

#include "bi_internal.h"
#include "bi_ptx.cuh"

namespace bi_kv4 {

constexpr int kBlockBytes = BI_KV4_BLOCK_BYTES;  // one (page, kv-head) block
constexpr int kScaleOffset = 1024;               // scales behind the codes
constexpr int kRowBytes = 64;                    // codes of one token
constexpr int kScaleRowBytes = 8;                // scales of one token
static_assert(kBlockBytes == BI_PAGE_SIZE * (kRowBytes + kScaleRowBytes), "block size");

// ---------------------------------------------------------------- reading ----
// The scales of two elements, and -136 s of both (17 * 8 * s: 8 significant
// bits, exact).
struct ScalePair {
    uint32_t s, off;
};

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}

constexpr uint32_t kMinus136x2 = 0xC308C308u;  // -136 as bf16, twice

__device__ __forceinline__ ScalePair scale_pair(uint32_t s2) {
    return {s2, mul_bf16x2(s2, kMinus136x2)};
}

// The values of the codes at bits 4p .. 4p + 3 of both halves of w, as
// bf16x2.  Putting an integer into the mantissa of a float of fixed exponent is the
// known way to convert small integers without a conversion instruction; here the
// subtraction of its exponent's value, of the codes' offset and the scale are one
// fma.  0x4300 | code is the bf16 number 128 + code; (128 + code) s - 136 s
// = (code - 8) s has one rounding, of an exact bf16 value.
__device__ __forceinline__ uint32_t kv4_pair(uint32_t w, int p, const ScalePair& sp) {
    uint32_t c;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;"  // (a & b) | c in one instruction
        : "=r"(c)
        : "r"(w >> (4 * p)), "r"(0x000F000Fu), "r"(0x43004300u));
    return fma_bf16x2(c, sp.s, sp.off);
}

// ---------------------------------------------------------------- writing ----
// A row of 128 bf16 values as a half-warp holds it: lane l of 16 has dims
// 4l .. 4l + 3 (lo) and 64 + 4l .. 64 + 4l + 3 (hi), two values a register.
struct RowPart {
    uint2 lo, hi;
};

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// s from the bf16 bits of the largest magnitude of the group (as a whole number,
// so that a NaN is largest of all).  amax * (1/7) is off by 2^-24 and would miss
// the ties of the rounding to 4 bits; those are 5-bit numbers and everything
// else is 2^-9 away from them, so rounding to 21 bits first puts them back.
__device__ __forceinline__ float group_scale(uint32_t amax_bits) {
    uint32_t b = __float_as_uint(__fmul_rn(__uint_as_float(amax_bits << 16), 1.f / 7.f));
    b = (b + 4u) & ~7u;
    b = (b + 0x7FFFFu + ((b >> 20) & 1u)) & 0xFFF00000u;
    if (amax_bits >= 0x7D00u) b = 0x7FFF0000u;  // 2^123 and more, inf, NaN
    if (amax_bits < 0x0380u) b = 0u;            // below 2^-120
    return __uint_as_float(b);
}

// 0x4B400000 + n + 8, n = rne(x / s).  inv is 1 / s to 1 ulp, so x * inv is
// within 2^-20 of x / s, which (8 bits over 4) is a tie k + 1/2 exactly or at
// least 2^-9 away from one: rounded to multiples of 2^-11 (the fma adds 6144)
// it lies on every tie and on the right side of the others.  The addition
// rounds that to nearest even.  inv = 0 for s = 0 (n = 0); for s = NaN the byte is
// 0xFF, which spoils codes of the same group only, and any code reads as NaN.
__device__ __forceinline__ uint32_t code_of(float x, float inv) {
    return __float_as_uint(__fadd_rn(__fmaf_rn(x, inv, 6144.f), 12582912.f + 8.f - 6144.f));
}

// The codes of four values (two registers of bf16 pairs), one a byte.
__device__ __forceinline__ uint32_t four_codes(uint2 v, float inv) {
    const uint32_t c0 = code_of(__uint_as_float(v.x << 16), inv);
    const uint32_t c1 = code_of(__uint_as_float(v.x & 0xffff0000u), inv);
    const uint32_t c2 = code_of(__uint_as_float(v.y << 16), inv);
    const uint32_t c3 = code_of(__uint_as_float(v.y & 0xffff0000u), inv);
    // a code's own byte, and a zero byte above it
    return __byte_perm(__byte_perm(c0, c1, 0x0040), __byte_perm(c2, c3, 0x0040), 0x5410);
}

// Quantise one row and write it as token `off` of `block` where `live`; every
// lane of the warp takes part.
template <bool kIsV>
__device__ __forceinline__ void write_row(const RowPart& r, uint8_t* block, int off, int l, bool live) {
    constexpr uint32_t kAll = 0xffffffffu, kAbs = 0x7FFF7FFFu;
    // largest magnitudes of the lo and the hi group side by side, over the 8
    // lanes of a group
    const uint32_t alo = max_u16x2(r.lo.x & kAbs, r.lo.y & kAbs);
    const uint32_t ahi = max_u16x2(r.hi.x & kAbs, r.hi.y & kAbs);
    uint32_t am = max_u16x2(__byte_perm(alo, ahi, 0x5410), __byte_perm(alo, ahi, 0x7632));
#pragma unroll
    for (int o = 1; o <= 4; o <<= 1) am = max_u16x2(am, __shfl_xor_sync(kAll, am, o));
    const float slo = group_scale(am & 0xffffu), shi = group_scale(am >> 16);
    const float ilo = slo == 0.f ? 0.f : bi::rcp_approx(slo);
    const float ihi = shi == 0.f ? 0.f : bi::rcp_approx(shi);
    const uint32_t clo = four_codes(r.lo, ilo), chi = four_codes(r.hi, ihi);
    // A lane's eight codes belong to eight words (V) or four (K).  Three
    // exchanges with the lanes 2, 4 and (V) 8 away, whose codes go into the same
    // words, leave every lane with one whole word: lanes keep the lo or the hi
    // codes, nibbles becoming bytes, then two of the four bytes, then a half.
    const bool b1 = l & 2, b2 = l & 4, b3 = l & 8;
    const uint32_t got = __shfl_xor_sync(kAll, b1 ? clo : chi, 2);
    const uint32_t even = b1 ? got : clo, odd = b1 ? chi : got;
    uint32_t word = even + 16u * odd;
    word = __byte_perm(word, __shfl_xor_sync(kAll, word, 4), b2 ? 0x3726 : 0x5140);
    int at;  // its byte
    if (!kIsV) {
        // word (t, j): t = 2 (l % 2) + b2, j = l / 8 + 2 b1
        at = kRowBytes * off + 16 * (2 * (l & 1) + (b2 ? 1 : 0)) + 4 * ((l >> 3) + (b1 ? 2 : 0));
    } else {
        word = __byte_perm(word, __shfl_xor_sync(kAll, word, 8), b3 ? 0x3276 : 0x5410);
        // word (g, w): g = 4 (l % 2) + 2 b2 + b3, w = b1
        const int g = 4 * (l & 1) + (b2 ? 2 : 0) + (b3 ? 1 : 0);
        at = 512 * (off >> 3) + 64 * g + 8 * (off & 7) + (b1 ? 4 : 0);
    }
    // lane 0 holds the scales of groups 0 and 2, lane 8 those of 1 and 3
    const uint32_t mine = __byte_perm(__float_as_uint(slo), __float_as_uint(shi), 0x7632);
    const uint32_t other = __shfl_xor_sync(kAll, mine, 8);
    if (!live) return;
    *reinterpret_cast<uint32_t*>(block + at) = word;
    if (l == 0)
        *reinterpret_cast<uint2*>(block + kScaleOffset + kScaleRowBytes * off) =
            make_uint2(__byte_perm(mine, other, 0x5410), __byte_perm(mine, other, 0x7632));
}

}  // namespace bi_kv4
