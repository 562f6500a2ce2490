// The 4-bit KV-cache format: quantising a group, placing codes, reading them
// back.  Shared by the append, read-back and decode-attention kernels.
//
// A group is 32 consecutive dims of one token and kv-head (4 groups per row):
//     s = RN4(max|x| / 7)                  4 significant bits, nearest even
//     n = rne(x / s) clamped to -7 .. 7,   code = n + 8;   x^ = n * s
// RN4 moves s by at most a factor 1 +- 1/17, so max|x| / s < 7.5: no value is
// off by more than s / 2.  n has 3 significant bits and s 4, so n * s is a
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

namespace bi_kv4 {

constexpr int kBlockBytes = BI_KV4_BLOCK_BYTES;  // one (page, kv-head) block
constexpr int kScaleOffset = 1024;               // scales behind the codes
constexpr int kRowBytes = 64;                    // codes of one token
constexpr int kScaleRowBytes = 8;                // scales of one token
static_assert(kBlockBytes == BI_PAGE_SIZE * (kRowBytes + kScaleRowBytes), "block size");

// ---------------------------------------------------------------- reading ----
// A group's scale twice over, and -136 s twice over (17 * 8 * s: 8 significant
// bits, exact), from the scale's bf16 bits in the low half (kHigh: the high
// half) of `two`.
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

// scales of two elements (low, high half) -> the pair kv4_pair takes
__device__ __forceinline__ ScalePair scale_pair(uint32_t s2) {
    return {s2, mul_bf16x2(s2, kMinus136x2)};
}

// The values of the codes at bits 4p .. 4p + 3 of both halves of w, as
// bf16x2.  0x4300 | code is the bf16 number 128 + code; (128 + code) s - 136 s
// = (code - 8) s has one rounding, of an exact bf16 value.
__device__ __forceinline__ uint32_t kv4_pair(uint32_t w, int p, const ScalePair& sp) {
    uint32_t c;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;"  // (a & b) | c in one instruction
        : "=r"(c)
        : "r"(w >> (4 * p)), "r"(0x000F000Fu), "r"(0x43004300u));
    return fma_bf16x2(c, sp.s, sp.off);
}

// ---------------------------------------------------------------- writing ----
// s from the largest magnitude of the group (bits of |x| as an unsigned
// number, so that a NaN is largest of all)
__device__ __forceinline__ float group_scale(uint32_t amax_bits) {
    if (amax_bits >= 0x7D000000u) return __uint_as_float(0x7FFFFFFFu);  // 2^123 and more, inf, NaN
    if (amax_bits < 0x03800000u) return 0.f;                            // below 2^-120
    const uint32_t b = __float_as_uint(__fdiv_rn(__uint_as_float(amax_bits), 7.f));
    return __uint_as_float((b + 0x7FFFFu + ((b >> 20) & 1u)) & 0xFFF00000u);
}

// code = rne(x / s) + 8.  With inv = 1 / s correctly rounded, y = x * inv is
// within 2^-20 of x / s.  x / s (8 bits over 4) is a tie k + 1/2 exactly or at
// least 2^-9 away from one, so y rounded to multiples of 2^-11 (by adding and
// taking away 6144) lands on every tie and on the right side of the others,
// and the last addition rounds it to nearest even.  inv = 0 for s = 0 (n = 0),
// NaN for s = NaN (any code will do).
__device__ __forceinline__ uint32_t code_of(float x, float inv) {
    float y = __fmul_rn(x, inv);
    y = fminf(fmaxf(y, -7.f), 7.f);  // also takes a NaN away
    y = __fsub_rn(__fadd_rn(y, 6144.f), 6144.f);
    return __float_as_uint(__fadd_rn(y, 12582912.f + 8.f)) & 15u;
}

__device__ __forceinline__ uint32_t amax4(const float* x) {
    const uint32_t m = 0x7FFFFFFFu;
    return max(max(__float_as_uint(x[0]) & m, __float_as_uint(x[1]) & m),
               max(__float_as_uint(x[2]) & m, __float_as_uint(x[3]) & m));
}

// Quantise one row of 128 values held by a half-warp (lane l of 16: dims
// 4l .. 4l + 3 in x[0..3], dims 64 + 4l .. in x[4..7]; every lane of the warp
// takes part) and write it as token `off` of `block` where `live`.
template <bool kIsV>
__device__ __forceinline__ void write_row(const float (&x)[8], uint8_t* block, int off, int l,
                                          bool live) {
    constexpr uint32_t kAll = 0xffffffffu;
    uint32_t alo = amax4(x), ahi = amax4(x + 4);
#pragma unroll
    for (int o = 1; o <= 4; o <<= 1) {  // the 8 lanes of a group
        alo = max(alo, __shfl_xor_sync(kAll, alo, o));
        ahi = max(ahi, __shfl_xor_sync(kAll, ahi, o));
    }
    const float slo = group_scale(alo), shi = group_scale(ahi);
    const float ilo = slo == 0.f ? 0.f : __frcp_rn(slo), ihi = shi == 0.f ? 0.f : __frcp_rn(shi);
    uint32_t c[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        c[e] = code_of(x[e], ilo);
        c[4 + e] = code_of(x[4 + e], ihi);
    }
    // every lane adds its codes to several words; a reduce-scatter over the
    // lanes that share them leaves one whole word per lane
    uint32_t word;
    int at;  // its byte
    const bool b1 = l & 2, b2 = l & 4, b3 = l & 8;
    if (!kIsV) {
        const int sh = 4 * ((l & 7) >> 1);
        // words (t, j): t = 2 (l & 1) and the next, j = l / 8 and 2 more
        const uint32_t a0 = (c[0] | (c[1] << 16)) << sh, b0 = (c[2] | (c[3] << 16)) << sh;
        const uint32_t a1 = (c[4] | (c[5] << 16)) << sh, b1w = (c[6] | (c[7] << 16)) << sh;
        const uint32_t a = (b1 ? a1 : a0) | __shfl_xor_sync(kAll, b1 ? a0 : a1, 2);
        const uint32_t b = (b1 ? b1w : b0) | __shfl_xor_sync(kAll, b1 ? b0 : b1w, 2);
        word = (b2 ? b : a) | __shfl_xor_sync(kAll, b2 ? a : b, 4);
        at = kRowBytes * off + 16 * (2 * (l & 1) + (b2 ? 1 : 0)) + 4 * ((l >> 3) + (b1 ? 2 : 0));
    } else {
        const int sh = 4 * (l >> 1);
        // words (g, w): g = 4 (l & 1) + i, w = 0 for x[i], 1 for x[4 + i]
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            u[i] = ((b1 ? c[4 + i] : c[i]) << sh) |
                   __shfl_xor_sync(kAll, (b1 ? c[i] : c[4 + i]) << sh, 2);
        const uint32_t u0 = (b2 ? u[2] : u[0]) | __shfl_xor_sync(kAll, b2 ? u[0] : u[2], 4);
        const uint32_t u1 = (b2 ? u[3] : u[1]) | __shfl_xor_sync(kAll, b2 ? u[1] : u[3], 4);
        word = (b3 ? u1 : u0) | __shfl_xor_sync(kAll, b3 ? u0 : u1, 8);
        const int g = 4 * (l & 1) + (b2 ? 2 : 0) + (b3 ? 1 : 0);
        at = 512 * (off >> 3) + 64 * g + 8 * (off & 7) + (b1 ? 4 : 0);
    }
    // lane 0 holds the scales of groups 0 and 2, lane 8 those of 1 and 3
    const uint32_t mine = (__float_as_uint(slo) >> 16) | (__float_as_uint(shi) & 0xffff0000u);
    const uint32_t other = __shfl_xor_sync(kAll, mine, 8);
    if (!live) return;
    *reinterpret_cast<uint32_t*>(block + at) = word;
    if (l == 0)
        *reinterpret_cast<uint2*>(block + kScaleOffset + kScaleRowBytes * off) =
            make_uint2((mine & 0xffffu) | (other << 16), (mine >> 16) | (other & 0xffff0000u));
}

}  // namespace bi_kv4
