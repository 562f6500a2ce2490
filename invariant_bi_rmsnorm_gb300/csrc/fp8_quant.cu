// bi_quantize_fp8 and bi_fp8_read: bf16 rows to the 8-bit format and back.
//
// A warp holds 512 consecutive values of one row (two 16-byte vectors a lane),
// which is one 32-bit word of scale bytes: the four block maxima take one
// packed butterfly over the half-warps, and no value is read twice.  A row's
// bytes depend on that row alone.
//
// Bound by HBM: 3 bytes and 1/128 a value.  At 16384 x 4096 the quantiser takes
// 32.0 us (6.29 TB/s of its bytes) and the read-back 30.5 us (6.60 TB/s), against
// 6.75 TB/s of a plain copy; two thirds of the issue slots are taken.  One item a
// warp, not a loop over items: the grid's tail is under 1 % at that size, and a
// row of 4096 is 8 warps, so that one row already has a whole CTA's loads in
// flight.
#include <cuda_bf16.h>

#include "bi_internal.h"
#include "bi_ptx.cuh"
#include "fp8.cuh"

namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float lo16(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float hi16(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

// largest magnitude of 8 bf16 values, as bf16 bits (NaN above infinity above the rest)
__device__ __forceinline__ uint32_t amax8(const uint4& u) {
    const uint32_t a = __vmaxu2(u.x & 0x7fff7fffu, u.y & 0x7fff7fffu);
    const uint32_t b = __vmaxu2(u.z & 0x7fff7fffu, u.w & 0x7fff7fffu);
    const uint32_t m = __vmaxu2(a, b);
    return max(m & 0xffffu, m >> 16);
}

__device__ __forceinline__ uint2 codes8(const uint4& u, float inv) {
    return make_uint2(bi_fp8::codes4(__fmul_rn(lo16(u.x), inv), __fmul_rn(hi16(u.x), inv),
                                     __fmul_rn(lo16(u.y), inv), __fmul_rn(hi16(u.y), inv)),
                      bi_fp8::codes4(__fmul_rn(lo16(u.z), inv), __fmul_rn(hi16(u.z), inv),
                                     __fmul_rn(lo16(u.w), inv), __fmul_rn(hi16(u.w), inv)));
}

__global__ void __launch_bounds__(kThreads)
    quantize_kernel(const __nv_bfloat16* __restrict__ x, int64_t ld_x, int64_t items, int nvec,
                    int spans, uint8_t* __restrict__ q, int64_t ld_q,
                    uint8_t* __restrict__ scales) {
    bi::launch_dependents();
    bi::grid_dependency_wait();  // nothing global is touched before the previous kernel ends
    const int lane = threadIdx.x & 31;
    const int64_t item = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
    if (item >= items) return;  // whole warps
    const int64_t row = item / spans;
    const int span = static_cast<int>(item - row * spans);
    const uint4* xr = reinterpret_cast<const uint4*>(x + row * ld_x);
    uint2* qr = reinterpret_cast<uint2*>(q + row * ld_q);
    const int v0 = span * 64 + lane, v1 = v0 + 32;
    const uint4 none = make_uint4(0, 0, 0, 0);
    const uint4 a = v0 < nvec ? __ldcs(xr + v0) : none;
    const uint4 b = v1 < nvec ? __ldcs(xr + v1) : none;
    uint32_t m = amax8(a) | (amax8(b) << 16);  // both vectors' maxima in one word
#pragma unroll
    for (int o = 8; o >= 1; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
    // lanes 0-15 hold blocks 0 and 2 of the span, lanes 16-31 blocks 1 and 3
    const uint32_t b0 = bi_fp8::scale_byte(m << 16), b1 = bi_fp8::scale_byte(m & 0xffff0000u);
    const uint32_t mine = b0 | (b1 << 16);
    const uint32_t word = mine | (__shfl_xor_sync(0xffffffffu, mine, 16) << 8);
    if (lane == 0)
        *reinterpret_cast<uint32_t*>(scales + bi_fp8::scale_word(row, span, spans)) = word;
    if (v0 < nvec) qr[v0] = codes8(a, bi_fp8::inverse_scale(b0));
    if (v1 < nvec) qr[v1] = codes8(b, bi_fp8::inverse_scale(b1));
}

// two bf16 values from two e4m3 codes and the scale's bits: the code as fp16
// (exact), then one product by a power of two (exact: 4 significant bits; past
// bf16's largest number it is an infinity)
__device__ __forceinline__ uint32_t read2(uint32_t code2, float scale) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(code2)));
    float lo, hi;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(lo), "=f"(hi)
        : "r"(h));
    return bi::pack_bf16x2(__fmul_rn(lo, scale), __fmul_rn(hi, scale));
}

__global__ void __launch_bounds__(kThreads)
    read_kernel(const uint8_t* __restrict__ q, int64_t ld_q, const uint8_t* __restrict__ scales,
                int64_t items, int nvec, int spans, __nv_bfloat16* __restrict__ out,
                int64_t ld_out) {
    bi::launch_dependents();
    bi::grid_dependency_wait();
    const int lane = threadIdx.x & 31;
    const int64_t item = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
    if (item >= items) return;
    const int64_t row = item / spans;
    const int span = static_cast<int>(item - row * spans);
    const uint2* qr = reinterpret_cast<const uint2*>(q + row * ld_q);
    uint4* yr = reinterpret_cast<uint4*>(out + row * ld_out);
    const int v0 = span * 64 + lane, v1 = v0 + 32;
    const uint2 none = make_uint2(0, 0);
    const uint2 a = v0 < nvec ? __ldcs(qr + v0) : none;
    const uint2 b = v1 < nvec ? __ldcs(qr + v1) : none;
    const uint32_t word =
        *reinterpret_cast<const uint32_t*>(scales + bi_fp8::scale_word(row, span, spans));
    const uint32_t half = lane >> 4;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int v = i ? v1 : v0;
        if (v >= nvec) continue;
        const uint2 c = i ? b : a;
        const uint32_t byte = (word >> (16 * i + 8 * half)) & 255u;
        // 255 is an infinity's exponent; the codes beside it are NaN
        const float s = byte ? __uint_as_float(byte << 23) : 0x1p-127f;
        yr[v] = make_uint4(read2(c.x & 0xffffu, s), read2(c.x >> 16, s), read2(c.y & 0xffffu, s),
                           read2(c.y >> 16, s));
    }
}

bi_status check(int64_t rows, int32_t K, int64_t ld_a, int64_t ld_q, const void* a, const void* q,
                const void* scales) {
    if (rows < 0 || rows > 0x7fffffffLL) return BI_ERR_INVALID_ARG;
    if (K < 16 || (K & 15)) return BI_ERR_UNSUPPORTED_SHAPE;
    if (ld_a < K || ld_q < K) return BI_ERR_INVALID_ARG;
    if ((ld_a & 7) || (ld_q & 15)) return BI_ERR_MISALIGNED;
    if (rows == 0) return BI_OK;
    if (!a || !q || !scales) return BI_ERR_INVALID_ARG;
    if (!bi::aligned16(a) || !bi::aligned16(q) || !bi::aligned16(scales)) return BI_ERR_MISALIGNED;
    const int64_t items = rows * bi_fp8::spans_of(K);
    if (items > 0x7fffffffLL * (kThreads / 32)) return BI_ERR_UNSUPPORTED_SHAPE;  // the grid
    return BI_OK;
}

}  // namespace

extern "C" size_t bi_fp8_scales_size(int64_t rows, int32_t K) {
    if (rows < 0 || rows > 0x7fffffffLL || K < 16 || (K & 15)) return 0;
    return static_cast<size_t>((rows + 127) / 128) * bi_fp8::spans_of(K) * bi_fp8::kTileBytes;
}

extern "C" bi_status bi_quantize_fp8(const void* x, int64_t ld_x, int64_t rows, int32_t K, void* q,
                                     int64_t ld_q, void* scales, cudaStream_t stream) {
    const bi_status st = check(rows, K, ld_x, ld_q, x, q, scales);
    if (st != BI_OK || rows == 0) return st;
    const int spans = bi_fp8::spans_of(K);
    const int64_t items = rows * spans;
    const unsigned grid = static_cast<unsigned>((items + kThreads / 32 - 1) / (kThreads / 32));
    return bi::launch_pdl(quantize_kernel, dim3(grid), dim3(kThreads), 0, stream,
                          static_cast<const __nv_bfloat16*>(x), ld_x, items, K / 8, spans,
                          static_cast<uint8_t*>(q), ld_q, static_cast<uint8_t*>(scales)) == cudaSuccess
               ? BI_OK
               : BI_ERR_CUDA;
}

extern "C" bi_status bi_fp8_read(const void* q, int64_t ld_q, const void* scales, int64_t rows,
                                 int32_t K, void* out, int64_t ld_out, cudaStream_t stream) {
    const bi_status st = check(rows, K, ld_out, ld_q, out, q, scales);
    if (st != BI_OK || rows == 0) return st;
    const int spans = bi_fp8::spans_of(K);
    const int64_t items = rows * spans;
    const unsigned grid = static_cast<unsigned>((items + kThreads / 32 - 1) / (kThreads / 32));
    return bi::launch_pdl(read_kernel, dim3(grid), dim3(kThreads), 0, stream,
                          static_cast<const uint8_t*>(q), ld_q, static_cast<const uint8_t*>(scales),
                          items, K / 8, spans, static_cast<__nv_bfloat16*>(out), ld_out) == cudaSuccess
               ? BI_OK
               : BI_ERR_CUDA;
}
