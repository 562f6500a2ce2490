// bi_rmsnorm: data-parallel RMSNorm, one row per CTA.
//
// "Defeating Nondeterminism in LLM Inference: The Core Role of Batch
// Invariance", section "1. Batch-Invariant RMSNorm": keeping each row's whole
// reduction inside one core makes its order independent of the batch size;
// splitting one row over several cores at small batch would change it, so
// that is never done here.
//
// Reduction order (a function of `hidden` only):
//   1. thread t owns the 16-byte vectors t, t+T, t+2T, ... of the row
//      (T = threads per CTA); it sums x^2 over its vectors in that order,
//      each vector's 8 elements left to right, with fused multiply-adds;
//   2. each warp folds its 32 partials with an xor butterfly (16,8,4,2,1) and
//      lane 0's result is taken;
//   3. every thread folds the per-warp sums in warp order 0, 1, 2, ...
// (hidden 4096: T = 256 threads, 2 vectors each.)
// Then r = rsqrt(sum / hidden + eps) and y = bf16_rn((x * r) * w) in fp32.
#include <cuda_bf16.h>

#include "bi_internal.h"
#include "bi_ptx.cuh"
#include "fp8.cuh"

namespace {

// 256 threads per row: each thread keeps two 16-byte loads in flight at
// hidden 4096, and 8 rows (CTAs) fit on an SM, which is what it takes to keep
// HBM busy with one row per CTA (512 threads x 1 load left it latency-bound).
constexpr int kMaxThreads = 256;

// Rows resident at once are few (8 CTAs per SM, 8 KiB each at hidden 4096),
// which leaves HBM short of requests. Each CTA therefore asks L2 to fetch the
// input of the row about kPrefetchAheadBytes of input ahead of its own; that
// row's CTA then finds it in L2. A prefetch moves data only: the arithmetic
// and its order are the same whether it hits or not.
// 16 MiB was the best of 0-40 MiB on GB300 at 16384 x 4096, plain and fused.
constexpr int64_t kPrefetchAheadBytes = int64_t{16} << 20;

__device__ __forceinline__ void prefetch_l2(const void* p, uint32_t bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}

__device__ __forceinline__ float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

// kAdd: the fused form -- first res = bf16(res + x) (fp32 add, one rounding),
// stored back, then the RMSNorm of that sum with exactly the reduction below.
// kFp8: (x * r) * w goes to 8 bits instead of bf16, rounded once (fp8.cuh): the
// 16 threads that hold a block of 128 values find its largest magnitude by a
// butterfly, and the row's scale bytes leave by way of shared memory, a word of
// four at a time.  16384 x 4096: 41.5 us plain (3 bytes a value, 4.85 TB/s) and 69.9
// us with the sum (7 bytes a value, 6.72 TB/s of HBM's 6.75).  The plain form is bound by
// issue, 83 % of the slots: a thread takes 98 instructions a vector and 120 more that
// do not depend on how many it has (the sums' folds, the division and the root, two barriers,
// the scale words, addresses), and at 4096 values it has two.  At 8192 values, four a thread,
// the instructions are a fifth fewer and the registers (52 for 32) halve the warps: the same
// time for the same bytes.  Two products or three maxima an
// instruction (fp8.cuh) took the plain form from 44.6 to 41.0 us; bytes stored without
// the step through shared memory cost more in long rows (hidden 12288: 82.6 ->
// 96.6 us for 16384 rows).
// kFew, for up to 512 rows: the weight is asked for before the sum is known, which saves a wait
// (4096 values, one row 2.3 -> 2.0 us, 300 rows with the sum 4.6 -> 3.9; 16384 values, one row
// 4.5 -> 3.4) and costs registers, which more rows miss (16384 x 4096 41.5 -> 43.2, 4096 x
// 16384 44.3 -> 51.9).
struct Fp8Out {
    uint8_t* scales;
    int spans;
    __nv_bfloat16* res_out;  // where the sum goes: res itself, or another buffer
    int64_t ld_res_out;
};

// bf16(a + b) of 8 values: fp32 sums, one rounding
__device__ __forceinline__ uint4 add8(const uint4& a, const uint4& b) {
    const uint32_t au[4] = {a.x, a.y, a.z, a.w}, bu[4] = {b.x, b.y, b.z, b.w};
    uint32_t o[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
        o[e] = bi::pack_bf16x2(__fadd_rn(bf16_lo(bu[e]), bf16_lo(au[e])),
                               __fadd_rn(bf16_hi(bu[e]), bf16_hi(au[e])));
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// s plus the squares of 8 values, left to right
__device__ __forceinline__ float add_squares(float s, const uint4& x) {
    const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float a = bf16_lo(u[e]), b = bf16_hi(u[e]);
        s = __fmaf_rn(a, a, s);
        s = __fmaf_rn(b, b, s);
    }
    return s;
}

// The 8 values (x * r) * w as codes at `to`, `in` the row; the scale byte of their block, which
// 16 neighbouring threads hold.  All of a warp's threads come here.
__device__ __forceinline__ uint32_t put_block(const uint4& x, const uint4& w, float r, bool in,
                                              uint2* to) {
    const uint32_t xu[4] = {x.x, x.y, x.z, x.w}, wu[4] = {w.x, w.y, w.z, w.w};
    float2 f[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
        f[e] = bi_fp8::mul2(bi_fp8::mul2(make_float2(bf16_lo(xu[e]), bf16_hi(xu[e])),
                                         make_float2(r, r)),
                            make_float2(bf16_lo(wu[e]), bf16_hi(wu[e])));
    float most = bi_fp8::max3_abs(f[0].x, f[0].y, f[1].x);
    most = bi_fp8::max3_abs(most, f[1].y, f[2].x);
    most = bi_fp8::max3_abs(most, f[2].y, f[3].x);
    most = bi_fp8::max3_abs(most, f[3].y, f[3].y);
    // threads past the row's end hold zeros of no row, and must not bring in 0 * r = NaN;
    // as integers NaN comes after infinity and that after the rest
    uint32_t top = in ? __float_as_uint(most) : 0u;
#pragma unroll
    for (int o = 8; o >= 1; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    const uint32_t b = bi_fp8::scale_byte(top);
    if (in) {
        const float inv = bi_fp8::inverse_scale(b);
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = bi_fp8::mul2(f[e], make_float2(inv, inv));
        *to = make_uint2(bi_fp8::codes4(f[0].x, f[0].y, f[1].x, f[1].y),
                         bi_fp8::codes4(f[2].x, f[2].y, f[3].x, f[3].y));
    }
    return b;
}

template <int VPT, bool kAdd, bool kFp8, bool kFew = false>
__global__ void __launch_bounds__(kMaxThreads)
    rmsnorm_kernel(const __nv_bfloat16* x, const __nv_bfloat16* __restrict__ w, void* y,
                   int hidden, int64_t ld_x, int64_t ld_y, float eps, __nv_bfloat16* res,
                   int64_t ld_res, int64_t rows, int64_t ahead, Fp8Out fp8) {
    bi::launch_dependents();
    bi::grid_dependency_wait();  // nothing global is touched before the previous kernel ends
    __shared__ float warp_sums[kMaxThreads / 32];
    const int nvec = hidden >> 3;
    const int tid = threadIdx.x;
    const int T = blockDim.x;
    const int64_t row = blockIdx.x;
    const uint4* xr = reinterpret_cast<const uint4*>(x + row * ld_x);
    const uint4* wr = reinterpret_cast<const uint4*>(w);

    if (tid == 0 && ahead > 0 && row + ahead < rows) {
        prefetch_l2(x + (row + ahead) * ld_x, static_cast<uint32_t>(hidden) * 2u);
        if constexpr (kAdd)
            prefetch_l2(res + (row + ahead) * ld_res, static_cast<uint32_t>(hidden) * 2u);
    }

    uint4 xv[VPT];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int v = tid + j * T;
        xv[j] = (v < nvec) ? __ldcs(xr + v) : make_uint4(0, 0, 0, 0);
    }
    if constexpr (kAdd) {
        const uint4* rr = reinterpret_cast<const uint4*>(res + row * ld_res);
        uint4* ro = reinterpret_cast<uint4*>(kFp8 ? fp8.res_out + row * fp8.ld_res_out
                                                  : res + row * ld_res);
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int v = tid + j * T;
            if (v >= nvec) continue;
            xv[j] = add8(xv[j], rr[v]);
            ro[v] = xv[j];
        }
    }

    uint4 wv[kFew ? VPT : 1];
    if constexpr (kFew) {
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int v = tid + j * T;
            wv[j] = v < nvec ? __ldg(wr + v) : make_uint4(0, 0, 0, 0);
        }
    }
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) s = add_squares(s, xv[j]);
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    if ((tid & 31) == 0) warp_sums[tid >> 5] = s;
    __syncthreads();
    const int nwarps = T >> 5;
    float total = warp_sums[0];
    for (int i = 1; i < nwarps; ++i) total += warp_sums[i];
    const float r = rsqrtf(__fdiv_rn(total, static_cast<float>(hidden)) + eps);

    if constexpr (kFp8) {
        __shared__ uint8_t s_byte[32768 / bi_fp8::kBlock];
        uint2* qr = reinterpret_cast<uint2*>(static_cast<uint8_t*>(y) + row * ld_y);
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int v = tid + j * T;
            if constexpr (!kFew) wv[0] = v < nvec ? __ldg(wr + v) : make_uint4(0, 0, 0, 0);
            const uint32_t b = put_block(xv[j], wv[kFew ? j : 0], r, v < nvec, qr + v);
            if (v < nvec && (tid & 15) == 0) s_byte[v >> 4] = static_cast<uint8_t>(b);
        }
        __syncthreads();
        for (int i = tid; i < fp8.spans; i += T) {
            uint32_t word = 0;
#pragma unroll
            for (int c = 0; c < 4; ++c)
                if (4 * i + c < (nvec + 15) >> 4) word |= static_cast<uint32_t>(s_byte[4 * i + c]) << (8 * c);
            *reinterpret_cast<uint32_t*>(fp8.scales + bi_fp8::scale_word(row, i, fp8.spans)) = word;
        }
        return;
    }
    uint4* yr = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(y) + row * ld_y);
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int v = tid + j * T;
        if (v >= nvec) continue;
        const uint4 wv = __ldg(wr + v);
        const uint32_t xu[4] = {xv[j].x, xv[j].y, xv[j].z, xv[j].w};
        const uint32_t wu[4] = {wv.x, wv.y, wv.z, wv.w};
        uint32_t o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float a = __fmul_rn(__fmul_rn(bf16_lo(xu[e]), r), bf16_lo(wu[e]));
            const float b = __fmul_rn(__fmul_rn(bf16_hi(xu[e]), r), bf16_hi(wu[e]));
            o[e] = bi::pack_bf16x2(a, b);
        }
        yr[v] = make_uint4(o[0], o[1], o[2], o[3]);
    }
}

// The 8-bit norm of short rows, a warp a row: the grid above starts a CTA a row, and starting
// them takes 1.03 ns each, whatever a row's length (16384 rows of 16 values 16.9 us).  Lane l
// holds the vectors l, l + 32, ... that thread l of each of the other kernel's W warps would, and
// takes each of those warps' sums and its butterfly by itself, so every sum has its order; warps past
// the row's end add 0.
template <int W, bool kAdd>
__global__ void __launch_bounds__(256, 3)
    rmsnorm_fp8_rows_kernel(const __nv_bfloat16* x, const __nv_bfloat16* __restrict__ w, uint8_t* q,
                            int hidden, int64_t ld_x, int64_t ld_q, float eps,
                            const __nv_bfloat16* res, int64_t ld_res, int64_t rows, Fp8Out fp8) {
    bi::launch_dependents();
    bi::grid_dependency_wait();  // nothing global is touched before the previous kernel ends
    const int64_t row = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    if (row >= rows) return;  // whole warps
    const int lane = threadIdx.x & 31;
    const int nvec = hidden >> 3;
    const uint4* xr = reinterpret_cast<const uint4*>(x + row * ld_x);
    const uint4* wr = reinterpret_cast<const uint4*>(w);
    uint2* qr = reinterpret_cast<uint2*>(q + row * ld_q);

    uint4 xv[W];
#pragma unroll
    for (int i = 0; i < W; ++i) {
        const int v = lane + 32 * i;
        xv[i] = v < nvec ? __ldcs(xr + v) : make_uint4(0, 0, 0, 0);
    }
    if constexpr (kAdd) {
        const uint4* rr = reinterpret_cast<const uint4*>(res + row * ld_res);
        uint4* ro = reinterpret_cast<uint4*>(fp8.res_out + row * fp8.ld_res_out);
        uint4 rv[W];  // all read before any is written: res_out may be res
#pragma unroll
        for (int i = 0; i < W; ++i) {
            const int v = lane + 32 * i;
            rv[i] = v < nvec ? rr[v] : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < W; ++i) {
            const int v = lane + 32 * i;
            xv[i] = add8(xv[i], rv[i]);
            if (v < nvec) ro[v] = xv[i];
        }
    }

    float s[W];
#pragma unroll
    for (int i = 0; i < W; ++i) s[i] = add_squares(0.f, xv[i]);
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1)
#pragma unroll
        for (int i = 0; i < W; ++i) s[i] += __shfl_xor_sync(0xffffffffu, s[i], off);
    float total = s[0];
#pragma unroll
    for (int i = 1; i < W; ++i) total += s[i];
    const float r = rsqrtf(__fdiv_rn(total, static_cast<float>(hidden)) + eps);

    uint32_t word = 0;
#pragma unroll
    for (int i = 0; i < W; ++i) {
        const int v = lane + 32 * i;
        const uint32_t b = put_block(xv[i], v < nvec ? __ldg(wr + v) : make_uint4(0, 0, 0, 0), r,
                                     v < nvec, qr + v);
        word |= ((v & ~15) < nvec ? b : 0u) << (16 * (i & 1));  // lanes 0-15's block, or 16-31's
        if ((i & 1) == 0 && i + 1 < W) continue;
        word |= __shfl_xor_sync(0xffffffffu, word, 16) << 8;
        if (lane == 0 && i / 2 < fp8.spans)
            *reinterpret_cast<uint32_t*>(fp8.scales + bi_fp8::scale_word(row, i / 2, fp8.spans)) = word;
        word = 0;
    }
}

}  // namespace

namespace {

template <bool kAdd, bool kFp8>
bi_status launch_rmsnorm(const void* x, const void* w, void* y, int64_t rows, int32_t hidden,
                         int64_t ld_x, int64_t ld_y, float eps, void* res, int64_t ld_res,
                         const Fp8Out& fp8, cudaStream_t stream) {
    constexpr int kMask = kFp8 ? 15 : 7;  // 16-byte rows of y
    if (rows < 0 || rows > 0x7fffffffLL) return BI_ERR_INVALID_ARG;
    if (!(eps >= 0.f) || eps != eps || eps > 3.0e38f) return BI_ERR_INVALID_ARG;
    if (hidden < 8 || hidden > 32768 || (hidden & kMask)) return BI_ERR_UNSUPPORTED_SHAPE;
    if (ld_x < hidden || ld_y < hidden) return BI_ERR_INVALID_ARG;
    if ((ld_x & 7) || (ld_y & kMask)) return BI_ERR_MISALIGNED;
    if (kAdd && ld_res < hidden) return BI_ERR_INVALID_ARG;
    if (kAdd && (ld_res & 7)) return BI_ERR_MISALIGNED;
    if (kAdd && kFp8 && fp8.ld_res_out < hidden) return BI_ERR_INVALID_ARG;
    if (kAdd && kFp8 && (fp8.ld_res_out & 7)) return BI_ERR_MISALIGNED;
    if (rows == 0) return BI_OK;
    if (!x || !w || !y || (kAdd && !res) || (kFp8 && !fp8.scales) || (kAdd && kFp8 && !fp8.res_out))
        return BI_ERR_INVALID_ARG;
    if (!bi::aligned16(x) || !bi::aligned16(w) || !bi::aligned16(y) ||
        (kAdd && !bi::aligned16(res)) || (kFp8 && !bi::aligned16(fp8.scales)) ||
        (kAdd && kFp8 && !bi::aligned16(fp8.res_out)))
        return BI_ERR_MISALIGNED;

    // Thread count and vectors per thread depend on `hidden` alone.
    const int nvec = hidden / 8;
    int threads, vpt;
    if (nvec <= kMaxThreads) {
        threads = (nvec + 31) / 32 * 32;
        vpt = 1;
    } else {
        threads = kMaxThreads;
        vpt = (nvec + kMaxThreads - 1) / kMaxThreads;  // 2 .. 16
    }
    const auto* xb = static_cast<const __nv_bfloat16*>(x);
    const auto* wb = static_cast<const __nv_bfloat16*>(w);
    auto* rb = static_cast<__nv_bfloat16*>(res);
    const dim3 grid(static_cast<unsigned>(rows));
    const int64_t ahead = kPrefetchAheadBytes / (int64_t{hidden} * 2 * (kAdd ? 2 : 1));
    const auto launch = [&](auto kernel) {
        return bi::launch_pdl(kernel, grid, dim3(threads), 0, stream, xb, wb, y, hidden, ld_x, ld_y,
                              eps, rb, ld_res, rows, ahead, fp8);
    };
    cudaError_t err;
    if constexpr (kFp8) {
        // Measured, us, plain / with the sum, a CTA a row against a warp a row: 512 values, 304 rows
        // 2.1 / 2.2 against 2.0 / 2.3, 16384 rows 16.9 / 17.0 against 5.9 / 7.5; 1024 values, 1216 rows
        // 2.9 / 3.2 against 2.9 / 3.4, 2432 rows 4.4 / 5.0 against 3.1 / 4.1; 2048 values, 4864 rows
        // 9.4 / 11.0 against 9.1 / 11.8, 16384 rows 27.8 / 36.7 against 20.7 / 38.2; 4096 values, 16384
        // rows 41.1 against 56.1.
        const auto launch_rows = [&](auto kernel) {
            return bi::launch_pdl(kernel, dim3(static_cast<unsigned>((rows + 7) / 8)), dim3(256), 0, stream, xb,
                                  wb, static_cast<uint8_t*>(y), hidden, ld_x, ld_y, eps, rb, ld_res, rows, fp8);
        };
        const bool a_warp_a_row = hidden <= 512 || (hidden <= 1024 && rows >= 2048) ||
                                  (!kAdd && hidden <= 2048 && rows >= 8192);
        if (a_warp_a_row) {
            if (hidden <= 256)
                err = launch_rows(rmsnorm_fp8_rows_kernel<1, kAdd>);
            else if (hidden <= 512)
                err = launch_rows(rmsnorm_fp8_rows_kernel<2, kAdd>);
            else if (kAdd || hidden <= 1024)
                err = launch_rows(rmsnorm_fp8_rows_kernel<4, kAdd>);
            else
                err = launch_rows(rmsnorm_fp8_rows_kernel<8, false>);
            if (err != cudaSuccess) return BI_ERR_CUDA;
            return cudaGetLastError() == cudaSuccess ? BI_OK : BI_ERR_CUDA;
        }
        if (rows <= 512 && vpt > 1) {
            err = vpt == 2   ? launch(rmsnorm_kernel<2, kAdd, true, true>)
                  : vpt <= 4 ? launch(rmsnorm_kernel<4, kAdd, true, true>)
                  : vpt <= 8 ? launch(rmsnorm_kernel<8, kAdd, true, true>)
                             : launch(rmsnorm_kernel<16, kAdd, true, true>);
            if (err != cudaSuccess) return BI_ERR_CUDA;
            return cudaGetLastError() == cudaSuccess ? BI_OK : BI_ERR_CUDA;
        }
    }
    if (vpt == 1)
        err = launch(rmsnorm_kernel<1, kAdd, kFp8>);
    else if (vpt == 2)
        err = launch(rmsnorm_kernel<2, kAdd, kFp8>);
    else if (vpt <= 4)
        err = launch(rmsnorm_kernel<4, kAdd, kFp8>);
    else if (vpt <= 8)
        err = launch(rmsnorm_kernel<8, kAdd, kFp8>);
    else
        err = launch(rmsnorm_kernel<16, kAdd, kFp8>);
    if (err != cudaSuccess) return BI_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? BI_OK : BI_ERR_CUDA;
}

}  // namespace

extern "C" bi_status bi_rmsnorm(const void* x, const void* w, void* y, int64_t rows,
                                int32_t hidden, int64_t ld_x, int64_t ld_y, float eps,
                                cudaStream_t stream) {
    return launch_rmsnorm<false, false>(x, w, y, rows, hidden, ld_x, ld_y, eps, nullptr, hidden, {},
                                        stream);
}

extern "C" bi_status bi_add_rmsnorm(const void* x, void* residual, const void* w, void* y,
                                    int64_t rows, int32_t hidden, int64_t ld_x, int64_t ld_res,
                                    int64_t ld_y, float eps, cudaStream_t stream) {
    return launch_rmsnorm<true, false>(x, w, y, rows, hidden, ld_x, ld_y, eps, residual, ld_res, {},
                                       stream);
}

extern "C" bi_status bi_rmsnorm_fp8(const void* x, const void* w, void* q, void* scales,
                                    int64_t rows, int32_t hidden, int64_t ld_x, int64_t ld_q,
                                    float eps, cudaStream_t stream) {
    const Fp8Out fp8{static_cast<uint8_t*>(scales), bi_fp8::spans_of(hidden), nullptr, 0};
    return launch_rmsnorm<false, true>(x, w, q, rows, hidden, ld_x, ld_q, eps, nullptr, hidden, fp8,
                                       stream);
}

extern "C" bi_status bi_add_rmsnorm_fp8(const void* x, const void* residual, void* residual_out,
                                        const void* w, void* q, void* scales, int64_t rows,
                                        int32_t hidden, int64_t ld_x, int64_t ld_res,
                                        int64_t ld_res_out, int64_t ld_q, float eps,
                                        cudaStream_t stream) {
    const Fp8Out fp8{static_cast<uint8_t*>(scales), bi_fp8::spans_of(hidden),
                     static_cast<__nv_bfloat16*>(residual_out), ld_res_out};
    return launch_rmsnorm<true, true>(x, w, q, rows, hidden, ld_x, ld_q, eps,
                                      const_cast<void*>(residual), ld_res, fp8, stream);
}
