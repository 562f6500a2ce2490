// bi_kv4_append and bi_kv4_read: writing rows of K and V into a 4-bit paged
// cache, and reading the pages of sequences back into a bf16 one (kv4.cuh has
// the format and its arithmetic).
//
// Both are per row: "Defeating Nondeterminism in LLM Inference: The Core Role
// of Batch Invariance", section "3. Batch-Invariant Attention", asks that a
// token's K/V be the same whichever step and batch it was written in, and here
// a row's codes depend on its own 128 values only.
#include <cuda_bf16.h>

#include <algorithm>

#include "bi_internal.h"
#include "bi_ptx.cuh"
#include "kv4.cuh"

namespace {

constexpr int kD = 128;
constexpr int kThreads = 256;
constexpr int kHalfWarps = kThreads / 16;

struct AppendArgs {
    const __nv_bfloat16* k;
    const __nv_bfloat16* v;
    int64_t ld_k, ld_v;
    uint32_t rows;  // T * Hkv
    uint32_t Hkv;
    const int32_t* slots;
    uint8_t* k_cache;
    uint8_t* v_cache;
    int32_t num_slots;
    uint32_t* err;
};

__device__ __forceinline__ bi_kv4::RowPart load_row(const __nv_bfloat16* p, int l) {
    return {*reinterpret_cast<const uint2*>(p + 4 * l), *reinterpret_cast<const uint2*>(p + kD / 2 + 4 * l)};
}

// A half-warp takes kRows (token, kv-head) pairs, the K row and the V row of
// each, all loads before any arithmetic.  8192 tokens of 8 heads (33.6 MB read,
// 9.4 MB written) take 11.9 us cold, 3.6 TB/s: about 140 instructions for a
// warp's two rows are what bounds it (1 pair 12.4 us, 4 pairs 12.3).
constexpr int kRows = 2;

__global__ void __launch_bounds__(kThreads) kv4_append_kernel(const AppendArgs a) {
    bi::launch_dependents();
    bi::grid_dependency_wait();  // nothing global is touched before the previous kernel ends
    const int l = threadIdx.x & 15;
    bi_kv4::RowPart xk[kRows], xv[kRows];
    int32_t slot[kRows];
    uint32_t head[kRows];
    bool live[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const uint32_t row = (blockIdx.x * kRows + i) * kHalfWarps + (threadIdx.x >> 4);
        live[i] = row < a.rows;
        const uint32_t t = live[i] ? row / a.Hkv : 0;
        head[i] = live[i] ? row - t * a.Hkv : 0;
        xk[i] = load_row(a.k + t * a.ld_k + head[i] * kD, l);
        xv[i] = load_row(a.v + t * a.ld_v + head[i] * kD, l);
        slot[i] = a.slots[t];
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        if (slot[i] < 0 || slot[i] >= a.num_slots) {
            if (live[i] && l == 0 && head[i] == 0)
                bi::report_error(a.err, bi::kErrBadInput | bi::kWhereDecoderOps);
            live[i] = false;
        }
        const int off = slot[i] & (BI_PAGE_SIZE - 1);
        const int64_t block = live[i] ? static_cast<int64_t>(slot[i] / BI_PAGE_SIZE) * a.Hkv + head[i] : 0;
        bi_kv4::write_row<false>(xk[i], a.k_cache + block * bi_kv4::kBlockBytes, off, l, live[i]);
        bi_kv4::write_row<true>(xv[i], a.v_cache + block * bi_kv4::kBlockBytes, off, l, live[i]);
    }
}

struct ReadArgs {
    const uint8_t* k_cache;
    const uint8_t* v_cache;
    const int32_t* block_table;
    int max_pages_per_seq;
    const int32_t* seq_lens;
    int Hkv, num_pages, max_seq_len;
    __nv_bfloat16* k_out;
    __nv_bfloat16* v_out;
    uint32_t* err;
};

// One CTA per (sequence, page, kHeads kv-heads), pages gridDim.x apart: thread
// (r, c) writes dims 8c .. 8c + 7 of token r of every head, all loads before any
// store.  Bound by HBM and the latency of a CTA's three dependent loads (length,
// page, codes): 8192 tokens of 8 heads (9.4 MB read, 33.6 MB written) take 10.5
// us cold, 4.1 TB/s (16.3 us with a loop over the heads, 10.7 with one head or
// four a CTA).
constexpr int kHeads = 2;
// CTAs of a launch: a bound far above the lengths would ask for very many that
// find no page.  29 sequences of 32 .. 512 tokens under a bound of 131072 take
// 7.8 us (958 with a CTA a page, 18 with 16384 CTAs), one of 131072 tokens 134
// (138, 133).
constexpr int64_t kMostCtas = 4096;

__global__ void __launch_bounds__(kThreads) kv4_read_kernel(const ReadArgs a) {
    bi::launch_dependents();
    bi::grid_dependency_wait();  // nothing global is touched before the previous kernel ends
    const int s = blockIdx.y;
    const int h0 = blockIdx.z * kHeads;
    const int L = a.seq_lens[s];
    if (L < 0 || L > a.max_seq_len) {
        if (threadIdx.x == 0 && blockIdx.x == 0 && h0 == 0)
            bi::report_error(a.err, bi::kErrBadInput | bi::kWhereDecoderOps);
        return;
    }
    const int r = threadIdx.x >> 4, c = threadIdx.x & 15;
    const int pages = L / BI_PAGE_SIZE + (L % BI_PAGE_SIZE != 0);
    for (int p = blockIdx.x; p < pages; p += gridDim.x) {
        const int pg = a.block_table[static_cast<int64_t>(s) * a.max_pages_per_seq + p];
        if (pg < 0 || pg >= a.num_pages) {
            if (threadIdx.x == 0 && h0 == 0) bi::report_error(a.err, bi::kErrBadInput | bi::kWhereDecoderOps);
            continue;
        }
        if (r >= L - p * BI_PAGE_SIZE) continue;  // rows behind the sequence stay as they were
        const int k_at = 64 * r + 4 * (c >> 2);                                  // word (t = 0, j = c / 4)
        const int v_at = 512 * (r >> 3) + 8 * (r & 7) + 4 * (c >> 3);            // word (g = 0, w = c / 8)
        const int s_at = bi_kv4::kScaleOffset + bi_kv4::kScaleRowBytes * r + 2 * (c >> 2);
        const int64_t blk0 = static_cast<int64_t>(pg) * a.Hkv + h0;
        uint32_t kw[kHeads][4], vw[kHeads][8], ks[kHeads], vs[kHeads];
#pragma unroll
        for (int i = 0; i < kHeads; ++i) {
            if (h0 + i >= a.Hkv) break;
            const uint8_t* kb = a.k_cache + (blk0 + i) * bi_kv4::kBlockBytes;
            const uint8_t* vb = a.v_cache + (blk0 + i) * bi_kv4::kBlockBytes;
#pragma unroll
            for (int t = 0; t < 4; ++t) kw[i][t] = *reinterpret_cast<const uint32_t*>(kb + k_at + 16 * t);
#pragma unroll
            for (int g = 0; g < 8; ++g) vw[i][g] = *reinterpret_cast<const uint32_t*>(vb + v_at + 64 * g);
            ks[i] = *reinterpret_cast<const uint16_t*>(kb + s_at);
            vs[i] = *reinterpret_cast<const uint16_t*>(vb + s_at);
        }
#pragma unroll
        for (int i = 0; i < kHeads; ++i) {
            if (h0 + i >= a.Hkv) break;
            const int64_t out = ((blk0 + i) * BI_PAGE_SIZE + r) * kD + 8 * c;
            uint32_t ko[4], vo[4];
            const bi_kv4::ScalePair kp = bi_kv4::scale_pair(ks[i] * 0x10001u);
            const bi_kv4::ScalePair vp = bi_kv4::scale_pair(vs[i] * 0x10001u);
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                ko[t] = bi_kv4::kv4_pair(kw[i][t], c & 3, kp);
                // dims 8c + 2t, 8c + 2t + 1: code c % 8 of words g = 2t, 2t + 1
                const uint32_t lo = vw[i][2 * t] >> (4 * (c & 7)), hi = vw[i][2 * t + 1] >> (4 * (c & 7));
                vo[t] = bi_kv4::kv4_pair(__byte_perm(lo, hi, 0x5410), 0, vp);
            }
            *reinterpret_cast<uint4*>(a.k_out + out) = make_uint4(ko[0], ko[1], ko[2], ko[3]);
            *reinterpret_cast<uint4*>(a.v_out + out) = make_uint4(vo[0], vo[1], vo[2], vo[3]);
        }
    }
}

bool misaligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; }

}  // namespace

extern "C" bi_status bi_kv4_append(const void* k, int64_t ld_k, const void* v, int64_t ld_v,
                                   int32_t T, int32_t Hkv, int32_t D, const int32_t* slots,
                                   void* k_cache, void* v_cache, int32_t num_pages,
                                   int32_t page_size, cudaStream_t stream) {
    if (T < 0 || Hkv <= 0 || num_pages < 1) return BI_ERR_INVALID_ARG;
    if (D != kD || page_size != BI_PAGE_SIZE) return BI_ERR_UNSUPPORTED_SHAPE;
    if (static_cast<int64_t>(num_pages) * Hkv * BI_PAGE_SIZE >= (int64_t{1} << 31))
        return BI_ERR_UNSUPPORTED_SHAPE;
    const int64_t width = static_cast<int64_t>(Hkv) * kD;
    if (ld_k < width || ld_v < width) return BI_ERR_INVALID_ARG;
    if ((ld_k & 7) || (ld_v & 7)) return BI_ERR_MISALIGNED;
    const int64_t rows = static_cast<int64_t>(T) * Hkv;
    const int64_t ctas = (rows + kRows * kHalfWarps - 1) / (kRows * kHalfWarps);
    if (rows > 0x7fffff00LL) return BI_ERR_UNSUPPORTED_SHAPE;
    if (T == 0) return BI_OK;
    if (!k || !v || !slots || !k_cache || !v_cache) return BI_ERR_INVALID_ARG;
    if (!bi::aligned16(k) || !bi::aligned16(v) || !bi::aligned16(k_cache) ||
        !bi::aligned16(v_cache) || misaligned4(slots))
        return BI_ERR_MISALIGNED;
    AppendArgs a;
    a.k = static_cast<const __nv_bfloat16*>(k);
    a.v = static_cast<const __nv_bfloat16*>(v);
    a.ld_k = ld_k;
    a.ld_v = ld_v;
    a.rows = static_cast<uint32_t>(rows);
    a.Hkv = static_cast<uint32_t>(Hkv);
    a.slots = slots;
    a.k_cache = static_cast<uint8_t*>(k_cache);
    a.v_cache = static_cast<uint8_t*>(v_cache);
    a.num_slots = num_pages * BI_PAGE_SIZE;
    a.err = bi::device_error_word();
    return bi::launch_pdl(kv4_append_kernel, dim3(static_cast<unsigned>(ctas)), dim3(kThreads), 0,
                          stream, a) == cudaSuccess
               ? BI_OK
               : BI_ERR_CUDA;
}

extern "C" bi_status bi_kv4_read(const void* k_cache, const void* v_cache,
                                 const int32_t* block_table, int32_t max_pages_per_seq,
                                 const int32_t* seq_lens, int32_t S, int32_t Hkv, int32_t D,
                                 int32_t page_size, int32_t num_pages, int32_t max_seq_len,
                                 void* k_out, void* v_out, cudaStream_t stream) {
    if (S < 0 || Hkv <= 0 || max_pages_per_seq < 1 || num_pages < 1 || max_seq_len < 1)
        return BI_ERR_INVALID_ARG;
    if (D != kD || page_size != BI_PAGE_SIZE) return BI_ERR_UNSUPPORTED_SHAPE;
    if (S > 65535 || Hkv > 65535) return BI_ERR_UNSUPPORTED_SHAPE;
    if (static_cast<int64_t>(num_pages) * Hkv * BI_PAGE_SIZE >= (int64_t{1} << 31))
        return BI_ERR_UNSUPPORTED_SHAPE;
    if (static_cast<int64_t>(max_seq_len) > static_cast<int64_t>(max_pages_per_seq) * BI_PAGE_SIZE)
        return BI_ERR_INVALID_ARG;
    if (S == 0) return BI_OK;
    if (!k_cache || !v_cache || !block_table || !seq_lens || !k_out || !v_out)
        return BI_ERR_INVALID_ARG;
    if (!bi::aligned16(k_cache) || !bi::aligned16(v_cache) || !bi::aligned16(k_out) ||
        !bi::aligned16(v_out) || misaligned4(block_table) || misaligned4(seq_lens))
        return BI_ERR_MISALIGNED;
    ReadArgs a;
    a.k_cache = static_cast<const uint8_t*>(k_cache);
    a.v_cache = static_cast<const uint8_t*>(v_cache);
    a.block_table = block_table;
    a.max_pages_per_seq = max_pages_per_seq;
    a.seq_lens = seq_lens;
    a.Hkv = Hkv;
    a.num_pages = num_pages;
    a.max_seq_len = max_seq_len;
    a.k_out = static_cast<__nv_bfloat16*>(k_out);
    a.v_out = static_cast<__nv_bfloat16*>(v_out);
    a.err = bi::device_error_word();
    const int64_t pages = (static_cast<int64_t>(max_seq_len) + BI_PAGE_SIZE - 1) / BI_PAGE_SIZE;
    const int64_t heads = (Hkv + kHeads - 1) / kHeads;
    const dim3 grid(static_cast<unsigned>(std::min(pages, std::max<int64_t>(1, kMostCtas / (S * heads)))),
                    static_cast<unsigned>(S), static_cast<unsigned>(heads));
    return bi::launch_pdl(kv4_read_kernel, grid, dim3(kThreads), 0, stream, a) == cudaSuccess
               ? BI_OK
               : BI_ERR_CUDA;
}
