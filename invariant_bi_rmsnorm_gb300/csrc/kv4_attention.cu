// bi_decode_attention_kv4: bi_decode_attention over a paged cache held in 4
// bits (kv4.cuh has the format).
//
// "Defeating Nondeterminism in LLM Inference: The Core Role of Batch
// Invariance", section "3. Batch-Invariant Attention" ("Fixed Size Split KV
// Strategy"): the same 256-token chunks, pages, per-page steps and folds as
// the kernel over a bf16 cache (attn_common.cuh, attn_fold.cuh).  A code's
// value n * s is a bf16 number, so a page's operands are exactly those that a
// read-back bf16 cache would give, and so are the result's bits.
//
// One CTA (4 warps) per (sequence, kv-head, chunk).  The bytes of a chunk are
// a quarter of a bf16 chunk's but its arithmetic is the same and the codes
// have to be turned into numbers besides, so what bounds the kernel is the
// instructions it issues; the work of a chunk is dealt out so that none is
// done twice and every warp has a few pages' independent work at hand:
//   0  warp 0 copies the chunk's up to 16 pages into shared memory, two bulk
//      copies (K, V) a lane;
//   1  scores: warp w takes pages w, w + 4, ..., and their maxima;
//   2  the pages' reference maxima, one after the other (8 columns, one lane
//      each; a few instructions a page);
//   3  weights: warp w, its own pages; the split weights go to shared memory in
//      the order of mma.sync's B operand, over the K blocks, which are done with;
//   4  output: warp w takes dims 32w .. 32w + 31 (one group) over all pages.
// A lane takes its fragments of K and V from a block with 16-byte loads, in
// the order of mma.sync's A operand (ldmatrix has no 4-bit form), and turns
// them into bf16 pairs in registers: a shift, an and-or and one fma for two
// values.
#include <cuda_bf16.h>

#include <atomic>
#include <cmath>

#include "attn_common.cuh"
#include "attn_fold.cuh"
#include "bi_internal.h"
#include "bi_ptx.cuh"
#include "kv4.cuh"

namespace {

using bi_attn::ceil_div;
using bi_attn::kChunk;
using bi_attn::kD;
using bi_attn::kFoldFloats;
using bi_attn::kMaxCounters;
using bi_attn::kMaxGroup;
using bi_attn::kPage;
using bi_attn::kPagesPerChunk;
using bi_attn::kThreads;
using bi_attn::kWarps;
using bi_attn::SplitArgs;
using bi_kv4::kBlockBytes;
using bi_kv4::kScaleOffset;
using bi_kv4::kScaleRowBytes;
using bi_kv4::ScalePair;

constexpr int kPagesPerWarp = kPagesPerChunk / kWarps;
constexpr int kMatBytes = kPagesPerChunk * kBlockBytes;  // the chunk's K (or V) blocks
constexpr int kStagingBytes = 2 * kMatBytes;
constexpr int kSmemBytes = kStagingBytes + kFoldFloats * 4;
static_assert(kPagesPerChunk * 32 * 16 <= kMatBytes, "the weights fit over the K blocks");

// Tables of the chunk in the shared memory that the fold uses afterwards.
struct Tables {
    float pmax[kPagesPerChunk][kMaxGroup];   // a page's largest score (log2 units)
    float ref[kPagesPerChunk][kMaxGroup];    // what the page's scores are taken relative to
    float alpha[kPagesPerChunk][kMaxGroup];  // the factor O and l are rescaled by before it
    float psum[kPagesPerChunk][kMaxGroup];   // the page's weight sum
    float m[kMaxGroup], l[kMaxGroup];        // the chunk's reference and weight sum
    uint32_t moved;                          // pages with an alpha other than 1
};
static_assert(sizeof(Tables) <= kFoldFloats * 4, "the tables fit where the fold works");

struct Kv4Args {
    SplitArgs s;
    const uint8_t* k_cache;
    const uint8_t* v_cache;
};

// `bytes` (a multiple of 16) global -> shared by the bulk-copy engine; both
// addresses 16-byte aligned; completion counted on `bar`.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
            bi::smem_u32(dst)),
        "l"(src), "r"(bytes), "r"(bi::smem_u32(bar))
        : "memory");
}

__device__ __forceinline__ uint32_t lo_halves(uint32_t a, uint32_t b) { return __byte_perm(a, b, 0x5410); }
__device__ __forceinline__ uint32_t hi_halves(uint32_t a, uint32_t b) { return __byte_perm(a, b, 0x7632); }

// bi_attn::page_scores over a 4-bit K block.
__device__ __forceinline__ void page_scores_kv4(float (&sc)[4], const uint8_t* kb,
                                                const uint32_t (&qb0)[8], const uint32_t (&qb1)[8],
                                                int lane) {
    const uint4 ca = *reinterpret_cast<const uint4*>(kb + 16 * lane);        // token l / 4
    const uint4 cb = *reinterpret_cast<const uint4*>(kb + 512 + 16 * lane);  // token l / 4 + 8
    const uint8_t* sp = kb + kScaleOffset + kScaleRowBytes * (lane >> 2);
    const uint2 sa = *reinterpret_cast<const uint2*>(sp);
    const uint2 sb = *reinterpret_cast<const uint2*>(sp + 8 * kScaleRowBytes);
    const uint32_t wa[4] = {ca.x, ca.y, ca.z, ca.w}, wb[4] = {cb.x, cb.y, cb.z, cb.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) sc[i] = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {  // the group of dims 32j .. 32j + 31: two 16-deep steps
        const uint32_t da = j < 2 ? sa.x : sa.y, db = j < 2 ? sb.x : sb.y;
        const ScalePair pa = bi_kv4::scale_pair(j & 1 ? hi_halves(da, da) : lo_halves(da, da));
        const ScalePair pb = bi_kv4::scale_pair(j & 1 ? hi_halves(db, db) : lo_halves(db, db));
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int ks = 2 * j + e;
            bi::mma_bf16_16816(sc, bi_kv4::kv4_pair(wa[j], 2 * e, pa), bi_kv4::kv4_pair(wb[j], 2 * e, pb),
                               bi_kv4::kv4_pair(wa[j], 2 * e + 1, pa),
                               bi_kv4::kv4_pair(wb[j], 2 * e + 1, pb), qb0[ks], qb1[ks]);
        }
    }
}

// The values of the 32 dims of group `gr` of a V block, as the A operands of
// their two 16-dim tiles: a[i][0..3].  Tokens from `valid` on stand for zeros,
// whatever the block holds there.
__device__ __forceinline__ void v_operands(uint32_t (&a)[2][4], const uint8_t* vb, int gr, int valid,
                                           int lane) {
    // this lane's tokens 2(l%4), 2(l%4) + 1 and the two 8 further on
    const uint4 ca = *reinterpret_cast<const uint4*>(vb + 16 * lane);
    const uint4 cb = *reinterpret_cast<const uint4*>(vb + 512 + 16 * lane);
    const uint8_t* sp = vb + kScaleOffset + 2 * kScaleRowBytes * (lane & 3) + 4 * (gr >> 1);
    uint32_t s0 = *reinterpret_cast<const uint32_t*>(sp);
    uint32_t s1 = *reinterpret_cast<const uint32_t*>(sp + kScaleRowBytes);
    uint32_t s8 = *reinterpret_cast<const uint32_t*>(sp + 8 * kScaleRowBytes);
    uint32_t s9 = *reinterpret_cast<const uint32_t*>(sp + 9 * kScaleRowBytes);
    if (valid < kPage) {
        const int t = 2 * (lane & 3);
        if (t >= valid) s0 = 0u;
        if (t + 1 >= valid) s1 = 0u;
        if (t + 8 >= valid) s8 = 0u;
        if (t + 9 >= valid) s9 = 0u;
    }
    // codes of (even token, odd token) side by side; their scales likewise
    const uint32_t e0 = gr & 2 ? ca.y : ca.x, o0 = gr & 2 ? ca.w : ca.z;
    const uint32_t e1 = gr & 2 ? cb.y : cb.x, o1 = gr & 2 ? cb.w : cb.z;
    const uint32_t sel = gr & 1 ? 0x7632u : 0x5410u;
    const uint32_t wa = __byte_perm(e0, o0, sel), wb = __byte_perm(e1, o1, sel);
    const ScalePair pa = bi_kv4::scale_pair(__byte_perm(s0, s1, sel));
    const ScalePair pb = bi_kv4::scale_pair(__byte_perm(s8, s9, sel));
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        a[i][0] = bi_kv4::kv4_pair(wa, 2 * i, pa);
        a[i][1] = bi_kv4::kv4_pair(wa, 2 * i + 1, pa);
        a[i][2] = bi_kv4::kv4_pair(wb, 2 * i, pb);
        a[i][3] = bi_kv4::kv4_pair(wb, 2 * i + 1, pb);
    }
}

// One butterfly for the two columns of every lane over the 8 lanes that share
// them (4, 8, 16 apart): its first step deals the columns out, lane l goes on
// with column 2(l%4) + (l/4)%2 alone.
template <typename F>
__device__ __forceinline__ float reduce_columns(float v0, float v1, int lane, F f) {
    const bool odd = lane & 4;
    float v = odd ? v1 : v0;
    v = f(v, __shfl_xor_sync(0xffffffffu, odd ? v0 : v1, 4));
    v = f(v, __shfl_xor_sync(0xffffffffu, v, 8));
    return f(v, __shfl_xor_sync(0xffffffffu, v, 16));
}

__global__ void __launch_bounds__(kThreads, 5) attn_chunk_kv4_kernel(const Kv4Args ka) {
    bi::launch_dependents();
    bi::grid_dependency_wait();  // nothing global is touched before the previous kernel ends
    const SplitArgs& a = ka.s;
    const int c = blockIdx.x;  // chunk
    const int g = blockIdx.y;
    const int s = blockIdx.z;
    const int tid = threadIdx.x;
    const int warp = tid >> 5;
    const int lane = tid & 31;

    const int L = a.seq_lens[s];
    if (L < 1 || L > a.max_seq_len) {
        if (tid == 0 && c == 0 && g == 0) bi::report_error(a.err, bi::kErrBadInput | bi::kWhereAttnSplit);
        return;
    }
    const int nch = (L + kChunk - 1) / kChunk;
    if (c >= nch) return;
    const int tokens = min(kChunk, L - c * kChunk);
    const int np = (tokens + kPage - 1) / kPage;
    // several CTAs share a longer sequence and the last one to arrive folds it
    uint32_t* const ctr = nch > 1 ? a.counters + static_cast<int64_t>(s) * a.Hkv + g : nullptr;

    extern __shared__ __align__(16) uint8_t smem[];
    uint8_t* const ks = smem;
    uint8_t* const vs = smem + kMatBytes;
    uint4* const weights = reinterpret_cast<uint4*>(ks);  // [page][lane], from phase 3 on
    float* const small = reinterpret_cast<float*>(smem + kStagingBytes);
    Tables& tb = *reinterpret_cast<Tables*>(small);
    __shared__ uint64_t bars[2];  // K landed, V landed
    __shared__ int bad_page;

    // ---- 0: copies ----
    if (warp == 0) {
        int pg = 0;
        if (lane < np)
            pg = a.block_table[static_cast<int64_t>(s) * a.max_pages_per_seq + c * kPagesPerChunk + lane];
        const bool bad = __any_sync(0xffffffffu, pg < 0 || pg >= a.num_pages);
        if (lane == 0) {
            bad_page = bad;
            bi::mbar_init(&bars[0], 1);
            bi::mbar_init(&bars[1], 1);
            bi::fence_mbar_init();
            if (!bad) {
                bi::mbar_arrive_expect_tx(&bars[0], np * kBlockBytes);
                bi::mbar_arrive_expect_tx(&bars[1], np * kBlockBytes);
            }
        }
        __syncwarp();
        if (!bad && lane < np) {
            const int64_t at = (static_cast<int64_t>(pg) * a.Hkv + g) * kBlockBytes;
            bulk_load(ks + lane * kBlockBytes, ka.k_cache + at, kBlockBytes, &bars[0]);
            bulk_load(vs + lane * kBlockBytes, ka.v_cache + at, kBlockBytes, &bars[1]);
        }
    }
    // column n of the mma tile = query head g*group + n (n < group)
    uint32_t qb0[8], qb1[8];
    {
        const int n = lane >> 2;
        bi_attn::load_q_frags(
            n < a.group ? a.q + (static_cast<int64_t>(s) * a.Hq + g * a.group + n) * kD : nullptr,
            lane, qb0, qb1);
    }
    __syncthreads();  // barriers and bad_page are set
    if (bad_page) {
        if (tid == 0) {
            bi::report_error(a.err, bi::kErrBadInput | bi::kWhereAttnSplit);
            if (nch > 1) bi_attn::arrive_bad(ctr, nch);
        }
        return;
    }

    // ---- 1: scores of this warp's pages, in log2 units, and their maxima ----
    const bool k_here = bi::mbar_wait(&bars[0], 0);
    float x[kPagesPerWarp][4];
    if (k_here) {
#pragma unroll
        for (int i = 0; i < kPagesPerWarp; ++i) {
            const int p = warp + kWarps * i;
            if (p >= np) break;
            page_scores_kv4(x[i], ks + p * kBlockBytes, qb0, qb1, lane);
#pragma unroll
            for (int e = 0; e < 4; ++e) x[i][e] = __fmul_rn(x[i][e], a.scale_log2);
            const int valid = tokens - p * kPage;
            if (valid < kPage) {
                if ((lane >> 2) >= valid) x[i][0] = x[i][1] = -INFINITY;
                if ((lane >> 2) + 8 >= valid) x[i][2] = x[i][3] = -INFINITY;
            }
            const float mx = reduce_columns(fmaxf(x[i][0], x[i][2]), fmaxf(x[i][1], x[i][3]), lane,
                                            [](float u, float v) { return fmaxf(u, v); });
            if (lane < 8) tb.pmax[p][2 * (lane & 3) + (lane >> 2)] = mx;
        }
    }
    const bool v_here = bi::mbar_wait(&bars[1], 0);
    if (__syncthreads_or(!k_here || !v_here)) {
        if (tid == 0) {
            bi::report_error(a.err, bi::kErrTimeout | bi::kWhereAttnSplit);
            // the copies still write to this CTA's shared memory: one more bounded wait each
            bi::mbar_wait_for(&bars[0], 0, bi::kDrainNs);
            bi::mbar_wait_for(&bars[1], 0, bi::kDrainNs);
            if (nch > 1) bi_attn::arrive_bad(ctr, nch);
        }
        return;
    }

    // ---- 2: the online softmax's reference maxima (bi_attn::softmax_step) ----
    if (warp == 0) {
        const int n = lane & 7;
        float m = -INFINITY;
        uint32_t moved = 0;
        for (int p = 0; p < np; ++p) {
            const float mx = tb.pmax[p][n];
            const float mn = mx > __fadd_rn(m, bi_attn::kRescaleSlack) ? mx : m;
            const float al = mn == m ? 1.f : bi_attn::exp2_ftz(__fsub_rn(m, mn));
            if (__any_sync(0xffffffffu, mn != m)) moved |= 1u << p;
            m = mn;
            if (lane < 8) {
                // no visible score so far: every score is -inf, and so is its
                // difference from 0
                tb.ref[p][n] = m == -INFINITY ? 0.f : m;
                tb.alpha[p][n] = al;
            }
        }
        if (lane < 8) tb.m[n] = m;
        if (lane == 0) tb.moved = moved & ~1u;  // before page 0 there is nothing to rescale
    }
    __syncthreads();

    // ---- 3: weights p = 2^(x - m) of this warp's pages, split into bf16 high
    // part and remainder, transposed into mma B fragments ----
#pragma unroll
    for (int i = 0; i < kPagesPerWarp; ++i) {
        const int p = warp + kWarps * i;
        if (p >= np) break;
        const float2 m = *reinterpret_cast<const float2*>(&tb.ref[p][2 * (lane & 3)]);
        const float p0 = bi_attn::exp2_ftz(__fsub_rn(x[i][0], m.x));
        const float p1 = bi_attn::exp2_ftz(__fsub_rn(x[i][1], m.y));
        const float p2 = bi_attn::exp2_ftz(__fsub_rn(x[i][2], m.x));
        const float p3 = bi_attn::exp2_ftz(__fsub_rn(x[i][3], m.y));
        const uint32_t pA = bi::pack_bf16x2(p0, p1);
        const uint32_t pB = bi::pack_bf16x2(p2, p3);
        const uint32_t rA = bi::pack_bf16x2(__fsub_rn(p0, __uint_as_float(pA << 16)),
                                            __fsub_rn(p1, __uint_as_float(pA & 0xffff0000u)));
        const uint32_t rB = bi::pack_bf16x2(__fsub_rn(p2, __uint_as_float(pB << 16)),
                                            __fsub_rn(p3, __uint_as_float(pB & 0xffff0000u)));
        weights[p * 32 + lane] = make_uint4(bi::movmatrix_trans(pA), bi::movmatrix_trans(pB),
                                            bi::movmatrix_trans(rA), bi::movmatrix_trans(rB));
        const float ps = reduce_columns(__fadd_rn(p0, p2), __fadd_rn(p1, p3), lane,
                                        [](float u, float v) { return __fadd_rn(u, v); });
        if (lane < 8) tb.psum[p][2 * (lane & 3) + (lane >> 2)] = ps;
    }
    __syncthreads();

    // ---- 4: O^T of this warp's 32 dims, page after page; l beside it ----
    const uint32_t moved = tb.moved;
    if (warp == kWarps - 1 && lane < 8) {
        float l = 0.f;
        for (int p = 0; p < np; ++p) l = __fmaf_rn(l, tb.alpha[p][lane], tb.psum[p][lane]);
        tb.l[lane] = l;
    }
    float acc[2][4];
#pragma unroll
    for (int i = 0; i < 2; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
#pragma unroll 2
    for (int p = 0; p < np; ++p) {
        uint32_t va[2][4];
        v_operands(va, vs + p * kBlockBytes, warp, tokens - p * kPage, lane);
        const uint4 w = weights[p * 32 + lane];
        if (moved >> p & 1u) {
            const float2 al = *reinterpret_cast<const float2*>(&tb.alpha[p][2 * (lane & 3)]);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                acc[i][0] = __fmul_rn(acc[i][0], al.x);
                acc[i][1] = __fmul_rn(acc[i][1], al.y);
                acc[i][2] = __fmul_rn(acc[i][2], al.x);
                acc[i][3] = __fmul_rn(acc[i][3], al.y);
            }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            bi::mma_bf16_16816(acc[i], va[i][0], va[i][1], va[i][2], va[i][3], w.x, w.y);
            bi::mma_bf16_16816(acc[i], va[i][0], va[i][1], va[i][2], va[i][3], w.z, w.w);
        }
    }
    __syncthreads();  // l is there

    const int h0 = 2 * (lane & 3);
    const int d0 = 32 * warp + (lane >> 2);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int h = h0 + e;
        if (h >= a.group) continue;
        const int64_t row = static_cast<int64_t>(s) * a.Hq + g * a.group + h;
        if (nch == 1) {  // the whole sequence: bf16(O / l)
            const float il = bi_attn::inv_weight(tb.l[h]);
            __nv_bfloat16* o = a.out + row * kD + d0;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                o[16 * i] = __float2bfloat16_rn(bi_attn::normalise(acc[i][e], il));
                o[16 * i + 8] = __float2bfloat16_rn(bi_attn::normalise(acc[i][2 + e], il));
            }
        } else {  // the chunk's partial
            float* o = a.ws_acc + (row * a.max_chunks + c) * kD + d0;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                o[16 * i] = acc[i][e];
                o[16 * i + 8] = acc[i][2 + e];
            }
            if (warp == 0 && lane < 4)
                *reinterpret_cast<float2*>(a.ws_ml + (row * a.max_chunks + c) * 2) =
                    make_float2(tb.m[h], tb.l[h]);
        }
    }
    if (nch == 1) return;
    // the last CTA of this (sequence, kv-head) to arrive folds it
    bi_attn::arrive_and_fold<kStagingBytes>(a, ctr, nch, s, g, nch, smem, small, tid);
}

// set once per device; any thread may race to set it, the attribute is idempotent
std::atomic<bool> g_attr_set[64] = {};

}  // namespace

extern "C" bi_status bi_decode_attention_kv4(const void* q, const void* k_cache,
                                             const void* v_cache, const int32_t* block_table,
                                             int32_t max_pages_per_seq, const int32_t* seq_lens,
                                             int32_t B, int32_t Hq, int32_t Hkv, int32_t D,
                                             int32_t page_size, int32_t num_pages,
                                             int32_t max_seq_len, float scale, void* out,
                                             void* workspace, size_t workspace_bytes,
                                             cudaStream_t stream) {
    if (B < 0 || Hq <= 0 || Hkv <= 0 || max_pages_per_seq < 1 || num_pages < 1 || max_seq_len < 1)
        return BI_ERR_INVALID_ARG;
    if (!(scale > 0.f) || !std::isfinite(scale)) return BI_ERR_INVALID_ARG;
    if (D != kD || page_size != kPage) return BI_ERR_UNSUPPORTED_SHAPE;
    if (Hq % Hkv != 0 || Hq / Hkv > kMaxGroup) return BI_ERR_UNSUPPORTED_SHAPE;
    if (B > 65535 || Hkv > 65535) return BI_ERR_UNSUPPORTED_SHAPE;
    if (static_cast<int64_t>(num_pages) * Hkv * kPage >= (int64_t{1} << 31))
        return BI_ERR_UNSUPPORTED_SHAPE;
    if (static_cast<int64_t>(max_seq_len) > static_cast<int64_t>(max_pages_per_seq) * kPage)
        return BI_ERR_INVALID_ARG;
    if (B == 0) return BI_OK;
    if (!q || !k_cache || !v_cache || !block_table || !seq_lens || !out) return BI_ERR_INVALID_ARG;
    if (!bi::aligned16(q) || !bi::aligned16(k_cache) || !bi::aligned16(v_cache) ||
        !bi::aligned16(out) || (reinterpret_cast<uintptr_t>(block_table) & 3) ||
        (reinterpret_cast<uintptr_t>(seq_lens) & 3))
        return BI_ERR_MISALIGNED;
    const int max_chunks = ceil_div(max_seq_len, kChunk);
    // one arrival counter per (sequence, kv-head), of 16 bits
    if (max_chunks > 1 && (static_cast<int64_t>(B) * Hkv > kMaxCounters || max_chunks > 65535))
        return BI_ERR_UNSUPPORTED_SHAPE;
    const size_t need = bi_decode_attention_workspace_size(B, Hq, D, max_seq_len);
    if (need > 0) {
        if (!workspace || workspace_bytes < need) return BI_ERR_WORKSPACE_TOO_SMALL;
        if (!bi::aligned16(workspace)) return BI_ERR_MISALIGNED;
    }

    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return BI_ERR_CUDA;
    if (!g_attr_set[dev]) {
        if (cudaFuncSetAttribute(attn_chunk_kv4_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kSmemBytes) != cudaSuccess)
            return BI_ERR_CUDA;
        g_attr_set[dev] = true;
    }

    Kv4Args ka;
    SplitArgs& args = ka.s;
    ka.k_cache = static_cast<const uint8_t*>(k_cache);
    ka.v_cache = static_cast<const uint8_t*>(v_cache);
    args.q = static_cast<const __nv_bfloat16*>(q);
    args.block_table = block_table;
    args.seq_lens = seq_lens;
    args.out = static_cast<__nv_bfloat16*>(out);
    // workspace: [counters, BI_DECODE_COUNTER_BYTES][acc partials][(m, l) partials]
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    args.counters = need ? reinterpret_cast<uint32_t*>(ws) : nullptr;
    args.ws_acc = need ? reinterpret_cast<float*>(ws + BI_DECODE_COUNTER_BYTES) : nullptr;
    args.ws_ml = need ? args.ws_acc + static_cast<size_t>(B) * Hq * max_chunks * kD : nullptr;
    args.err = bi::device_error_word();
    args.max_pages_per_seq = max_pages_per_seq;
    args.Hq = Hq;
    args.Hkv = Hkv;
    args.group = Hq / Hkv;
    args.num_pages = num_pages;
    args.max_seq_len = max_seq_len;
    args.max_chunks = max_chunks;
    args.num_splits = 0;
    args.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
    args.chunks_per_cta = 1;
    return bi::launch_pdl(attn_chunk_kv4_kernel, dim3(max_chunks, Hkv, B), dim3(kThreads), kSmemBytes,
                          stream, ka) == cudaSuccess
               ? BI_OK
               : BI_ERR_CUDA;
}
