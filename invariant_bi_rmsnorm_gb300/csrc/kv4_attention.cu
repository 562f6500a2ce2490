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
// A lane takes its fragments of K and V from a block with 16-byte loads, in
// the order of mma.sync's A operand (ldmatrix has no 4-bit form), and turns
// them into bf16 pairs in registers: a shift, an and-or and one fma for two
// values.
//
// The bytes of a chunk are little over a quarter of a bf16 chunk's but its
// arithmetic is the same, and the codes have to be turned into numbers besides:
// about 350 instructions a page and kv-head, 24 of them mma.sync.  An SM takes 145
// cycles for a page where HBM would deliver it in 98 (the warp kernel below, every
// chunk full: 32 sequences of 8192 tokens).  Its four schedulers' instructions
// would take 88 of them and the tensor pipe 49 (2.04 a mma.sync, measured alone).
// Neither is full, and nor is HBM; that the two together are within 6 % of what is
// measured suggests that they hardly overlap.  Lengths even over 1 .. 8192 cost
// more, 165 cycles at B = 64 and 152 at B = 256: half of the launch's warps find no
// chunk, and last pages are not full.  SMs also start late and run out of chunks
// before the last one does (10 and 6 % of the kernel), and the fold's launch
// follows (9 and 16 us).  On GB300, cold, GQA 32/8, lengths even over 1 .. 8192: B =
// 256 292 us (1.21 GB, 4.2 TB/s, 0.61 of the copy rate; the bf16 cache's 4.3 GB
// take 599 us), B = 64 83 us.
//
// mma.sync, not tcgen05, although the two give the same bits: a page is three
// products too small for tcgen05, each of which takes 44-59 cycles to issue (the
// three as much as the whole page takes here), and its operands would have to be
// written to shared memory as bf16 first.
//
// Few chunks: one CTA (4 warps) per (sequence, kv-head, chunk), which finishes
// a chunk soonest (one sequence of 8192 tokens 11.1 us, of 300 6.7 us).  The
// chunk's work is dealt out so that none is done twice:
//   0  warp w copies pages w, w + 4, ... into shared memory, asynchronously;
//   1  scores: warp w takes its own pages, and their maxima;
//   2  the pages' reference maxima, one after the other (8 columns, one lane
//      each; a few instructions a page);
//   3  weights: warp w, its own pages; the split weights go to shared memory in
//      the order of mma.sync's B operand, over the K blocks, which are done with;
//   4  output: warp w takes dims 32w .. 32w + 31 (one group) over all pages.
// Five CTAs share an SM (39 KB each); four were 12 % slower, seven (V copied
// over K once the scores are there) 3 % faster in the middle and 28 % slower
// for one sequence.  Many chunks: one warp per chunk, see below.
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "attn_common.cuh"
#include "attn_fold.cuh"
#include "bi_internal.h"
#include "bi_ptx.cuh"
#include "kv4.cuh"

namespace {

using bi_attn::ceil_div;
using bi_attn::kChunk;
using bi_attn::kD;
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
static_assert(kPagesPerChunk * 32 * 16 <= kMatBytes, "the weights fit over the K blocks");

// Tables of the chunk, in shared memory.
struct Tables {
    float pmax[kPagesPerChunk][kMaxGroup];   // a page's largest score (log2 units)
    float ref[kPagesPerChunk][kMaxGroup];    // what the page's scores are taken relative to
    float alpha[kPagesPerChunk][kMaxGroup];  // the factor O and l are rescaled by before it
    float psum[kPagesPerChunk][kMaxGroup];   // the page's weight sum
    float m[kMaxGroup], l[kMaxGroup];        // the chunk's reference and weight sum
    uint32_t moved;                          // pages with an alpha other than 1; kRefPerPage
};
constexpr uint32_t kAll = 0xffffffffu;
constexpr uint32_t kRefPerPage = 1u << 31;  // else ref[0] is every page's and alpha is not set
static_assert(kPagesPerChunk < 31, "a bit per page");
constexpr int kFactorBytes = kWarps * 32 * sizeof(float4);  // fold_row's, where the tables were
constexpr int kSmemBytes =
    kStagingBytes + (sizeof(Tables) > kFactorBytes ? sizeof(Tables) : kFactorBytes);
static_assert(kSmemBytes <= 48 * 1024, "no more than a launch may ask for without an attribute");

struct Kv4Args {
    SplitArgs s;
    const uint8_t* k_cache;
    const uint8_t* v_cache;
};

// The low (high) half twice, as moves: the compiler takes them into the operand
// of the bf16 arithmetic, which it does not with a byte permutation.
__device__ __forceinline__ uint32_t twice_lo(uint32_t a) {
    uint32_t d;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tmov.b32 %0, {l, l};\n\t}" : "=r"(d) : "r"(a));
    return d;
}
__device__ __forceinline__ uint32_t twice_hi(uint32_t a) {
    uint32_t d;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tmov.b32 %0, {h, h};\n\t}" : "=r"(d) : "r"(a));
    return d;
}

// The values of the codes at bits 4p .. 4p + 3 of both halves of w, p = 0 .. 3.
__device__ __forceinline__ void four_pairs(uint32_t (&v)[4], uint32_t w, const ScalePair& sp) {
#pragma unroll
    for (int p = 0; p < 4; ++p) v[p] = bi_kv4::kv4_pair(w, p, sp);
}

// bi::mma_bf16_16816 onto zeros.
__device__ __forceinline__ void mma_onto_zero(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                              uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

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
    for (int j = 0; j < 4; ++j) {  // the group of dims 32j .. 32j + 31: two 16-deep steps
        const uint32_t da = j < 2 ? sa.x : sa.y, db = j < 2 ? sb.x : sb.y;
        uint32_t va[4], vb[4];
        four_pairs(va, wa[j], bi_kv4::scale_pair(j & 1 ? twice_hi(da) : twice_lo(da)));
        four_pairs(vb, wb[j], bi_kv4::scale_pair(j & 1 ? twice_hi(db) : twice_lo(db)));
        if (j == 0) mma_onto_zero(sc, va[0], vb[0], va[1], vb[1], qb0[0], qb1[0]);
        else bi::mma_bf16_16816(sc, va[0], vb[0], va[1], vb[1], qb0[2 * j], qb1[2 * j]);
        bi::mma_bf16_16816(sc, va[2], vb[2], va[3], vb[3], qb0[2 * j + 1], qb1[2 * j + 1]);
    }
}

// A page's scores in log2 units (bi_attn::softmax_step's x); tokens from
// `valid` on are not there.
__device__ __forceinline__ void page_logs(float (&x)[4], const uint8_t* kb, const uint32_t (&qb0)[8],
                                          const uint32_t (&qb1)[8], int valid, float scale_log2,
                                          int lane) {
    page_scores_kv4(x, kb, qb0, qb1, lane);
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = __fmul_rn(x[e], scale_log2);
    if (valid < kPage) {
        if ((lane >> 2) >= valid) x[0] = x[1] = -INFINITY;
        if ((lane >> 2) + 8 >= valid) x[2] = x[3] = -INFINITY;
    }
}

// A page's weights p (tokens l/4, l/4 + 8; two columns each), split into bf16
// high part and remainder and transposed into mma B fragments.
__device__ __forceinline__ void split_weights(const float (&p)[4], bi_attn::PFrags& pf) {
    const uint32_t pA = bi::pack_bf16x2(p[0], p[1]);
    const uint32_t pB = bi::pack_bf16x2(p[2], p[3]);
    const uint32_t rA = bi::pack_bf16x2(__fsub_rn(p[0], __uint_as_float(pA << 16)),
                                        __fsub_rn(p[1], __uint_as_float(pA & 0xffff0000u)));
    const uint32_t rB = bi::pack_bf16x2(__fsub_rn(p[2], __uint_as_float(pB << 16)),
                                        __fsub_rn(p[3], __uint_as_float(pB & 0xffff0000u)));
    pf.hi0 = bi::movmatrix_trans(pA);
    pf.hi1 = bi::movmatrix_trans(pB);
    pf.lo0 = bi::movmatrix_trans(rA);
    pf.lo1 = bi::movmatrix_trans(rB);
}

// A lane's part of a V block: codes and scales of tokens 2(l%4) and the next
// (a), and of the two tokens 8 further on (b).  Tokens from `valid` on stand
// for zeros, whatever the block holds there.
struct VFrags {
    uint4 ca, cb, sa, sb;
};

__device__ __forceinline__ void load_v(VFrags& f, const uint8_t* vb, int valid, int lane) {
    f.ca = *reinterpret_cast<const uint4*>(vb + 16 * lane);
    f.cb = *reinterpret_cast<const uint4*>(vb + 512 + 16 * lane);
    const uint8_t* sp = vb + kScaleOffset + 2 * kScaleRowBytes * (lane & 3);
    f.sa = *reinterpret_cast<const uint4*>(sp);
    f.sb = *reinterpret_cast<const uint4*>(sp + 8 * kScaleRowBytes);
    if (valid < kPage) {
        const int t = 2 * (lane & 3);
        if (t >= valid) f.sa.x = f.sa.y = 0u;
        if (t + 1 >= valid) f.sa.z = f.sa.w = 0u;
        if (t + 8 >= valid) f.sb.x = f.sb.y = 0u;
        if (t + 9 >= valid) f.sb.z = f.sb.w = 0u;
    }
}

// bi_attn::pv_step for a group of 32 dims, two 16-dim tiles of O^T.  wa, wb:
// codes of the even and the odd token side by side (tokens 2(l%4) and the next;
// 8 further on); sa, sb: their scales likewise.
__device__ __forceinline__ void pv_tiles(float (&acc0)[4], float (&acc1)[4], uint32_t wa, uint32_t wb,
                                         uint32_t sa, uint32_t sb, const bi_attn::PFrags& pf) {
    uint32_t va[4], vb[4];
    four_pairs(va, wa, bi_kv4::scale_pair(sa));
    four_pairs(vb, wb, bi_kv4::scale_pair(sb));
    bi::mma_bf16_16816(acc0, va[0], va[1], vb[0], vb[1], pf.hi0, pf.hi1);
    bi::mma_bf16_16816(acc0, va[0], va[1], vb[0], vb[1], pf.lo0, pf.lo1);
    bi::mma_bf16_16816(acc1, va[2], va[3], vb[2], vb[3], pf.hi0, pf.hi1);
    bi::mma_bf16_16816(acc1, va[2], va[3], vb[2], vb[3], pf.lo0, pf.lo1);
}

// pv_tiles for group `gr` (a constant) of a loaded V block.
__device__ __forceinline__ void pv_group(float (&acc0)[4], float (&acc1)[4], const VFrags& f, int gr,
                                         const bi_attn::PFrags& pf) {
    const uint32_t half = gr & 1 ? 0x7632u : 0x5410u;
    const bool up = gr & 2;
    pv_tiles(acc0, acc1, __byte_perm(up ? f.ca.y : f.ca.x, up ? f.ca.w : f.ca.z, half),
             __byte_perm(up ? f.cb.y : f.cb.x, up ? f.cb.w : f.cb.z, half),
             __byte_perm(up ? f.sa.y : f.sa.x, up ? f.sa.w : f.sa.z, half),
             __byte_perm(up ? f.sb.y : f.sb.x, up ? f.sb.w : f.sb.z, half), pf);
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

// A chunk's partial in the workspace: O's dims of a row
// in the order of the accumulators, position 16mt + 2g + i for dim 16mt + g +
// 8i.
__device__ __forceinline__ float* partial_o(const SplitArgs& a, int64_t row, int c) {
    return a.ws_acc + (row * a.max_chunks + c) * kD;
}

__device__ __forceinline__ float2* partial_ml(const SplitArgs& a, int64_t row, int c) {
    return reinterpret_cast<float2*>(a.ws_ml) + row * a.max_chunks + c;
}

// bf16(O / l) of a folded row, lane l with positions 4l .. 4l + 3: dims d, d + 8,
// d + 1, d + 9.
__device__ __forceinline__ void store_row(const SplitArgs& a, int64_t row, const float4& o, float l, int lane) {
    const int d = 16 * (lane >> 2) + 2 * (lane & 3);
    const float il = bi_attn::inv_weight(l);
    uint32_t* out = reinterpret_cast<uint32_t*>(a.out + row * kD + d);
    out[0] = bi::pack_bf16x2(bi_attn::normalise(o.x, il), bi_attn::normalise(o.z, il));
    out[4] = bi::pack_bf16x2(bi_attn::normalise(o.y, il), bi_attn::normalise(o.w, il));
}

// (m, l) of a chunk with a page index out of range: no weight sum is negative.
constexpr float kNoChunk = -1.f;

// The factors (2^(M - M'), 2^(m_c - M'), l_c) of 32 chunks of a row, lane = chunk
// with (m_c, l_c) = ml ((-inf, 0) past the last): the running maxima M' are a
// prefix maximum, as in bi_attn::fold_sequence.  m: the running maximum before
// them (unless they are the first), then after them.
__device__ __forceinline__ float4 fold_factors(const float2& ml, float& m, bool first, int lane) {
    float v = ml.x;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const float u = __shfl_up_sync(kAll, v, off);
        if (lane >= off) v = fmaxf(v, u);
    }
    if (!first) v = fmaxf(m, v);
    float before = __shfl_up_sync(kAll, v, 1);
    if (lane == 0) before = first ? 0.f : m;
    m = __shfl_sync(kAll, v, 31);
    return make_float4(bi_attn::exp2_ftz(before - v), bi_attn::exp2_ftz(ml.x - v), ml.y, 0.f);
}

// The fold of a row's chunks, a warp per row (sequence, query head), in
// ascending chunk order with bi_attn::attn_merge_kernel's operations.  Lane l
// has positions 4l .. 4l + 3 of the row; the partials of kAhead chunks are on
// their way together.
//
// A launch of its own, where the rows are folded side by side: the warp
// that arrives last at its (sequence, kv-head) could fold its rows as well, but does
// it alone while the SMs run dry (32 sequences of 8192 tokens 81 against 72 us,
// B = 64 up to 8192 92.6 against 83.1, B = 256 308 against 289).  Sixteen
// partials on their way instead of eight: 78, 89, 296 us.
constexpr int kMergeWarps = 4;

__global__ void __launch_bounds__(32 * kMergeWarps)
    merge_rows_kv4_kernel(const SplitArgs a, int64_t rows) {
    bi::launch_dependents();
    bi::grid_dependency_wait();  // the partials are there
    constexpr int kAhead = 8;
    __shared__ float4 all_factors[kMergeWarps][32];
    float4* const factors = all_factors[threadIdx.x / 32];
    const int lane = threadIdx.x & 31;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * kMergeWarps + threadIdx.x / 32;
    if (row >= rows) return;
    const int L = a.seq_lens[row / a.Hq];
    if (L <= kChunk || L > a.max_seq_len) return;  // written, or reported, by the attention kernel
    const int nch = (L + kChunk - 1) / kChunk;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    float l = 0.f, m = 0.f;
    for (int cb = 0; cb < nch; cb += 32) {
        const int nb = min(32, nch - cb);
        float4 part[kAhead];
        auto load = [&](int i0) {
#pragma unroll
            for (int u = 0; u < kAhead; ++u)
                if (i0 + u < nb)
                    part[u] = __ldcg(reinterpret_cast<const float4*>(partial_o(a, row, cb + i0 + u)) + lane);
        };
        const float2 ml = lane < nb ? __ldcg(partial_ml(a, row, cb + lane)) : make_float2(-INFINITY, 0.f);
        load(0);
        if (__any_sync(kAll, ml.y == kNoChunk)) return;  // the output stays as it was
        const float4 f = fold_factors(ml, m, cb == 0, lane);
        __syncwarp();  // every lane is done with the last factors
        factors[lane] = f;
        __syncwarp();
        for (int i0 = 0; i0 < nb; i0 += kAhead) {
            if (i0 > 0) load(i0);
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                if (i0 + u >= nb) break;
                const float4 f = factors[i0 + u];
                if (cb + i0 + u == 0) {
                    o = part[u];
                    l = f.z;
                } else {
                    o.x = bi_attn::fold_value(o.x, f.x, part[u].x, f.y);
                    o.y = bi_attn::fold_value(o.y, f.x, part[u].y, f.y);
                    o.z = bi_attn::fold_value(o.z, f.x, part[u].z, f.y);
                    o.w = bi_attn::fold_value(o.w, f.x, part[u].w, f.y);
                    l = bi_attn::fold_value(l, f.x, f.z, f.y);
                }
            }
        }
    }
    store_row(a, row, o, l, lane);
}

// The same fold for few rows: a CTA per row, thread p has position p, and 32
// chunks' partials are loaded while the 32 before them are folded, the first
// before the length is known.  One sequence of 32768 tokens (the whole call) 20.0
// against 22.5 us, of 8192 11.3 against 11.6; from 512 rows on it is no faster (B
// = 24 up to 2048 17.2 against 17.0 us, B = 64 up to 8192 86.4 against 83).
constexpr int64_t kFewRows = 512;

__global__ void __launch_bounds__(kD) merge_row_kv4_kernel(const SplitArgs a) {
    bi::launch_dependents();
    bi::grid_dependency_wait();  // the partials are there
    __shared__ float4 all_factors[kD / 32][32];
    const int lane = threadIdx.x & 31;
    float4* const factors = all_factors[threadIdx.x / 32];
    const int64_t row = blockIdx.x;
    const float* const parts = partial_o(a, row, 0) + threadIdx.x;
    const float2* const mls = partial_ml(a, row, 0);
    float next[32];
    float2 next_ml;
    auto load = [&](int c0, int end) {
#pragma unroll
        for (int u = 0; u < 32; ++u)
            if (c0 + u < end) next[u] = __ldcg(parts + (c0 + u) * kD);
    };
    auto load_ml = [&](int c0, int end) {
        next_ml = c0 + lane < end ? __ldcg(mls + c0 + lane) : make_float2(-INFINITY, 0.f);
    };
    // before the length is known: the rows' memory is there, whatever it holds
    load_ml(0, a.max_chunks);
    load(0, a.max_chunks);
    const int L = a.seq_lens[row / a.Hq];
    if (L <= kChunk || L > a.max_seq_len) return;  // written, or reported, by the attention kernel
    const int nch = (L + kChunk - 1) / kChunk;
    float o = 0.f, l = 0.f, m = 0.f;
    for (int cb = 0; cb < nch; cb += 32) {
        const int nb = min(32, nch - cb);
        const float2 ml = lane < nb ? next_ml : make_float2(-INFINITY, 0.f);
        if (__any_sync(kAll, ml.y == kNoChunk)) return;  // the output stays as it was
        load_ml(cb + 32, nch);
        const float4 f = fold_factors(ml, m, cb == 0, lane);
        __syncwarp();  // every lane is done with the last factors
        factors[lane] = f;
        __syncwarp();
        float part[32];
#pragma unroll
        for (int u = 0; u < 32; ++u) part[u] = next[u];
        load(cb + 32, nch);
#pragma unroll
        for (int u = 0; u < 32; ++u) {
            if (u >= nb) break;
            const float4 f = factors[u];
            if (cb + u == 0) {
                o = part[u];
                l = f.z;
            } else {
                o = bi_attn::fold_value(o, f.x, part[u], f.y);
                l = bi_attn::fold_value(l, f.x, f.z, f.y);
            }
        }
    }
    // position 16mt + 2g + i: dim 16mt + g + 8i
    const int d = (threadIdx.x & ~15) + ((threadIdx.x & 15) >> 1) + 8 * (threadIdx.x & 1);
    a.out[row * kD + d] = __float2bfloat16_rn(bi_attn::normalise(o, bi_attn::inv_weight(l)));
}

// Chunks of a sequence up to which the chunk kernel's last CTA folds it.  A launch
// of its own takes the host 3 us (a call for few sequences is bound by the host)
// and folds faster: one sequence of 4096 tokens 9.5 us, against 8.6 folded in
// place, 8192 11.7 and 11.2, 16384 13.6 and 16.5, 32768 19.5 and 27.8.
constexpr int kMaxFolded = 32;

// The fold of a row of up to kMaxFolded chunks by a warp of the CTA that arrived
// last: a round of merge_rows_kv4_kernel with the partials in two halves of shared
// memory (2 * kFoldHalf rows of 512 bytes), the next chunks' on their way while
// the last are folded.
constexpr int kFoldHalf = 8;
static_assert(kWarps * 2 * kFoldHalf * kD * 4 <= kStagingBytes, "a warp's part of the staging memory");

__device__ __forceinline__ void fold_row(const SplitArgs& a, int64_t row, int nch, float4* stage,
                                         float4* factors, int lane) {
    const float4* const parts = reinterpret_cast<const float4*>(partial_o(a, row, 0)) + lane;
    auto copy = [&](int c0, float4* to) {
#pragma unroll
        for (int u = 0; u < kFoldHalf; ++u)
            if (c0 + u < nch) bi::cp_async_16(to + 32 * u + lane, parts + (c0 + u) * (kD / 4));
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    const float2 ml = lane < nch ? __ldcg(partial_ml(a, row, lane)) : make_float2(-INFINITY, 0.f);
    copy(0, stage);
    copy(kFoldHalf, stage + 32 * kFoldHalf);
    float m = 0.f;
    static_assert(kMaxFolded <= 32, "a factor a lane");
    factors[lane] = fold_factors(ml, m, true, lane);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    float l = 0.f;
    for (int cb = 0; cb < nch; cb += kFoldHalf) {
        float4* const half = stage + (cb / kFoldHalf & 1) * 32 * kFoldHalf;
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        __syncwarp();
#pragma unroll
        for (int u = 0; u < kFoldHalf; ++u) {
            if (cb + u >= nch) break;
            const float4 x = half[32 * u + lane];
            const float4 f = factors[cb + u];
            if (cb + u == 0) {
                o = x;
                l = f.z;
            } else {
                o.x = bi_attn::fold_value(o.x, f.x, x.x, f.y);
                o.y = bi_attn::fold_value(o.y, f.x, x.y, f.y);
                o.z = bi_attn::fold_value(o.z, f.x, x.z, f.y);
                o.w = bi_attn::fold_value(o.w, f.x, x.w, f.y);
                l = bi_attn::fold_value(l, f.x, f.z, f.y);
            }
        }
        __syncwarp();  // every lane is done with the half, and in the end with the factors
        copy(cb + 2 * kFoldHalf, half);
    }
    store_row(a, row, o, l, lane);
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
    // several CTAs share a longer sequence; the last one to arrive folds it, if a
    // launch of its own does not
    uint32_t* const ctr = nch > 1 && a.counters ? a.counters + static_cast<int64_t>(s) * a.Hkv + g : nullptr;
    const int64_t row0 = static_cast<int64_t>(s) * a.Hq + g * a.group;

    extern __shared__ __align__(16) uint8_t smem[];
    uint8_t* const ks = smem;
    uint8_t* const vs = smem + kMatBytes;
    uint4* const weights = reinterpret_cast<uint4*>(ks);  // [page][lane], from phase 3 on
    Tables& tb = *reinterpret_cast<Tables*>(smem + kStagingBytes);

    // ---- 0: copies ---- (every warp reads the chunk's pages and copies its own)
    {
        int pg = 0;
        if (lane < np)
            pg = a.block_table[static_cast<int64_t>(s) * a.max_pages_per_seq + c * kPagesPerChunk + lane];
        if (__any_sync(kAll, pg < 0 || pg >= a.num_pages)) {
            if (tid == 0) bi::report_error(a.err, bi::kErrBadInput | bi::kWhereAttnSplit);
            if (ctr) {
                if (tid == 0) bi_attn::arrive_bad(ctr, nch);
            } else if (nch > 1 && tid < a.group) {
                *partial_ml(a, row0 + tid, c) = make_float2(-INFINITY, kNoChunk);
            }
            return;
        }
        const int64_t at = (static_cast<int64_t>(pg) * a.Hkv + g) * kBlockBytes;
        int64_t from[kPagesPerWarp];
#pragma unroll
        for (int i = 0; i < kPagesPerWarp; ++i) from[i] = __shfl_sync(kAll, at, warp + kWarps * i) + 16 * lane;
        auto copy = [&](uint8_t* to, const uint8_t* cache) {
#pragma unroll
            for (int i = 0; i < kPagesPerWarp; ++i) {
                const int p = warp + kWarps * i;
                if (p >= np) break;
                uint8_t* dst = to + p * kBlockBytes + 16 * lane;
                bi::cp_async_16(dst, cache + from[i]);
                bi::cp_async_16(dst + 512, cache + from[i] + 512);
                if (lane < kBlockBytes / 16 - 64) bi::cp_async_16(dst + 1024, cache + from[i] + 1024);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        copy(ks, ka.k_cache);
        copy(vs, ka.v_cache);
    }
    // column n of the mma tile = query head g*group + n (n < group)
    uint32_t qb0[8], qb1[8];
    {
        const int n = lane >> 2;
        bi_attn::load_q_frags(n < a.group ? a.q + (row0 + n) * kD : nullptr, lane, qb0, qb1);
    }

    // ---- 1: scores of this warp's pages, in log2 units, and their maxima ----
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    __syncwarp();  // K, every lane's copies
    float x[kPagesPerWarp][4];
#pragma unroll
    for (int i = 0; i < kPagesPerWarp; ++i) {
        const int p = warp + kWarps * i;
        if (p >= np) break;
        page_logs(x[i], ks + p * kBlockBytes, qb0, qb1, tokens - p * kPage, a.scale_log2, lane);
        const float mx = reduce_columns(fmaxf(x[i][0], x[i][2]), fmaxf(x[i][1], x[i][3]), lane,
                                        [](float u, float v) { return fmaxf(u, v); });
        if (lane < 8) tb.pmax[p][2 * (lane & 3) + (lane >> 2)] = mx;
    }
    bi::cp_async_wait_all();
    __syncthreads();  // the maxima, and V

    // ---- 2: the online softmax's reference maxima (bi_attn::softmax_step) ----
    if (warp == 0) {
        const int n = lane & 7;
        const float m0 = tb.pmax[0][n];  // the first page's maximum is its reference
        float top = m0;
        for (int p = lane >> 3; p < np; p += 4) top = fmaxf(top, tb.pmax[p][n]);
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
        // no page moves it further (as a rule): one reference, no rescaling
        if (__all_sync(0xffffffffu, m0 > -INFINITY && !(top > __fadd_rn(m0, bi_attn::kRescaleSlack)))) {
            if (lane < 8) tb.ref[0][n] = tb.m[n] = m0;
            if (lane == 0) tb.moved = 0u;
        } else {
            float m = -INFINITY;
            uint32_t moved = kRefPerPage;
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
    }
    __syncthreads();
    const uint32_t moved = tb.moved;

    // ---- 3: weights p = 2^(x - m) of this warp's pages, split into bf16 high
    // part and remainder, transposed into mma B fragments ----
#pragma unroll
    for (int i = 0; i < kPagesPerWarp; ++i) {
        const int p = warp + kWarps * i;
        if (p >= np) break;
        const float2 m = *reinterpret_cast<const float2*>(&tb.ref[moved & kRefPerPage ? p : 0][2 * (lane & 3)]);
        const float w[4] = {bi_attn::exp2_ftz(__fsub_rn(x[i][0], m.x)), bi_attn::exp2_ftz(__fsub_rn(x[i][1], m.y)),
                            bi_attn::exp2_ftz(__fsub_rn(x[i][2], m.x)), bi_attn::exp2_ftz(__fsub_rn(x[i][3], m.y))};
        bi_attn::PFrags pf;
        split_weights(w, pf);
        weights[p * 32 + lane] = make_uint4(pf.hi0, pf.hi1, pf.lo0, pf.lo1);
        const float ps = reduce_columns(__fadd_rn(w[0], w[2]), __fadd_rn(w[1], w[3]), lane,
                                        [](float u, float v) { return __fadd_rn(u, v); });
        if (lane < 8) tb.psum[p][2 * (lane & 3) + (lane >> 2)] = ps;
    }
    __syncthreads();

    // ---- 4: O^T of this warp's 32 dims, page after page; l beside it ----
    if (warp == kWarps - 1 && lane < 8) {
        float l = 0.f;
        for (int p = 0; p < np; ++p)
            l = __fmaf_rn(l, moved >> p & 1u ? tb.alpha[p][lane] : 1.f, tb.psum[p][lane]);
        tb.l[lane] = l;
    }
    float acc[2][4];
#pragma unroll
    for (int i = 0; i < 2; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
    const bool up = warp & 2;  // which words and halves hold this warp's group
    const uint32_t half = warp & 1 ? 0x7632u : 0x5410u;
    auto output_page = [&](int p, int valid) {
        const uint8_t* vb = vs + p * kBlockBytes;
        const uint4 ca = *reinterpret_cast<const uint4*>(vb + 16 * lane);
        const uint4 cb = *reinterpret_cast<const uint4*>(vb + 512 + 16 * lane);
        const uint8_t* sp = vb + kScaleOffset + 2 * kScaleRowBytes * (lane & 3) + 4 * (warp >> 1);
        uint32_t s0 = *reinterpret_cast<const uint32_t*>(sp);
        uint32_t s1 = *reinterpret_cast<const uint32_t*>(sp + kScaleRowBytes);
        uint32_t s8 = *reinterpret_cast<const uint32_t*>(sp + 8 * kScaleRowBytes);
        uint32_t s9 = *reinterpret_cast<const uint32_t*>(sp + 9 * kScaleRowBytes);
        if (valid < kPage) {  // as load_v
            const int t = 2 * (lane & 3);
            if (t >= valid) s0 = 0u;
            if (t + 1 >= valid) s1 = 0u;
            if (t + 8 >= valid) s8 = 0u;
            if (t + 9 >= valid) s9 = 0u;
        }
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
        pv_tiles(acc[0], acc[1], __byte_perm(up ? ca.y : ca.x, up ? ca.w : ca.z, half),
                 __byte_perm(up ? cb.y : cb.x, up ? cb.w : cb.z, half), __byte_perm(s0, s1, half),
                 __byte_perm(s8, s9, half), bi_attn::PFrags{w.x, w.y, w.z, w.w});
    };
#pragma unroll 4
    for (int p = 0; p < np - 1; ++p) output_page(p, kPage);
    output_page(np - 1, tokens - (np - 1) * kPage);  // whose last tokens may not be there
    __syncthreads();  // l is there

    const int h0 = 2 * (lane & 3);
    const int d0 = 32 * warp + (lane >> 2);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int h = h0 + e;
        if (h >= a.group) continue;
        const int64_t row = row0 + h;
        if (nch == 1) {  // the whole sequence: bf16(O / l)
            const float il = bi_attn::inv_weight(tb.l[h]);
            __nv_bfloat16* o = a.out + row * kD + d0;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                o[16 * i] = __float2bfloat16_rn(bi_attn::normalise(acc[i][e], il));
                o[16 * i + 8] = __float2bfloat16_rn(bi_attn::normalise(acc[i][2 + e], il));
            }
        } else {  // the chunk's partial
            float2* o = reinterpret_cast<float2*>(partial_o(a, row, c)) + 16 * warp + (lane >> 2);
#pragma unroll
            for (int i = 0; i < 2; ++i) o[8 * i] = make_float2(acc[i][e], acc[i][2 + e]);
            if (warp == 0 && lane < 4) *partial_ml(a, row, c) = make_float2(tb.m[h], tb.l[h]);
        }
    }
    if (!ctr || !bi_attn::arrive_last(a, ctr, nch, tid)) return;
    float4* const stage = reinterpret_cast<float4*>(smem) + warp * 2 * kFoldHalf * 32;
    float4* const factors = reinterpret_cast<float4*>(smem + kStagingBytes) + 32 * warp;
    for (int h = warp; h < a.group; h += kWarps) fold_row(a, row0 + h, nch, stage, factors, lane);
}

// ---------------------------------------------------------------------------
// The many-chunk form: one warp, alone in its CTA, per (sequence, kv-head,
// chunk), so that nothing ever waits for another warp and a finished chunk's
// place on the SM is taken at once.  Pages come through a ring of kRing
// stages; while a page's weights and output products are under way the next
// page's scores are formed (they depend on nothing before them).  351
// instructions a page in all, the chunk's share included; 16 warps per SM (20
// with fewer registers were no faster).  B = 256 up to 8192 tokens took 524 us
// in the four-warp CTA of the bf16 kernel, 341 in this form with bulk copies,
// 308 with per-lane copies in their place (see below), 289 with the fold in a
// launch of its own.

constexpr int kRing = 4;  // pages in flight
constexpr int kStageBytes = 2 * kBlockBytes;

// bi_attn::ColState of two columns, as the fast path of weights_step wants it.
struct WarpState {
    float th[2];   // reference maximum + slack
    float ref[2];  // reference maximum; 0 while it is -inf (then every score is
                   // -inf so far, and so is its difference from 0)
    float l;       // reduce_columns' column of this lane
    float acc[8][4];
};

// The page's weights from its scores in log2 units: bi_attn::softmax_step,
// operation by operation, without what changes nothing.  The reference maximum
// moves on few pages only; one vote finds the others, and there neither the
// page's maximum is formed nor O rescaled (by 1).
__device__ __forceinline__ void weights_step(WarpState& st, const float (&x)[4], bool first, int lane,
                                             bi_attn::PFrags& pf) {
    float mx0 = fmaxf(x[0], x[2]), mx1 = fmaxf(x[1], x[3]);
    float al = 1.f;
    if (__any_sync(kAll, mx0 > st.th[0] || mx1 > st.th[1])) {
#pragma unroll
        for (int off = 4; off <= 16; off <<= 1) {
            mx0 = fmaxf(mx0, __shfl_xor_sync(kAll, mx0, off));
            mx1 = fmaxf(mx1, __shfl_xor_sync(kAll, mx1, off));
        }
        const float m0 = st.th[0] == -INFINITY ? -INFINITY : st.ref[0];
        const float m1 = st.th[1] == -INFINITY ? -INFINITY : st.ref[1];
        const float mn0 = mx0 > st.th[0] ? mx0 : m0;
        const float mn1 = mx1 > st.th[1] ? mx1 : m1;
        const float al0 = mn0 == m0 ? 1.f : bi_attn::exp2_ftz(__fsub_rn(m0, mn0));
        const float al1 = mn1 == m1 ? 1.f : bi_attn::exp2_ftz(__fsub_rn(m1, mn1));
        al = lane & 4 ? al1 : al0;
        st.th[0] = __fadd_rn(mn0, bi_attn::kRescaleSlack);
        st.th[1] = __fadd_rn(mn1, bi_attn::kRescaleSlack);
        st.ref[0] = mn0 == -INFINITY ? 0.f : mn0;
        st.ref[1] = mn1 == -INFINITY ? 0.f : mn1;
        if (!first) {  // O is zero before the first page
#pragma unroll
            for (int mt = 0; mt < 8; ++mt) {
                st.acc[mt][0] = __fmul_rn(st.acc[mt][0], al0);
                st.acc[mt][1] = __fmul_rn(st.acc[mt][1], al1);
                st.acc[mt][2] = __fmul_rn(st.acc[mt][2], al0);
                st.acc[mt][3] = __fmul_rn(st.acc[mt][3], al1);
            }
        }
    }
    const float p[4] = {bi_attn::exp2_ftz(__fsub_rn(x[0], st.ref[0])), bi_attn::exp2_ftz(__fsub_rn(x[1], st.ref[1])),
                        bi_attn::exp2_ftz(__fsub_rn(x[2], st.ref[0])), bi_attn::exp2_ftz(__fsub_rn(x[3], st.ref[1]))};
    split_weights(p, pf);
    st.l = __fmaf_rn(st.l, al,
                     reduce_columns(__fadd_rn(p[0], p[2]), __fadd_rn(p[1], p[3]), lane,
                                    [](float u, float v) { return __fadd_rn(u, v); }));
}

// kLoop: a warp takes chunks gridDim.x apart, else its one.
template <bool kLoop>
__global__ void __launch_bounds__(32, 14) attn_warp_kv4_kernel(const Kv4Args ka) {
    bi::launch_dependents();
    bi::grid_dependency_wait();  // nothing global is touched before the previous kernel ends
    const SplitArgs& a = ka.s;
    const int g = blockIdx.y;
    const int s = blockIdx.z;
    const int lane = threadIdx.x;

    const int L = a.seq_lens[s];
    if (L < 1 || L > a.max_seq_len) {
        if (lane == 0 && blockIdx.x == 0 && g == 0) bi::report_error(a.err, bi::kErrBadInput | bi::kWhereAttnSplit);
        return;
    }
    const int nch = (L + kChunk - 1) / kChunk;
    int c = blockIdx.x;  // chunk
    if (c >= nch) return;
    const int64_t row0 = static_cast<int64_t>(s) * a.Hq + g * a.group;

    __shared__ __align__(16) uint8_t ring[kRing * kStageBytes];

    do {
        const int tokens = min(kChunk, L - c * kChunk);
        const int np = (tokens + kPage - 1) / kPage;
        // lane p keeps which block page p is
        int block = 0;
        {
            int pg = 0;
            if (lane < np)
                pg = a.block_table[static_cast<int64_t>(s) * a.max_pages_per_seq + c * kPagesPerChunk + lane];
            if (__any_sync(kAll, pg < 0 || pg >= a.num_pages)) {
                if (lane == 0) bi::report_error(a.err, bi::kErrBadInput | bi::kWhereAttnSplit);
                if (nch > 1 && lane < a.group)
                    *partial_ml(a, row0 + lane, c) = make_float2(-INFINITY, kNoChunk);
                continue;
            }
            block = pg * a.Hkv + g;
        }
        // A page's two blocks are 72 16-byte units each: two asynchronous copies a
        // lane for each block, and one for the 8 units that are left of either.
        // (Bulk copies, one lane's work, take the warp twice as many instructions,
        // and a barrier's on top.)  A page is a group, there or not.
        static_assert(kBlockBytes == 72 * 16, "units of a block");
        const uint8_t* const k_src = ka.k_cache + 16 * lane;
        const uint8_t* const v_src = ka.v_cache + 16 * lane;
        const uint8_t* const rest_src = 1024 + (lane < 8 ? k_src : v_src - 128);
        const int rest_dst = 1024 + (lane < 8 ? 16 * lane : kBlockBytes + 16 * (lane - 8));
        auto copy_page = [&](int p, uint8_t* stage) {
            if (p < np) {
                const int64_t at = static_cast<int64_t>(__shfl_sync(kAll, block, p)) * kBlockBytes;
                uint8_t* dst = stage + 16 * lane;
                bi::cp_async_16(dst, k_src + at);
                bi::cp_async_16(dst + 512, k_src + at + 512);
                bi::cp_async_16(dst + kBlockBytes, v_src + at);
                bi::cp_async_16(dst + kBlockBytes + 512, v_src + at + 512);
                if (lane < 16) bi::cp_async_16(stage + rest_dst, rest_src + at);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        // until at most kPending of the latest groups are on their way
        auto wait_pages = [](auto pending) {
            asm volatile("cp.async.wait_group %0;" ::"n"(decltype(pending)::value) : "memory");
            __syncwarp();  // every lane's copies, for every lane
        };
#pragma unroll
        for (int p = 0; p < kRing; ++p) copy_page(p, ring + p * kStageBytes);

        // column n of the mma tile = query head g*group + n (n < group)
        uint32_t qb0[8], qb1[8];
        bi_attn::load_q_frags((lane >> 2) < a.group ? a.q + (row0 + (lane >> 2)) * kD : nullptr, lane, qb0, qb1);

        WarpState st;
        st.th[0] = st.th[1] = -INFINITY;
        st.ref[0] = st.ref[1] = 0.f;
        st.l = 0.f;
#pragma unroll
        for (int mt = 0; mt < 8; ++mt) st.acc[mt][0] = st.acc[mt][1] = st.acc[mt][2] = st.acc[mt][3] = 0.f;

        uint8_t* cur = ring;  // the stage of page p
        wait_pages(std::integral_constant<int, kRing - 1>());
        float x[4];
        page_logs(x, cur, qb0, qb1, tokens, a.scale_log2, lane);
        // full pages with a page behind them
        for (int p = 0; p < np - 1; ++p) {
            uint8_t* next = cur + kStageBytes;
            if (next == ring + kRing * kStageBytes) next = ring;
            wait_pages(std::integral_constant<int, kRing - 2>());  // page p + 1 is here
            bi_attn::PFrags pf;
            weights_step(st, x, p == 0, lane, pf);
            VFrags f;
            load_v(f, cur + kBlockBytes, kPage, lane);
            __syncwarp();  // every lane is done with the stage
            copy_page(p + kRing, cur);
            page_logs(x, next, qb0, qb1, kPage, a.scale_log2, lane);
#pragma unroll
            for (int gr = 0; gr < 4; ++gr) pv_group(st.acc[2 * gr], st.acc[2 * gr + 1], f, gr, pf);
            cur = next;
        }
        {  // the last page, whose last tokens may not be there
            const int valid = tokens - (np - 1) * kPage;
            if (valid < kPage) {
                if ((lane >> 2) >= valid) x[0] = x[1] = -INFINITY;
                if ((lane >> 2) + 8 >= valid) x[2] = x[3] = -INFINITY;
            }
            bi_attn::PFrags pf;
            weights_step(st, x, np == 1, lane, pf);
            VFrags f;
            load_v(f, cur + kBlockBytes, valid, lane);
#pragma unroll
            for (int gr = 0; gr < 4; ++gr) pv_group(st.acc[2 * gr], st.acc[2 * gr + 1], f, gr, pf);
        }

        const int h0 = 2 * (lane & 3);
        // both columns' sums: lane l holds one of them, lane l ^ 4 the other
        const float other = __shfl_xor_sync(kAll, st.l, 4);
        const float l[2] = {lane & 4 ? other : st.l, lane & 4 ? st.l : other};
        if (nch == 1) {  // the whole sequence: bf16(O / l)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                if (h0 + e >= a.group) continue;
                const float il = bi_attn::inv_weight(l[e]);
                __nv_bfloat16* o = a.out + (row0 + h0 + e) * kD + (lane >> 2);
#pragma unroll
                for (int mt = 0; mt < 8; ++mt) {
                    o[16 * mt] = __float2bfloat16_rn(bi_attn::normalise(st.acc[mt][e], il));
                    o[16 * mt + 8] = __float2bfloat16_rn(bi_attn::normalise(st.acc[mt][2 + e], il));
                }
            }
            return;
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            if (h0 + e >= a.group) continue;
            float2* o = reinterpret_cast<float2*>(partial_o(a, row0 + h0 + e, c)) + (lane >> 2);
#pragma unroll
            for (int mt = 0; mt < 8; ++mt) o[8 * mt] = make_float2(st.acc[mt][e], st.acc[mt][2 + e]);
            if (lane < 4)
                *partial_ml(a, row0 + h0 + e, c) =
                    make_float2(st.th[e] == -INFINITY ? -INFINITY : st.ref[e], l[e]);
        }
        if (kLoop) __syncwarp();  // every lane is done with the ring
    } while (kLoop && (c += gridDim.x) < nch);
}

// Chunks per SM (at the launch's bound on the lengths; lengths spread up to the
// bound fill about half of them) from which on the warp kernel is taken.
// Measured on GB300 with 8 kv-heads, chunk kernel against warp kernel, folds
// included: 7 per SM (B = 4 up to 8192 tokens) 14.6 against 20.9 us, 14 (B = 8)
// 19.4 against 22.7, (B = 128 up to 512) 20.1 against 22.0, 27 (B = 16 up to
// 8192) 31.9 against 30.5, (B = 256 up to 512) 34.6 against 32.3, 40 (B = 24)
// 46.2 against 41.0, 108 (B = 64) 109 against 83.  The chunk kernel's four warps finish a chunk several times sooner;
// the warp kernel issues a third fewer instructions and has no barriers.  Below
// the rule there are far fewer chunks than arrival counters, and than an arrival
// counter can count.  A call captured under a bound far above its lengths takes the
// form that the bound asks for: 16 sequences of 300 tokens 16.9 us under a bound of
// 8192 (warp kernel), 9.1 under 512; 64 of 2000 tokens 54.2, and 40.5 under 2048.
constexpr int64_t kManyChunks = 22;

// Warps of a launch and of a (sequence, kv-head), about; where the bound on the
// lengths asks for more, a warp takes several chunks.  A warp without a chunk
// costs 0.7 ns, and a bound may be far above the lengths (captured graphs): 256
// sequences of 300 tokens under a bound of 131072 take 52 us, and 1060 with a
// warp a chunk, 8 of them 24 and 40.  Lengths even over 1 .. 8192, which fill
// half of the bound, B = 256, 291 against 289; 1 .. 131072, B = 16, 319 against
// 317.  Half as many warps: 46, 17, 296 and 330 us.
constexpr int64_t kMostWarps = 32768;
constexpr int64_t kMostWarpsOfOne = 256;

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
    const size_t need = bi_decode_attention_workspace_size(B, Hq, D, max_seq_len);
    if (need > 0) {
        if (!workspace || workspace_bytes < need) return BI_ERR_WORKSPACE_TOO_SMALL;
        if (!bi::aligned16(workspace)) return BI_ERR_MISALIGNED;
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
    const dim3 grid(max_chunks, Hkv, B);
    const int64_t most = std::min(
        kMostWarpsOfOne, std::max<int64_t>(1, kMostWarps / (static_cast<int64_t>(Hkv) * B)));
    const bool few =
        static_cast<int64_t>(max_chunks) * Hkv * B < kManyChunks * static_cast<int64_t>(bi::sm_count());
    if (max_chunks > kMaxFolded) args.counters = nullptr;
    const cudaError_t e =
        few
            ? bi::launch_pdl(attn_chunk_kv4_kernel, grid, dim3(kThreads), kSmemBytes, stream, ka)
        : max_chunks <= most
            ? bi::launch_pdl(attn_warp_kv4_kernel<false>, grid, dim3(32), 0, stream, ka)
            : bi::launch_pdl(attn_warp_kv4_kernel<true>, dim3(static_cast<unsigned>(most), Hkv, B), dim3(32),
                             0, stream, ka);
    if (e != cudaSuccess) return BI_ERR_CUDA;
    if (max_chunks == 1 || (few && args.counters)) return BI_OK;
    const int64_t rows = static_cast<int64_t>(B) * Hq;
    const cudaError_t f =
        rows < kFewRows ? bi::launch_pdl(merge_row_kv4_kernel, dim3(static_cast<unsigned>(rows)), dim3(kD),
                                         0, stream, args)
                        : bi::launch_pdl(merge_rows_kv4_kernel, dim3(ceil_div(rows, kMergeWarps)),
                                         dim3(32 * kMergeWarps), 0, stream, args, rows);
    return f == cudaSuccess ? BI_OK : BI_ERR_CUDA;
}
