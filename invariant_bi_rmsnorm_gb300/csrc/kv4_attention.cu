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
// One CTA (4 warps) per (sequence, kv-head, group of consecutive chunks), a
// warp per chunk.  The two 1152-byte blocks of a page (K, V) come by bulk copy
// into a ring of the warp's own; a lane takes its fragments of K and V from
// them with four 16-byte loads, in the order of mma.sync's A operand, and
// turns them into bf16 pairs in registers: a shift, an and-or and one fma for
// two values.
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
using bi_attn::kMaxChunksPerCta;
using bi_attn::kMaxCounters;
using bi_attn::kMaxGroup;
using bi_attn::kMaxPagesPerCta;
using bi_attn::kMergeWideRows;
using bi_attn::kPage;
using bi_attn::kPagesPerChunk;
using bi_attn::kThreads;
using bi_attn::kWarps;
using bi_attn::SplitArgs;
using bi_kv4::kBlockBytes;
using bi_kv4::kScaleOffset;
using bi_kv4::kScaleRowBytes;
using bi_kv4::ScalePair;

constexpr int kSPW = 4;  // pages in flight per warp
constexpr int kStages = kWarps * kSPW;
constexpr int kStageBytes = 2 * kBlockBytes;  // K + V of one page
constexpr int kRingBytes = kStages * kStageBytes;
constexpr int kSmemBytes = kRingBytes + kFoldFloats * 4 + 4 * kMaxPagesPerCta + 8 * kStages + 16 /*align*/;

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

// A lane's part of a 4-bit V block: codes and scales of tokens 2(l%4) and the
// next (a), and of the two tokens 8 further on (b).
struct VFrags {
    uint4 ca, cb, sa, sb;
};

__device__ __forceinline__ void load_v(VFrags& f, const uint8_t* vb, int lane) {
    f.ca = *reinterpret_cast<const uint4*>(vb + 16 * lane);
    f.cb = *reinterpret_cast<const uint4*>(vb + 512 + 16 * lane);
    const uint8_t* sp = vb + kScaleOffset + 2 * kScaleRowBytes * (lane & 3);
    f.sa = *reinterpret_cast<const uint4*>(sp);
    f.sb = *reinterpret_cast<const uint4*>(sp + 8 * kScaleRowBytes);
}

// Tokens from `valid` on stand for zeros, whatever the block holds there.
__device__ __forceinline__ void mask_v(VFrags& f, int valid, int lane) {
    const int t = 2 * (lane & 3);
    if (t >= valid) f.sa.x = f.sa.y = 0u;
    if (t + 1 >= valid) f.sa.z = f.sa.w = 0u;
    if (t + 8 >= valid) f.sb.x = f.sb.y = 0u;
    if (t + 9 >= valid) f.sb.z = f.sb.w = 0u;
}

// bi_attn::pv_step over a 4-bit V block.
__device__ __forceinline__ void pv_step_kv4(bi_attn::ColState& st, const bi_attn::PFrags& pf,
                                            const VFrags& f) {
#pragma unroll
    for (int gr = 0; gr < 4; ++gr) {  // the group of dims 32gr .. 32gr + 31: two 16-dim tiles
        // codes of (even token, odd token) side by side; their scales likewise
        const uint32_t ae = gr < 2 ? f.ca.x : f.ca.y, ao = gr < 2 ? f.ca.z : f.ca.w;
        const uint32_t be = gr < 2 ? f.cb.x : f.cb.y, bo = gr < 2 ? f.cb.z : f.cb.w;
        const uint32_t sae = gr < 2 ? f.sa.x : f.sa.y, sao = gr < 2 ? f.sa.z : f.sa.w;
        const uint32_t sbe = gr < 2 ? f.sb.x : f.sb.y, sbo = gr < 2 ? f.sb.z : f.sb.w;
        const uint32_t wa = gr & 1 ? hi_halves(ae, ao) : lo_halves(ae, ao);
        const uint32_t wb = gr & 1 ? hi_halves(be, bo) : lo_halves(be, bo);
        const ScalePair pa = bi_kv4::scale_pair(gr & 1 ? hi_halves(sae, sao) : lo_halves(sae, sao));
        const ScalePair pb = bi_kv4::scale_pair(gr & 1 ? hi_halves(sbe, sbo) : lo_halves(sbe, sbo));
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int mt = 2 * gr + e;
            const uint32_t a0 = bi_kv4::kv4_pair(wa, 2 * e, pa), a1 = bi_kv4::kv4_pair(wa, 2 * e + 1, pa);
            const uint32_t a2 = bi_kv4::kv4_pair(wb, 2 * e, pb), a3 = bi_kv4::kv4_pair(wb, 2 * e + 1, pb);
            bi::mma_bf16_16816(st.acc[mt], a0, a1, a2, a3, pf.hi0, pf.hi1);
            bi::mma_bf16_16816(st.acc[mt], a0, a1, a2, a3, pf.lo0, pf.lo1);
        }
    }
}

__global__ void __launch_bounds__(kThreads) attn_split_kv4_kernel(const Kv4Args ka) {
    bi::launch_dependents();
    bi::grid_dependency_wait();  // nothing global is touched before the previous kernel ends
    const SplitArgs& a = ka.s;
    const int cg = blockIdx.x;  // chunk group
    const int g = blockIdx.y;
    const int s = blockIdx.z;
    const int tid = threadIdx.x;
    const int warp = tid >> 5;
    const int lane = tid & 31;

    const int L = a.seq_lens[s];
    if (L < 1 || L > a.max_seq_len) {
        if (tid == 0 && cg == 0 && g == 0) bi::report_error(a.err, bi::kErrBadInput | bi::kWhereAttnSplit);
        return;
    }
    const int npg_total = (L + kPage - 1) / kPage;
    const int nch = (npg_total + kPagesPerChunk - 1) / kPagesPerChunk;
    const int c0 = cg * a.chunks_per_cta;
    if (c0 >= nch) return;
    const int c1 = min(nch, c0 + a.chunks_per_cta);
    const bool whole = (c0 == 0 && c1 == nch);  // this CTA folds the whole sequence
    const bool shared_fold = !whole && a.counters != nullptr;
    const uint32_t ngroups = static_cast<uint32_t>((nch + a.chunks_per_cta - 1) / a.chunks_per_cta);
    uint32_t* const ctr = shared_fold ? a.counters + static_cast<int64_t>(s) * a.Hkv + g : nullptr;
    const int pg0 = c0 * kPagesPerChunk;
    const int npg_group = min(c1 * kPagesPerChunk, npg_total) - pg0;

    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 15) & ~static_cast<uintptr_t>(15));
    float* fold_o = reinterpret_cast<float*>(smem + kRingBytes);  // [8 heads][128]
    float* fold_m = fold_o + kMaxGroup * kD;                      // [8]
    float* fold_l = fold_m + kMaxGroup;                           // [8]
    int32_t* blocks_s = reinterpret_cast<int32_t*>(fold_l + kMaxGroup);  // block per page
    uint64_t* bars = reinterpret_cast<uint64_t*>(blocks_s + kMaxPagesPerCta);
    __shared__ int bad_page;

    if (tid == 0) {
        bad_page = 0;
        for (int i = 0; i < kStages; ++i) bi::mbar_init(&bars[i], 1);
        bi::fence_mbar_init();
    }
    __syncthreads();
    for (int i = tid; i < npg_group; i += kThreads) {
        const int pg = a.block_table[static_cast<int64_t>(s) * a.max_pages_per_seq + pg0 + i];
        if (pg < 0 || pg >= a.num_pages) {
            bad_page = 1;
        } else {
            blocks_s[i] = pg * a.Hkv + g;
        }
    }
    __syncthreads();
    if (bad_page) {
        if (tid == 0) {
            bi::report_error(a.err, bi::kErrBadInput | bi::kWhereAttnSplit);
            if (shared_fold) bi_attn::arrive_bad(ctr, ngroups);
        }
        return;
    }

    auto pages_in = [&](int c) { return min(kPagesPerChunk, npg_total - c * kPagesPerChunk); };
    auto stage_ptr = [&](int st) { return smem + st * kStageBytes; };

    // this warp's pages in order, kSPW copies ahead of the compute loop
    int lc = c0 + warp, lp = 0, lj = 0;
    auto issue_next = [&]() {
        if (lc >= c1) return;
        if (lane == 0) {
            const int st = warp * kSPW + lj % kSPW;
            uint8_t* kd = stage_ptr(st);
            const int64_t at = static_cast<int64_t>(blocks_s[(lc - c0) * kPagesPerChunk + lp]) * kBlockBytes;
            bi::mbar_arrive_expect_tx(&bars[st], kStageBytes);
            bulk_load(kd, ka.k_cache + at, kBlockBytes, &bars[st]);
            bulk_load(kd + kBlockBytes, ka.v_cache + at, kBlockBytes, &bars[st]);
        }
        ++lj;
        if (++lp >= pages_in(lc)) {
            lc += kWarps;
            lp = 0;
        }
    };
#pragma unroll
    for (int i = 0; i < kSPW; ++i) issue_next();

    // column n of the mma tile = query head g*group + n (n < group)
    uint32_t qb0[8], qb1[8];
    {
        const int n = lane >> 2;
        bi_attn::load_q_frags(
            n < a.group ? a.q + (static_cast<int64_t>(s) * a.Hq + g * a.group + n) * kD : nullptr,
            lane, qb0, qb1);
    }
    bool timed_out = false;
    int j = 0;       // this warp's page counter (matches the loader's)
    int j_fail = 0;  // first page whose wait timed out
    const int rounds = (c1 - c0 + kWarps - 1) / kWarps;

    for (int r = 0; r < rounds; ++r) {
        const int c = c0 + r * kWarps + warp;  // this warp's chunk in round r
        bi_attn::ColState st;
        bi_attn::colstate_init(st);
        if (c < c1) {
            const int np = pages_in(c);
            for (int p = 0; p < np; ++p, ++j) {
                const int stg = warp * kSPW + j % kSPW;
                if (timed_out) continue;
                if (!__all_sync(0xffffffffu, bi::mbar_wait(&bars[stg], (j / kSPW) & 1))) {
                    timed_out = true;
                    j_fail = j;
                    continue;
                }
                const int valid = min(kPage, L - (c * kPagesPerChunk + p) * kPage);
                const uint8_t* kb = stage_ptr(stg);
                float sc[4];
                page_scores_kv4(sc, kb, qb0, qb1, lane);
                VFrags vf;
                load_v(vf, kb + kBlockBytes, lane);
                if (valid < kPage) mask_v(vf, valid, lane);
                bi_attn::PFrags pf;
                bi_attn::softmax_step(st, sc, valid, valid, a.scale_log2, lane, pf);
                pv_step_kv4(st, pf, vf);
                __syncwarp();  // every lane has read the stage
                issue_next();
            }
            if (!whole) bi_attn::store_partial(a, st, s, g, c, lane);
        }
        if (whole) {
            // fold this round's chunks into the running state, in chunk order
            for (int w = 0; w < kWarps; ++w) {
                if (warp == w && c < c1) bi_attn::fold_chunk(st, c, fold_o, fold_m, fold_l, lane);
                __syncthreads();
            }
        }
    }

    if (timed_out && lane == 0) {
        bi::report_error(a.err, bi::kErrTimeout | bi::kWhereAttnSplit);
        // pages j_fail .. lj-1 were issued and never seen to land: one more
        // bounded wait each before this warp's stages are released
        for (int i = j_fail; i < lj; ++i)
            bi::mbar_wait_for(&bars[warp * kSPW + i % kSPW], (i / kSPW) & 1, bi::kDrainNs);
    }
    if (whole) {
        bi_attn::write_folded(a, s, g, fold_o, fold_l, tid);
        return;
    }
    if (!shared_fold) return;  // the merge kernel folds
    // the last CTA of this (sequence, kv-head) to arrive folds it
    bi_attn::arrive_and_fold<kRingBytes>(a, ctr, ngroups, s, g, nch, smem, fold_o, tid);
}

// set once per device; any thread may race to set it, the attribute is idempotent
std::atomic<bool> g_attr_set[64] = {};

// Schedule (never the arithmetic): how many consecutive chunks one CTA walks.
int chunks_per_cta(int64_t B, int64_t Hkv, int64_t max_chunks) {
    return B * Hkv * max_chunks >= (int64_t{1} << 16) ? kMaxChunksPerCta : kWarps;
}

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

    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return BI_ERR_CUDA;
    if (!g_attr_set[dev]) {
        if (cudaFuncSetAttribute(attn_split_kv4_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
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
    const bool counted = need && static_cast<int64_t>(B) * Hkv <= kMaxCounters;
    args.counters = counted ? reinterpret_cast<uint32_t*>(ws) : nullptr;
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
    const int cpc = chunks_per_cta(B, Hkv, max_chunks);
    args.chunks_per_cta = cpc;
    if (bi::launch_pdl(attn_split_kv4_kernel, dim3(ceil_div(max_chunks, cpc), Hkv, B),
                       dim3(kThreads), kSmemBytes, stream, ka) != cudaSuccess)
        return BI_ERR_CUDA;
    if (max_chunks > cpc && !counted) {
        const cudaError_t e =
            static_cast<int64_t>(B) * Hq <= kMergeWideRows
                ? bi::launch_pdl(bi_attn::attn_merge_kernel<32>, dim3(Hq, B), dim3(kD), 0, stream,
                                 seq_lens, static_cast<const float*>(args.ws_acc),
                                 static_cast<const float*>(args.ws_ml), args.out, Hq, max_chunks,
                                 max_seq_len, 0, cpc)
                : bi::launch_pdl(bi_attn::attn_merge_kernel<8>, dim3(Hq, B), dim3(kD), 0, stream,
                                 seq_lens, static_cast<const float*>(args.ws_acc),
                                 static_cast<const float*>(args.ws_ml), args.out, Hq, max_chunks,
                                 max_seq_len, 0, cpc);
        if (e != cudaSuccess) return BI_ERR_CUDA;
    }
    return BI_OK;
}
