// What follows once a chunk's pages have been walked.  The decode-attention
// kernels over a bf16 cache and over a 4-bit cache share the launch's arguments,
// the workspace of chunk partials and its arrival counters (SplitArgs,
// arrive_last, arrive_bad).  The chunk geometry of both strategies, the folds of a
// sequence's partials in ascending chunk order and what stores and reads those
// partials are the bf16 cache's; the 4-bit kernels keep partials in another order
// and fold them with the same operations (kv4_attention.cu).
#pragma once
#include <cuda_bf16.h>

#include <cmath>

#include "attn_common.cuh"
#include "bi_internal.h"
#include "bi_ptx.cuh"

namespace bi_attn {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxPagesPerCta = 512;                                // pages one CTA walks
constexpr int kMaxChunksPerCta = kMaxPagesPerCta / kPagesPerChunk;  // 32
constexpr int kFoldFloats = kMaxGroup * kD + 2 * kMaxGroup;          // running fold (O, M, L)

// Arrival counters at the start of the workspace: one uint32 per (sequence,
// kv-head), low 16 bits = CTAs arrived, high bits set by a CTA that found a bad
// page index.  Every call leaves them zero.
constexpr int64_t kMaxCounters = BI_DECODE_COUNTER_BYTES / 4;
constexpr uint32_t kArrive = 1u;
constexpr uint32_t kArriveBad = 0x10001u;

struct SplitArgs {
    const __nv_bfloat16* q;
    const int32_t* block_table;
    const int32_t* seq_lens;
    __nv_bfloat16* out;
    float* ws_acc;  // [B][Hq][max_chunks][D]
    float* ws_ml;   // [B][Hq][max_chunks][2]
    uint32_t* counters;  // [B][Hkv] arrival counters; nullptr: the merge kernel folds
    uint32_t* err;
    int max_pages_per_seq;
    int Hq, Hkv, group;
    int num_pages;
    int max_seq_len;
    int max_chunks;
    int num_splits;    // 0: fixed 256-token chunks; > 0: fixed split count (comparison variant)
    int chunks_per_cta;  // consecutive chunks one CTA walks (a schedule choice only)
    float scale_log2;  // scale * log2(e)
};

// Chunk geometry of one sequence of L tokens: pages per chunk and chunk count.
// Fixed split size (num_splits == 0, the batch-invariant method): 16 pages =
// 256 tokens per chunk, whatever L is.  Fixed split count (num_splits > 0),
// the strategy the pages warn against and kept here only as a comparison: the
// sequence's pages are cut into num_splits nearly equal runs, so the chunk
// size, and with it the reduction order, changes as L grows.
__device__ __forceinline__ void chunk_geometry(int L, int num_splits, int& ppc, int& nch) {
    const int npg = (L + kPage - 1) / kPage;
    ppc = num_splits > 0 ? (npg + num_splits - 1) / num_splits : kPagesPerChunk;
    nch = (npg + ppc - 1) / ppc;
}

// The fold of one (sequence, kv-head) by the CTA that arrived last: for each
// of its G query heads h and dims d (thread d), the chunk partials are folded
// in ascending chunk order,
//     M' = max(M, m_c);  fo = 2^(M - M');  fc = 2^(m_c - M');
//     l' = fma(l_c, fc, l * fo);  O' = fma(O_c, fc, O * fo),
// starting from chunk 0's (m, l, O), and bf16(O / l) is written -- exactly the
// merge kernel's operations, on the same values.  Only the schedule differs:
//   - the running maxima M are a prefix maximum, exact in any evaluation
//     order, so a warp computes them for 32 chunks at once by a shuffle scan,
//     and with them every chunk's factors fo, fc;
//   - the recurrences of l and O then run in every thread from shared
//     memory, loads issued a few chunks ahead (each thread computes its
//     heads' l itself, the same operations on the same values).
// The partials are staged in shared memory (kStagingBytes of `stage`: the
// page ring, free by now) a batch of chunks at a time: the (m, l) pairs first,
// then the unnormalised outputs by cp.async while the factors are computed.
// ws reads go through L2 only (ld.cg, cp.async.cg): the data was written by
// other CTAs.
template <int G, int kStagingBytes>
__device__ __forceinline__ void fold_sequence(const SplitArgs& a, int s, int g, int nch,
                                              uint8_t* stage, float* small, int tid) {
    constexpr int kcb = kStagingBytes / (G * kD * 4);  // chunks per batch
    static_assert(kcb >= 1 && G * kcb <= kThreads, "one (m, l) pair per thread");
    // thread -> (head, G consecutive dims) when G divides 128 (vector loads,
    // one head per warp at G = 4); otherwise thread d -> dim d of every head
    constexpr bool kVec = kThreads % G == 0 && kD == kThreads;  // G = 1, 2, 4, 8
    constexpr int TPH = kVec ? kThreads / G : kThreads;  // threads per head
    constexpr int NH = kVec ? 1 : G;                     // heads per thread
    constexpr int ND = kVec ? G : 1;                     // dims per thread
    constexpr int U = kVec ? 4 : (16 / G > 0 ? 16 / G : 1);  // chunks loaded ahead
    float* acc_s = reinterpret_cast<float*>(stage);  // [kcb][G][kD]
    float* ml_s = small;                             // [kcb][G][2]  (m_c, l_c)
    float4* fl = reinterpret_cast<float4*>(small + 256);  // [kcb][G]  (fo, fc, l_c, -)
    float* mcarry = small + 768;                     // [G] running max before the batch
    const int lane = tid & 31, warp = tid >> 5;
    const int64_t row0 = static_cast<int64_t>(s) * a.Hq + g * G;
    const int h0 = kVec ? tid / TPH : 0;               // this thread's (first) head
    const int d0 = kVec ? (tid % TPH) * ND : tid;      // this thread's first dim
    float A[NH][ND], Lr[NH];
#pragma unroll
    for (int j = 0; j < NH; ++j) {
        Lr[j] = 0.f;
#pragma unroll
        for (int e = 0; e < ND; ++e) A[j][e] = 0.f;
    }
    for (int cb = 0; cb < nch; cb += kcb) {
        const int nb = min(kcb, nch - cb);
        float2 ml = make_float2(0.f, 0.f);  // one (m, l) pair per thread (nb * G <= 128)
        const int mi = tid / G, mh = tid - mi * G;
        if (mi < nb)
            ml = __ldcg(reinterpret_cast<const float2*>(a.ws_ml + ((row0 + mh) * a.max_chunks + cb + mi) * 2));
        for (int idx = tid; idx < nb * G * (kD / 4); idx += kThreads) {
            const int v = idx % (kD / 4);
            const int hg = idx / (kD / 4);  // i * G + h
            const int i = hg / G, h = hg - i * G;
            bi::cp_async_16(acc_s + hg * kD + 4 * v,
                            a.ws_acc + ((row0 + h) * a.max_chunks + cb + i) * kD + 4 * v);
        }
        if (mi < nb) *reinterpret_cast<float2*>(ml_s + 2 * tid) = ml;
        __syncthreads();  // (m, l) staged; the outputs may still be in flight
        for (int h = warp; h < G; h += kWarps) {
            float carry = cb == 0 ? -INFINITY : mcarry[h];
            for (int j0 = 0; j0 < nb; j0 += 32) {
                const int i = j0 + lane;
                const int k = i * G + h;
                const float mc = i < nb ? ml_s[2 * k] : -INFINITY;
                float v = mc;  // inclusive prefix maximum over the lanes
#pragma unroll
                for (int off = 1; off < 32; off <<= 1) {
                    const float o = __shfl_up_sync(0xffffffffu, v, off);
                    if (lane >= off) v = fmaxf(v, o);
                }
                // running max after chunk cb + i (chunk 0 starts the run)
                const float Mn = cb + j0 == 0 ? v : fmaxf(carry, v);
                float Mo = __shfl_up_sync(0xffffffffu, Mn, 1);
                if (lane == 0) Mo = carry;
                if (i < nb) {
                    const bool first = cb + i == 0;  // chunk 0: no factors
                    fl[k] = make_float4(first ? 0.f : bi_attn::exp2_ftz(Mo - Mn),
                                        first ? 0.f : bi_attn::exp2_ftz(mc - Mn), ml_s[2 * k + 1], 0.f);
                }
                carry = __shfl_sync(0xffffffffu, Mn, 31);
            }
            __syncwarp();
            if (lane == 0) mcarry[h] = carry;
        }
        bi::cp_async_wait_all();
        __syncthreads();  // factors and outputs staged
        for (int i0 = 0; i0 < nb; i0 += U) {
            float x[U][NH][ND];
            float4 f[U][NH];
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int j = 0; j < NH; ++j) {
                    const int k = (i0 + u) * G + h0 + j;
                    if (i0 + u < nb) {
                        f[u][j] = fl[k];
                        const float* xs = acc_s + k * kD + d0;
                        if constexpr (ND % 4 == 0) {
#pragma unroll
                            for (int e = 0; e < ND; e += 4) {
                                const float4 t = *reinterpret_cast<const float4*>(xs + e);
                                x[u][j][e] = t.x;
                                x[u][j][e + 1] = t.y;
                                x[u][j][e + 2] = t.z;
                                x[u][j][e + 3] = t.w;
                            }
                        } else if constexpr (ND == 2) {
                            const float2 t = *reinterpret_cast<const float2*>(xs);
                            x[u][j][0] = t.x;
                            x[u][j][1] = t.y;
                        } else {
                            x[u][j][0] = xs[0];
                        }
                    }
                }
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int j = 0; j < NH; ++j) {
                    if (i0 + u >= nb) continue;
                    if (cb + i0 + u == 0) {
                        Lr[j] = f[u][j].z;
#pragma unroll
                        for (int e = 0; e < ND; ++e) A[j][e] = x[u][j][e];
                    } else {
                        const float fo = f[u][j].x, fc = f[u][j].y;
                        Lr[j] = bi_attn::fold_value(Lr[j], fo, f[u][j].z, fc);
#pragma unroll
                        for (int e = 0; e < ND; ++e) A[j][e] = bi_attn::fold_value(A[j][e], fo, x[u][j][e], fc);
                    }
                }
        }
        __syncthreads();  // staging is reused by the next batch
    }
#pragma unroll
    for (int j = 0; j < NH; ++j) {
        __nv_bfloat16* o = a.out + (row0 + h0 + j) * kD + d0;
        const float il = bi_attn::inv_weight(Lr[j]);
        if constexpr (ND % 2 == 0) {
#pragma unroll
            for (int e = 0; e < ND; e += 2)
                *reinterpret_cast<__nv_bfloat162*>(o + e) = __halves2bfloat162(
                    __float2bfloat16_rn(bi_attn::normalise(A[j][e], il)),
                    __float2bfloat16_rn(bi_attn::normalise(A[j][e + 1], il)));
        } else {
            o[0] = __float2bfloat16_rn(bi_attn::normalise(A[j][0], il));
        }
    }
}

// fold_sequence for the launch's group size.
template <int kStagingBytes>
__device__ __forceinline__ void fold_group(const SplitArgs& a, int s, int g, int nch,
                                           uint8_t* stage, float* small, int tid) {
    switch (a.group) {
        case 1: fold_sequence<1, kStagingBytes>(a, s, g, nch, stage, small, tid); break;
        case 2: fold_sequence<2, kStagingBytes>(a, s, g, nch, stage, small, tid); break;
        case 3: fold_sequence<3, kStagingBytes>(a, s, g, nch, stage, small, tid); break;
        case 4: fold_sequence<4, kStagingBytes>(a, s, g, nch, stage, small, tid); break;
        case 5: fold_sequence<5, kStagingBytes>(a, s, g, nch, stage, small, tid); break;
        case 6: fold_sequence<6, kStagingBytes>(a, s, g, nch, stage, small, tid); break;
        case 7: fold_sequence<7, kStagingBytes>(a, s, g, nch, stage, small, tid); break;
        default: fold_sequence<8, kStagingBytes>(a, s, g, nch, stage, small, tid); break;
    }
}

// A chunk's final state (one warp) -> its partial in the workspace.
__device__ __forceinline__ void store_partial(const SplitArgs& a, const ColState& st, int s, int g,
                                              int c, int lane) {
    const int h0 = 2 * (lane & 3);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int h = h0 + e;
        if (h >= a.group) continue;
        const int64_t pidx = (static_cast<int64_t>(s) * a.Hq + g * a.group + h) * a.max_chunks + c;
#pragma unroll
        for (int mt = 0; mt < 8; ++mt) {
            const int d = 16 * mt + (lane >> 2);
            a.ws_acc[pidx * kD + d] = st.acc[mt][e];
            a.ws_acc[pidx * kD + d + 8] = st.acc[mt][2 + e];
        }
        if (lane < 4) {
            a.ws_ml[pidx * 2] = st.m[e];
            a.ws_ml[pidx * 2 + 1] = st.l[e];
        }
    }
}

// A chunk's final state (one warp) folded into the CTA's running state of the
// sequence, fold_o [8 heads][128], fold_m [8], fold_l [8] in shared memory;
// chunk 0 starts it.  The caller runs the chunks in order.
__device__ __forceinline__ void fold_chunk(const ColState& st, int c, float* fold_o, float* fold_m,
                                           float* fold_l, int lane) {
    const int h0 = 2 * (lane & 3);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int h = h0 + e;
        if (c == 0) {
#pragma unroll
            for (int mt = 0; mt < 8; ++mt) {
                const int d = 16 * mt + (lane >> 2);
                fold_o[h * kD + d] = st.acc[mt][e];
                fold_o[h * kD + d + 8] = st.acc[mt][2 + e];
            }
        } else {
            float Mn, fo, fc;
            fold_scalars(fold_m[h], st.m[e], Mn, fo, fc);
#pragma unroll
            for (int mt = 0; mt < 8; ++mt) {
                const int d = 16 * mt + (lane >> 2);
                float* o = fold_o + h * kD + d;
                o[0] = fold_value(o[0], fo, st.acc[mt][e], fc);
                o[8] = fold_value(o[8], fo, st.acc[mt][2 + e], fc);
            }
        }
    }
    __syncwarp();  // every lane has read M before lanes 0..3 replace it
    if (lane < 4) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int h = h0 + e;
            if (c == 0) {
                fold_m[h] = st.m[e];
                fold_l[h] = st.l[e];
            } else {
                float Mn, fo, fc;
                fold_scalars(fold_m[h], st.m[e], Mn, fo, fc);
                fold_l[h] = fold_value(fold_l[h], fo, st.l[e], fc);
                fold_m[h] = Mn;
            }
        }
    }
}

// bf16(O / l) of a sequence that one CTA folded whole (thread d: dim d).
__device__ __forceinline__ void write_folded(const SplitArgs& a, int s, int g, const float* fold_o,
                                             const float* fold_l, int tid) {
    for (int h = 0; h < a.group; ++h) {
        const int64_t row = static_cast<int64_t>(s) * a.Hq + g * a.group + h;
        a.out[row * kD + tid] =
            __float2bfloat16_rn(normalise(fold_o[h * kD + tid], inv_weight(fold_l[h])));
    }
}

// Count in a CTA that found a bad page, marking the sequence (its output stays
// unwritten); the last arrival still returns the counter to zero.
__device__ __forceinline__ void arrive_bad(uint32_t* ctr, uint32_t ngroups) {
    const uint32_t now = bi::atomic_add_acq_rel_gpu(ctr, kArriveBad) + kArriveBad;
    if ((now & 0xffffu) == ngroups) atomicExch(ctr, 0u);
}

// Count this CTA in on its (sequence, kv-head)'s counter once its partials
// are stored.  True in the last of `ngroups` CTAs to arrive, if none found a bad
// page: it folds the sequence.
__device__ __forceinline__ bool arrive_last(const SplitArgs& a, uint32_t* ctr, uint32_t ngroups, int tid) {
    __shared__ int fold_here;
    __syncthreads();  // every warp's partial stores precede the arrival
    if (tid == 0) {
        // release: this CTA's partials are visible before its arrival counts;
        // acquire: the last arrival sees every other CTA's partials
        const uint32_t now = bi::atomic_add_acq_rel_gpu(ctr, kArrive) + kArrive;
        const bool last = (now & 0xffffu) == ngroups;
        if (last) {
            atomicExch(ctr, 0u);  // ready for the next call
            if (now >> 16) bi::report_error(a.err, bi::kErrBadInput | bi::kWhereAttnSplit);
        }
        fold_here = last && (now >> 16) == 0;
    }
    __syncthreads();
    return fold_here;
}

template <int kStagingBytes>
__device__ __forceinline__ void arrive_and_fold(const SplitArgs& a, uint32_t* ctr, uint32_t ngroups,
                                                int s, int g, int nch, uint8_t* stage, float* small,
                                                int tid) {
    if (arrive_last(a, ctr, ngroups, tid)) fold_group<kStagingBytes>(a, s, g, nch, stage, small, tid);
}

// Fold the chunk partials of one (sequence, query head) in ascending chunk
// order:  M' = max(M, m_c);  l' = l 2^(M-M') + l_c 2^(m_c-M');
//         O' = O 2^(M-M') + O_c 2^(m_c-M');   out = bf16(O / l).
// kBatch: chunks whose partials are loaded before any of them is folded (a
// schedule choice; the fold stays strictly sequential in c).
template <int kBatch>
static __global__ void __launch_bounds__(kD)
    attn_merge_kernel(const int32_t* __restrict__ seq_lens, const float* __restrict__ ws_acc,
                      const float* __restrict__ ws_ml, __nv_bfloat16* __restrict__ out, int Hq,
                      int max_chunks, int max_seq_len, int num_splits, int chunks_per_cta) {
    bi::launch_dependents();
    bi::grid_dependency_wait();  // nothing global is touched before the previous kernel ends
    const int hq = blockIdx.x;
    const int s = blockIdx.y;
    const int d = threadIdx.x;
    const int L = seq_lens[s];
    if (L < 1 || L > max_seq_len) return;  // reported by the split kernel
    int ppc, nch;
    chunk_geometry(L, num_splits, ppc, nch);
    if (nch <= chunks_per_cta) return;  // one CTA walked and folded every chunk
    const int64_t base = (static_cast<int64_t>(s) * Hq + hq) * max_chunks;
    float M = ws_ml[base * 2];
    float Ls = ws_ml[base * 2 + 1];
    float A = ws_acc[base * kD + d];
    for (int cb = 1; cb < nch; cb += kBatch) {
        float mc[kBatch], lc[kBatch], ac[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            if (cb + i < nch) {
                const int64_t pc = base + cb + i;
                mc[i] = ws_ml[pc * 2];
                lc[i] = ws_ml[pc * 2 + 1];
                ac[i] = ws_acc[pc * kD + d];
            }
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            if (cb + i >= nch) break;
            float Mn, fo, fc;
            bi_attn::fold_scalars(M, mc[i], Mn, fo, fc);
            Ls = bi_attn::fold_value(Ls, fo, lc[i], fc);
            A = bi_attn::fold_value(A, fo, ac[i], fc);
            M = Mn;
        }
    }
    out[(static_cast<int64_t>(s) * Hq + hq) * kD + d] =
        __float2bfloat16_rn(bi_attn::normalise(A, bi_attn::inv_weight(Ls)));
}

inline int ceil_div(int64_t a, int64_t b) { return static_cast<int>((a + b - 1) / b); }

// (sequence, query head) rows up to which the merge batches 32 chunks' loads:
// at B = 1 that was 2-3 us faster than 8; at 64 sequences and more it was 2 %
// slower (more registers, fewer resident CTAs).
constexpr int64_t kMergeWideRows = 512;

}  // namespace bi_attn
