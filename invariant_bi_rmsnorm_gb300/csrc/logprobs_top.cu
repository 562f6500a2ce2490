// bi_logprobs_top: the log-sum-exp and target log-probability of a logits row
// (bi_logprobs' bits for logits within +-1024), the entropy of its softmax, and
// its k largest logits as token ids and log-probabilities (equal logits: the
// lower id first).
//
// "Defeating Nondeterminism in LLM Inference: The Core Role of Batch
// Invariance", section "Experimental Validation and Future Prospects" (true
// on-policy RL): what a sampler reports of a token must not depend on the
// batch.  One row per CTA; every reduction's order is fixed by the vocabulary
// size, and which logits are the k largest does not depend on any order.
//
// One pass over the row (HBM), as bi_logprobs: thread t folds its vectors t,
// t + 256, ... into (m, s) with the same operations, and beside them
//     T = sum_j 2^(d_j) d_j,   d_j = (x_j - m) log2(e)          (fp32)
// (m' = m + D moves d by -D log2(e): T' = (T + (m - m') log2(e) S) 2^(..)), so
//     entropy = -sum p ln p = ln S - ln 2 * T / S,
// in which nothing cancels: ln S >= 0 and T <= 0.  S is s and a small correction
// beside it (Run).
//
// The k largest: the pass also keeps the maximum of every segment (a few
// consecutive vectors of one thread) in shared memory.  The k-th largest of
// the 256 threads' maxima is at most the k-th largest logit, and few logits
// reach it (a little over k for a row without order): only segments whose
// maximum reaches it are read again (L2) and their logits at or above it
// become candidates, ranked by counting.  Rows with too many candidates
// (thousands of equal logits, as in a masked vocabulary) find the k-th largest
// value itself by bisection over the 16-bit values, then the lowest ids among
// its equals by a scan in id order.  That reads the row up to eight times more, a
// logit a lane: a row of 151936 with fewer than k numbers left takes 1094 us where
// the rest is -inf and 219 where it is -1e9, 256 such rows 1306 and 294; with 200
// left, or half of the vocabulary, a row costs what it costs unmasked.
//
// What bounds it is the instructions: 12.9 a logit in all (bi_logprobs 6.9), of
// which the exponential, its sum in bi_logprobs' order and T take 5, and moving
// the maximum (in most vectors of a row's first half some lane's does) 2.  1024
// rows of 151936 logits, k = 20: 71 us, 4.4 TB/s, 0.65 of the copy rate
// (bi_logprobs, without entropy and alternatives, 50 us); one row 18 us.
#include <cuda_bf16.h>

#include <cmath>

#include "bi_internal.h"
#include "bi_ptx.cuh"
#include "logprobs.cuh"

namespace {

using bi_lp::kLog2e;
using bi_lp::kThreads;

// Vectors a thread loads at a time, while it folds as many before them.  1024,
// 608 rows and one of 151936 logits, k = 20 (without Run::c): 4 (four CTAs per SM) 68.8, 44.1 and
// 17.9 us; nothing loaded ahead: 4 (five CTAs) 70.2, 50.2 and 19.0, 2 (six) 83
// (1024 rows), 8 (three) 85, 57 and 17.7; 8 loaded ahead (three) 93, 63 and 20.4.
constexpr int kUnroll = 4;
constexpr int kSegs = 32;      // segments per thread, at most
constexpr int kMaxTop = 32;
constexpr int kMaxCand = 512;
constexpr int kWarps = kThreads / 32;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNear = 1024.f;  // maxima up to here: d by one fma
constexpr float kQuiet = 44.f;   // up to here: 44 log2(e) < 64, so mc is 2^-19 off at most
constexpr float kLowest = -3.3895313892515355e38f;  // bf16's lowest finite value
constexpr uint32_t kNegInf2 = 0xFF80FF80u;  // two bf16 -inf

// A bf16 value as a 16-bit number of the same order; both zeros alike, NaN
// below every number.
__device__ __forceinline__ uint32_t key_of(uint32_t bits) {
    if ((bits & 0x7FFFu) > 0x7F80u) return 0u;
    if (bits == 0x8000u) bits = 0u;
    return bits & 0x8000u ? 0xFFFFu & ~bits : bits | 0x8000u;
}

__device__ __forceinline__ float value_of(uint32_t key) {
    if (key == 0u) return __uint_as_float(0x7FFFFFFFu);
    return __uint_as_float((key & 0x8000u ? key & 0x7FFFu : 0xFFFFu & ~key) << 16);
}

// Running reduction of one thread.  m starts at the lowest finite value instead
// of -inf, so that no difference with it is undefined: s is 0 until a logit
// reaches m, and what multiplies a zero s changes no bit.
//
// d is one fma, x log2(e) - mc, and mc the rounded product m log2(e), so d is
// mc - m log2(e) too low, up to 2^-14 at |m| = 1024.  That is nothing while the
// maximum stays: every term, and S with them, has the same factor.  But a
// rescaling by 2^((m - m') log2(e)) leaves the older terms the old maximum's, and
// so does joining threads whose maxima differ.  bi_logprobs' s is like that, and
// lse no worse than its own rounding.  The entropy weighs parts of the row against
// one another by -ln p: 2047 logits of 1012 below one of 1020 had it 9e-5 off.  So
// T is moved and rescaled by the difference of these deltas as well, and c = S - s
// keeps what that makes of s.  While the maxima lie within +-44, as a model's do,
// it is left out: that is 2.6e-6 of a part at most, and the roundings of a sum of
// hundreds of terms are allowed more.  1024 rows of 151936: 69.3 us with nothing of
// this, 71.0 so, 75.5 with it at every move.
struct Run {
    float m, mc, s, c;
    float2 t;   // T, in two halves (elements 0, 2, .. and 1, 3, .. of the vectors)
    int mode;   // of the warp: 2 with some lane's |m| > kNear, 1 with some |m| > kQuiet or c, else 0
};

__device__ __forceinline__ float delta_of(float m) {
    return fabsf(m) > kQuiet && fabsf(m) <= kNear ? __fmaf_rn(-m, kLog2e, __fmul_rn(m, kLog2e)) : 0.f;
}

// (a - b) log2(e) for a <= b, by which d falls as the maximum goes from a to
// b; bounded where 2^.. is 0 anyway, so that 0 times it stays 0
__device__ __forceinline__ float moved(float a, float b) {
    return fmaxf(__fmul_rn(__fsub_rn(a, b), kLog2e), -1024.f);
}

// c and T of terms whose d moves by `by` + dd, |dd| at most 2^-13, where f = 2^by
// rescales s: theirs is 2^(by + dd) = f + f ln 2 dd (to 2^-27), which is returned.
__device__ __forceinline__ float rescale_ct(float s, float& c, float& t, float f, float by, float dd) {
    const float extra = __fmul_rn(f, __fmul_rn(kLn2, dd));
    const float g = __fadd_rn(f, extra);
    t = __fmul_rn(__fmaf_rn(__fadd_rn(by, dd), __fadd_rn(s, c), t), g);
    c = __fmaf_rn(c, g, __fmul_rn(s, extra));
    return g;
}

__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, c, d;\n\t"
        "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}

// fold_vec of logprobs.cu with T beside s: the same s, operation by operation
// (a maximum that stays multiplies s by 1, a vector without a visible logit adds
// zeros to it).  Returns the vector's maximum.  The maximum of some lane moves
// in most vectors of a row's first half; the whole warp takes that branch or
// none of it does.
//
// d is one fma for |m| <= 1024.  Past that -- logits no model gives, but a thread may
// see nothing else than a mask's -1e9 or bf16's lowest value, whose m log2(e) is
// not even finite -- it is taken from the difference, which is exact where it
// counts.
__device__ __forceinline__ float fold_vec_t(Run& r, const uint4& u) {
    const uint32_t h = max_bf16x2(max_bf16x2(u.x, u.y), max_bf16x2(u.z, u.w));
    const float vm = fmaxf(bi_lp::lo16(h), bi_lp::hi16(h));
    if (__any_sync(0xffffffffu, vm > r.m)) {
        const float m = fmaxf(r.m, vm);
        const float by = __fmul_rn(__fsub_rn(r.m, m), kLog2e);
        const float f = exp2f(by);  // bi_lp::rescale(r.m, m)
        const float b = fmaxf(by, -1024.f);  // moved(r.m, m)
        if (!__any_sync(0xffffffffu, fabsf(m) > kQuiet) && r.mode == 0) {
            r.t.x = __fmul_rn(__fmaf_rn(b, r.s, r.t.x), f);
            r.t.y = __fmul_rn(r.t.y, f);
        } else {
            const float dd = __fsub_rn(delta_of(r.m), delta_of(m));
            r.t.y = __fmul_rn(r.t.y, rescale_ct(r.s, r.c, r.t.x, f, b, dd));
            r.mode = __any_sync(0xffffffffu, fabsf(m) > kNear)                   ? 2
                     : __any_sync(0xffffffffu, fabsf(m) > kQuiet || r.c != 0.f) ? 1
                                                                                : 0;
        }
        r.s = __fmul_rn(r.s, f);
        r.m = m;
        r.mc = __fmul_rn(m, kLog2e);
    }
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    if (r.mode < 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 d = fma2(make_float2(bi_lp::lo16(w[i]), bi_lp::hi16(w[i])),
                                  make_float2(kLog2e, kLog2e), make_float2(-r.mc, -r.mc));
            const float2 p = make_float2(bi_lp::ex2_term(d.x), bi_lp::ex2_term(d.y));
            r.s = __fadd_rn(r.s, p.x);
            r.s = __fadd_rn(r.s, p.y);
            // p is 0 from d = -127 down; the bound keeps 0 * -inf (a masked logit) out
            r.t = fma2(p, make_float2(fmaxf(d.x, -127.f), fmaxf(d.y, -127.f)), r.t);
        }
    } else {
        const bool far = fabsf(r.m) > kNear;  // this lane
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float x = e & 1 ? bi_lp::hi16(w[e >> 1]) : bi_lp::lo16(w[e >> 1]);
            const float d = far ? __fmul_rn(__fsub_rn(x, r.m), kLog2e) : __fmaf_rn(x, kLog2e, -r.mc);
            const float p = bi_lp::ex2_term(d);
            r.s = __fadd_rn(r.s, p);
            r.t.x = __fmaf_rn(p, fmaxf(d, -127.f), r.t.x);
        }
    }
    return vm;
}

// A thread's part of the row, reduced: combine of logprobs.cu with c and T
// beside s.
struct Part {
    float m, s, c, t;
};

__device__ __forceinline__ void combine_t(Part& a, Part b) {
    const float M = fmaxf(a.m, b.m);
    const float f1 = bi_lp::rescale(a.m, M), f2 = bi_lp::rescale(b.m, M);
    if (fmaxf(fabsf(a.m), fabsf(b.m)) <= kQuiet && a.c == 0.f && b.c == 0.f) {
        a.t = __fadd_rn(__fmul_rn(__fmaf_rn(moved(a.m, M), a.s, a.t), f1),
                        __fmul_rn(__fmaf_rn(moved(b.m, M), b.s, b.t), f2));
    } else {
        const float delta = delta_of(M);
        rescale_ct(a.s, a.c, a.t, f1, moved(a.m, M), __fsub_rn(delta_of(a.m), delta));
        rescale_ct(b.s, b.c, b.t, f2, moved(b.m, M), __fsub_rn(delta_of(b.m), delta));
        a.t = __fadd_rn(a.t, b.t);
        a.c = __fadd_rn(a.c, b.c);
    }
    a.s = __fadd_rn(__fmul_rn(a.s, f1), __fmul_rn(b.s, f2));
    a.m = M;
}

struct TopArgs {
    const __nv_bfloat16* logits;
    int64_t ld;
    int vocab;
    const int32_t* targets;
    float* logprob_out;
    float* lse_out;
    float* entropy_out;
    int k;
    int seg_vecs;  // vectors of one thread in one segment (a multiple of kUnroll)
    int32_t* top_ids;
    float* top_logprobs;
    uint32_t* err;
};

// Sum of one int over the CTA, in every thread.
__device__ __forceinline__ int block_sum(int v, int* red) {
    v = __reduce_add_sync(0xffffffffu, v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    int n = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) n += red[w];
    return n;
}

// f(id, key) for the logits at or above `least`: of the segments whose maximum
// reaches it, one after the other, a lane per logit.
template <typename F>
__device__ __forceinline__ void each_reaching(const uint16_t* x, int vocab, int seg_vecs,
                                              const uint16_t* seg_max, uint32_t least, F f) {
    const int tid = threadIdx.x, lane = tid & 31;
    for (int sg = 0; sg * seg_vecs * kThreads * 8 < vocab; ++sg) {
        uint32_t reach = __ballot_sync(0xffffffffu, seg_max[sg * kThreads + tid] >= least);
        for (; reach; reach &= reach - 1) {
            const int owner = tid - lane + __ffs(reach) - 1;  // the thread whose segment it is
            for (int j = lane; j < 8 * seg_vecs; j += 32) {
                const int id = 8 * ((sg * seg_vecs + (j >> 3)) * kThreads + owner) + (j & 7);
                const uint32_t key = id < vocab ? key_of(x[id]) : 0u;
                if (id < vocab && key >= least) f(id, key);
            }
        }
    }
}

__global__ void __launch_bounds__(kThreads, 4) logprobs_top_kernel(const TopArgs a) {
    bi::launch_dependents();
    bi::grid_dependency_wait();  // nothing global is touched before the previous kernel ends
    __shared__ uint16_t seg_max[kSegs * kThreads];
    __shared__ unsigned long long cand[kMaxCand];  // key above, ~id below: larger is better
    __shared__ __align__(16) uint16_t thread_max[kThreads];
    __shared__ uint32_t kth_s;
    __shared__ Part red_part[kWarps];
    __shared__ int red[kWarps];
    __shared__ float lse_s;
    __shared__ int ncand;
    const int64_t row = blockIdx.x;
    const int tid = threadIdx.x;
    const int lane = tid & 31, warp = tid >> 5;
    const __nv_bfloat16* x = a.logits + row * a.ld;
    const uint4* xv = reinterpret_cast<const uint4*>(x);
    const uint16_t* xb = reinterpret_cast<const uint16_t*>(x);
    const int nvec = a.vocab / 8;

    // ---- one pass: (m, s, T) and the segments' maxima ----
    Run run = {kLowest, 0.f, 0.f, 0.f, make_float2(0.f, 0.f), 2};
    uint32_t best = 0;
    auto load = [&](uint4 (&u)[kUnroll], int v0) {
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            const int v = v0 + i * kThreads;
            u[i] = v < nvec ? __ldcs(xv + v) : make_uint4(kNegInf2, kNegInf2, kNegInf2, kNegInf2);
        }
    };
    uint4 next[kUnroll];
    load(next, tid);
    for (int sg = 0, v0 = tid; sg * a.seg_vecs * kThreads < nvec; ++sg) {
        float sm = -INFINITY;
        for (int i0 = 0; i0 < a.seg_vecs; i0 += kUnroll, v0 += kUnroll * kThreads) {
            uint4 u[kUnroll];
#pragma unroll
            for (int i = 0; i < kUnroll; ++i) u[i] = next[i];
            load(next, v0 + kUnroll * kThreads);
#pragma unroll
            for (int i = 0; i < kUnroll; ++i) sm = fmaxf(sm, fold_vec_t(run, u[i]));
        }
        const uint32_t key = key_of(__float_as_uint(sm) >> 16);
        seg_max[sg * kThreads + tid] = static_cast<uint16_t>(key);
        best = max(best, key);
    }
    thread_max[tid] = static_cast<uint16_t>(best);
    Part r = {run.m, run.s, run.c, __fadd_rn(run.t.x, run.t.y)};
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1)
        combine_t(r, Part{__shfl_xor_sync(0xffffffffu, r.m, o), __shfl_xor_sync(0xffffffffu, r.s, o),
                          __shfl_xor_sync(0xffffffffu, r.c, o), __shfl_xor_sync(0xffffffffu, r.t, o)});
    if (lane == 0) red_part[warp] = r;
    if (tid == 0) ncand = 0;
    __syncthreads();
    if (tid == 0) {
        Part c = red_part[0];
        for (int i = 1; i < kWarps; ++i) combine_t(c, red_part[i]);
        const float lse = __fadd_rn(c.m, logf(c.s));
        lse_s = lse;
        if (a.lse_out) a.lse_out[row] = lse;
        if (a.entropy_out) {
            const float S = __fadd_rn(c.s, c.c);
            const float h = __fsub_rn(logf(S), __fmul_rn(kLn2, __fdiv_rn(c.t, S)));
            a.entropy_out[row] = h < 0.f ? 0.f : h;  // the last bit of ln S may differ; NaN stays
        }
        if (a.targets && a.logprob_out) {
            const int t = a.targets[row];
            if (t < 0 || t >= a.vocab) {
                bi::report_error(a.err, bi::kErrBadInput | bi::kWhereDecoderOps);
                a.logprob_out[row] = NAN;
            } else {
                a.logprob_out[row] = __fsub_rn(__bfloat162float(x[t]), lse);
            }
        }
    }
    if (warp == 1) {
        // the k-th largest of the threads' maxima: the largest key that k of them
        // reach, bit by bit (8 keys a lane)
        const uint4 t8 = reinterpret_cast<const uint4*>(thread_max)[lane];
        const uint32_t w[4] = {t8.x, t8.y, t8.z, t8.w};
        uint32_t kth = 0;
#pragma unroll 1
        for (uint32_t bit = 0x8000u; bit; bit >>= 1) {
            const uint32_t mid = kth | bit;
            int n = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) n += ((w[i] & 0xFFFFu) >= mid) + ((w[i] >> 16) >= mid);
            if (__reduce_add_sync(0xffffffffu, n) >= a.k) kth = mid;
        }
        if (lane == 0) kth_s = kth;
    }
    __syncthreads();

    // a maximum of -inf may be that of a thread without logits, or with NaN only:
    // then every logit is a candidate
    const uint32_t thr = kth_s <= 0x007Fu ? 0u : kth_s;

    // ---- candidates: every logit at or above it ----
    each_reaching(xb, a.vocab, a.seg_vecs, seg_max, thr, [&](int id, uint32_t key) {
        const int at = atomicAdd(&ncand, 1);
        if (at < kMaxCand)
            cand[at] = (static_cast<unsigned long long>(key) << 32) | (0xFFFFFFFFu - static_cast<uint32_t>(id));
    });
    __syncthreads();
    int n = ncand;
    if (n > kMaxCand) {
        // the k-th largest value: the largest key that k logits reach
        uint32_t lo = thr, hi = 0x10000u;  // reached by k and more; by fewer
        while (hi - lo > 1) {
            const uint32_t mid = (lo + hi) / 2;
            int mine = 0;
            each_reaching(xb, a.vocab, a.seg_vecs, seg_max, mid, [&](int, uint32_t) { ++mine; });
            if (block_sum(mine, red) >= a.k) lo = mid;
            else hi = mid;
        }
        __syncthreads();
        if (tid == 0) ncand = 0;
        __syncthreads();
        // fewer than k lie above it ...
        each_reaching(xb, a.vocab, a.seg_vecs, seg_max, lo + 1, [&](int id, uint32_t key) {
            cand[atomicAdd(&ncand, 1)] =
                (static_cast<unsigned long long>(key) << 32) | (0xFFFFFFFFu - static_cast<uint32_t>(id));
        });
        __syncthreads();
        n = ncand;
        // ... and the lowest ids among its equals fill the rest
        for (int v0 = 0; v0 < nvec && n < a.k; v0 += kThreads) {
            const int v = v0 + tid;
            const bool may = v < nvec && seg_max[(v0 / kThreads / a.seg_vecs) * kThreads + tid] >= lo;
            if (!__syncthreads_or(may)) continue;
            uint32_t eq = 0;
            if (may) {
                const uint4 u = xv[v];
                const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    eq |= (key_of((w[e >> 1] >> (16 * (e & 1))) & 0xFFFFu) == lo ? 1u : 0u) << e;
            }
            const int mine = __popc(eq);
            int before = mine;  // inclusive prefix over the warp
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, before, o);
                if (lane >= o) before += y;
            }
            if (lane == 31) red[warp] = before;
            __syncthreads();
            int at = n + before - mine, total = 0;
            for (int w = 0; w < kWarps; ++w) {
                if (w < warp) at += red[w];
                total += red[w];
            }
            for (uint32_t left = eq; left && at < a.k; left &= left - 1, ++at)
                cand[at] = (static_cast<unsigned long long>(lo) << 32) |
                           (0xFFFFFFFFu - static_cast<uint32_t>(8 * v + __ffs(left) - 1));
            n = min(a.k, n + total);
            __syncthreads();  // red is written again
        }
        __syncthreads();
    }

    // ---- rank the candidates: no two compare equal ----
    const float lse = lse_s;
    for (int i = tid; i < n; i += kThreads) {
        const unsigned long long c = cand[i];
        int rank = 0;
        for (int j = 0; j < n; ++j) rank += cand[j] > c;
        if (rank < a.k) {
            a.top_ids[row * a.k + rank] = static_cast<int32_t>(0xFFFFFFFFu - static_cast<uint32_t>(c));
            a.top_logprobs[row * a.k + rank] = __fsub_rn(value_of(static_cast<uint32_t>(c >> 32)), lse);
        }
    }
}

bool misaligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; }

}  // namespace

extern "C" bi_status bi_logprobs_top(const void* logits, int64_t rows, int32_t vocab, int64_t ld,
                                     const int32_t* targets, float* logprob_out, float* lse_out,
                                     float* entropy_out, int32_t k, int32_t* top_ids,
                                     float* top_logprobs, cudaStream_t stream) {
    if (rows < 0 || rows > 0x7fffffffLL || k < 1) return BI_ERR_INVALID_ARG;
    if (vocab < 8 || (vocab & 7) || vocab > (1 << 30) || k > kMaxTop || k > vocab)
        return BI_ERR_UNSUPPORTED_SHAPE;
    if (ld < vocab) return BI_ERR_INVALID_ARG;
    if (ld & 7) return BI_ERR_MISALIGNED;
    if (rows == 0) return BI_OK;
    if (!logits || !top_ids || !top_logprobs || (targets != nullptr) != (logprob_out != nullptr))
        return BI_ERR_INVALID_ARG;
    if (!bi::aligned16(logits) || misaligned4(targets) || misaligned4(logprob_out) ||
        misaligned4(lse_out) || misaligned4(entropy_out) || misaligned4(top_ids) ||
        misaligned4(top_logprobs))
        return BI_ERR_MISALIGNED;
    const int64_t per_thread = (vocab / 8 + kThreads - 1) / kThreads;
    TopArgs a;
    a.logits = static_cast<const __nv_bfloat16*>(logits);
    a.ld = ld;
    a.vocab = vocab;
    a.targets = targets;
    a.logprob_out = logprob_out;
    a.lse_out = lse_out;
    a.entropy_out = entropy_out;
    a.k = k;
    a.seg_vecs = static_cast<int>(kUnroll * ((per_thread + kUnroll * kSegs - 1) / (kUnroll * kSegs)));
    a.top_ids = top_ids;
    a.top_logprobs = top_logprobs;
    a.err = bi::device_error_word();
    return bi::launch_pdl(logprobs_top_kernel, dim3(static_cast<unsigned>(rows)), dim3(kThreads), 0,
                          stream, a) == cudaSuccess
               ? BI_OK
               : BI_ERR_CUDA;
}
