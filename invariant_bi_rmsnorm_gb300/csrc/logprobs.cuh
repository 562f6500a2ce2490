// The elementary steps of a logits row's softmax denominator, shared by
// bi_logprobs and bi_logprobs_top, which reduce in the same order (logprobs.cu).
#pragma once
#include <cmath>
#include <cstdint>

#include "bi_ptx.cuh"

namespace bi_lp {

constexpr int kThreads = 256;

__device__ __forceinline__ float lo16(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float hi16(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

constexpr float kLog2e = 1.4426950408889634f;

// exp(a - b) for a <= b, as 2^((a - b) c); 0 when a is -inf
__device__ __forceinline__ float rescale(float a, float b) {
    return exp2f(__fmul_rn(__fsub_rn(a, b), kLog2e));
}

// 2^x as one ex2.approx.ftz.f32 (bi::ex2_approx; subnormal results flushed
// to zero) for the per-element terms: exp2f() takes about three more
// instructions, and the kernel is issue-bound as much as it is HBM-bound.  A
// flushed term is below 2^-126.  The vector that sets the running maximum also
// adds that maximum's own term (about 1), so by the end of every vector the
// sum is near 1 or more, and terms that small round away: the row's (m, s) is
// unchanged.
__device__ __forceinline__ float ex2_term(float x) { return bi::ex2_approx(x); }

}  // namespace bi_lp
