// bi_gemm_fp8, bi_gemm_fp8_swiglu: y = x . W^T of two 8-bit matrices (fp8.cuh)
// on tcgen05 tensor cores, the scales applied by the MMA itself.
//
// Arithmetic, the same for every M ("Defeating Nondeterminism in LLM Inference:
// The Core Role of Batch Invariance", section "2. Batch-Invariant Matrix
// Multiplication": the reduction order must not follow the batch size).  K is cut
// into at most 8 parts of whole runs of 512 values, by K alone (parts_of).  A
// part's sum is one fp32 tensor-memory accumulator: its blocks of 128 ascending,
// each as four MMAs of depth 32 whose products carry the two scales (powers of
// two, so scaling rounds nothing).  The parts' sums are then added in ascending
// order in fp32.  The page warns against split-K because a split that follows the
// batch changes the order; this one is part of the definition, as the attention's
// 256-token chunks are, so a call may compute the parts on one SM after another
// or on several at once:
//   many rows   gemm_fp8_pair_kernel: 256 x 256 tiles on CTA pairs, a part's
//               accumulator drained into registers while the next part runs;
//   few rows    gemm_fp8_parts_kernel: a cluster of CTAs, one part each, whose sums
//               meet through distributed shared memory.  The weight is what such
//               a call has to read, and the parts are what spreads it over all SMs.
// Both give an output the same bits: the same MMA depth, kind and order, with the
// operands' roles swapped in the second (tests compare them, adversarial inputs
// included).
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>

#include "bi_internal.h"
#include "bi_ptx.cuh"
#include "fp8.cuh"

namespace {

constexpr int BK = bi_fp8::kBlock;          // bytes and values per k-block
constexpr int kTile = bi_fp8::kTileBytes;   // scales of 128 rows x 4 k-blocks

// K in parts of `blocks` k-blocks each (the last may be shorter): 1024 values at
// least, and 8 parts at most.
struct Parts {
    int count, blocks;
};
inline Parts parts_of(int32_t K) {
    const int spans = bi_fp8::spans_of(K);
    const int per = std::max(2, (spans + 7) / 8);
    return {(spans + per - 1) / per, 4 * per};
}

// Instruction descriptor, kind::mxf8f6f4 with block scales: A and B e4m3 (bits
// 7-9, 10-12 = 0), both K-major (bits 15, 16 = 0), N >> 3 at bits 17-22, scales
// E8M0 (bit 23 = 1), M >> 4 at bits 24-28; the byte of a scale word at bits 4-5
// for B and 29-30 for A.
__host__ __device__ constexpr uint32_t mx_idesc(int M, int N) {
    return (static_cast<uint32_t>(N >> 3) << 17) | (1u << 23) | (static_cast<uint32_t>(M >> 4) << 24);
}
__device__ __forceinline__ uint32_t with_byte(uint32_t idesc, int byte) {
    return idesc | (static_cast<uint32_t>(byte) << 4) | (static_cast<uint32_t>(byte) << 29);
}

// K-major rows of 128 bytes, 128-byte swizzle
__device__ __forceinline__ uint64_t operand_desc(uint32_t saddr) {
    return bi::sw128_desc_lbo_sbo(saddr, 16, 1024);
}
// a scale tile: 32 rows of 16 bytes, no swizzle, 8-row groups 128 bytes apart
__device__ __forceinline__ uint64_t scale_desc(uint32_t saddr) {
    return bi::plain_desc_lbo_sbo(saddr, 0, 128);
}

struct Out {
    void* y;          // bf16 [M][ld], or e4m3 [M][ld] with scales
    int64_t ld;
    uint8_t* scales;  // of an 8-bit output
    int spans;
};

// 8 fp32 values as bf16
__device__ __forceinline__ uint4 pack8(const float* f) {
    return make_uint4(bi::pack_bf16x2(f[0], f[1]), bi::pack_bf16x2(f[2], f[3]),
                      bi::pack_bf16x2(f[4], f[5]), bi::pack_bf16x2(f[6], f[7]));
}

// ---------------------------------------------------------- many rows ----
namespace pair {
constexpr int BMP = 256;  // tile rows of the pair; 128 per CTA
constexpr int BN = 256;
constexpr int kStages = 5;
constexpr int kABytes = 128 * BK;
constexpr int kStageBytes = 2 * kABytes;  // 128 rows of x, 2 x 64 rows of W
constexpr int kScaleBytes = 3 * kTile;    // 128 rows of x, 256 rows of W
constexpr int kEpiWarps = 8;
constexpr int kThreads = 128 + 32 * kEpiWarps;
// Registers a thread: 168 at launch (three warps share a sub-partition's 16384).  The
// epilogue holds 128 sums and loads 64 columns at once; the other four warps give
// theirs up for that.
constexpr int kFewRegs = 56, kManyRegs = 224;
static_assert(128 * kFewRegs + 32 * kEpiWarps * kManyRegs <= kThreads * 168, "registers");
// Tensor memory: three accumulators of 128 columns, and 8 places of 16 columns
// for scales.  The tile's two column halves are accumulators of their own, taken
// in turn out of three, so that a half's MMAs of the next part need not wait for
// the other half to be drained; two accumulators of 256 columns would leave no
// room for the scales.
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kScaleCol = 384;
constexpr int kOutBytes = 32 * 64;  // a warp's 32 rows x 32 bf16 columns on their way out
constexpr int kOutBufs = 3;          // of them in turn
constexpr int kOutOffset = (kStages * (kStageBytes + kScaleBytes) + 1023) / 1024 * 1024;
constexpr int kSmemBytes = kOutOffset + kEpiWarps * kOutBufs * kOutBytes + 1024 + 256;
constexpr uint32_t kIdesc = mx_idesc(BMP, 128);
}  // namespace pair

// Tile order, as in bi_gemm: groups of M-tiles whose x stays in L2.
__device__ __forceinline__ void tile_coords(int tile, int num_m, int num_n, int group_m, int& mb,
                                            int& nb) {
    const int per_group = group_m * num_n;
    const int g = tile / per_group;
    const int r = tile - g * per_group;
    const int gm = min(group_m, num_m - g * group_m);
    mb = g * group_m + r % gm;
    nb = r / gm;
}

template <bool kSwiGLU>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(pair::kThreads, 1)
    gemm_fp8_pair_kernel(const __grid_constant__ CUtensorMap tmap_x,
                         const __grid_constant__ CUtensorMap tmap_w,
                         const __grid_constant__ CUtensorMap tmap_xs,
                         const __grid_constant__ CUtensorMap tmap_ws,
                         const __grid_constant__ CUtensorMap tmap_y, Out out, int M, int N, int K,
                         int part_blocks, int group_m, uint32_t* err) {
    constexpr int kStages = pair::kStages, kABytes = pair::kABytes, kStageBytes = pair::kStageBytes;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t* smem_scales = smem + kStages * kStageBytes;
    uint8_t* smem_out = smem + pair::kOutOffset;
    uint64_t* full = reinterpret_cast<uint64_t*>(smem_out + pair::kEpiWarps * pair::kOutBufs *
                                                                pair::kOutBytes);
    uint64_t* empty = full + kStages;
    uint64_t* tfull = empty + kStages;
    uint64_t* tempty = tfull + 3;
    uint64_t* drain = tempty + 3;  // MMA completion after a timeout
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    __shared__ int s_timeout;   // a role of this CTA gave up on a wait
    __shared__ int s_issued;    // k-block loads the producer issued
    __shared__ int s_consumed;  // k-block loads the MMA thread saw land
    __shared__ uint32_t s_amax[2][2][128];  // SwiGLU: a row's maximum over either half of a block

    const uint32_t rank = bi::cluster_ctarank();
    const bool leader = rank == 0;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
    const int lane = threadIdx.x & 31;
    const int num_m = (M + pair::BMP - 1) / pair::BMP;
    const int num_n = (N + pair::BN - 1) / pair::BN;
    const int num_tiles = num_m * num_n;
    const int num_kb = (K + BK - 1) / BK;
    const int spans = (num_kb + 3) >> 2;
    const int pair_id = blockIdx.x >> 1;
    const int npairs = gridDim.x >> 1;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            bi::mbar_init(&full[i], 1);   // the leader's arrive (+ both CTAs' bytes)
            bi::mbar_init(&empty[i], 1);  // one pair-MMA commit
        }
        for (int i = 0; i < 3; ++i) {
            bi::mbar_init(&tfull[i], 1);
            bi::mbar_init(&tempty[i], 2 * pair::kEpiWarps);  // both CTAs' (leader's copy used)
        }
        bi::mbar_init(drain, 1);
        bi::fence_mbar_init();
        s_timeout = 0;
        s_issued = 0;
        s_consumed = 0;
        bi::tma_prefetch_desc(&tmap_x);
        bi::tma_prefetch_desc(&tmap_w);
        bi::tma_prefetch_desc(&tmap_xs);
        bi::tma_prefetch_desc(&tmap_ws);
    }
    if (warp == 1) {
        bi::tmem_alloc_pair(tmem_slot, pair::kTmemCols);
        bi::tmem_relinquish_pair();
    }
    bi::tc_fence_before();
    bi::cluster_sync();  // both CTAs' barriers exist before either signals the other
    bi::tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    bi::launch_dependents();
    bi::grid_dependency_wait();  // nothing global is touched before the previous kernel ends

    if (warp < 4) {
        bi::fewer_registers<pair::kFewRegs>();
    if (warp == 0) {  // the whole warp runs the loop, one lane issues
        const uint32_t bar0 = bi::mapa_shared(bi::smem_u32(full), 0);  // the leader's
        int stage = 0;
        uint32_t phase = 0;
        int issued = 0;
        bool ok = true;
        for (int tile = pair_id; tile < num_tiles && ok; tile += npairs) {
            int mb, nb;
            tile_coords(tile, num_m, num_n, group_m, mb, nb);
            const int m_tile = 2 * mb + static_cast<int>(rank);  // of 128 rows
            const int w_row = nb * pair::BN + static_cast<int>(rank) * 64;
            for (int kb = 0; kb < num_kb; ++kb) {
                if (!__all_sync(0xffffffffu, bi::mbar_wait(&empty[stage], phase ^ 1))) {
                    ok = false;
                    break;
                }
                const bool scales = (kb & 3) == 0;  // a tile of them serves four k-blocks
                uint8_t* sa = smem + stage * kStageBytes;
                const uint32_t bar = bar0 + 8 * stage;
                if (bi::elect_one()) {
                    if (leader)
                        bi::mbar_arrive_expect_tx(
                            &full[stage], 2 * (kStageBytes + (scales ? pair::kScaleBytes : 0)));
                    bi::tma_load_2d_pair(sa, &tmap_x, bar, kb * BK, m_tile * 128);
                    // a half's 128 W rows come half from each CTA (its share of B)
                    bi::tma_load_2d_pair(sa + kABytes, &tmap_w, bar, kb * BK, w_row);
                    bi::tma_load_2d_pair(sa + kABytes + 64 * BK, &tmap_w, bar, kb * BK, w_row + 128);
                    if (scales) {
                        uint8_t* sf = smem_scales + stage * pair::kScaleBytes;
                        bi::tma_load_2d_pair(sf, &tmap_xs, bar, 0, m_tile * spans + (kb >> 2));
                        bi::tma_load_2d_pair(sf + kTile, &tmap_ws, bar, 0,
                                             2 * nb * spans + (kb >> 2));
                        bi::tma_load_2d_pair(sf + 2 * kTile, &tmap_ws, bar, 0,
                                             (2 * nb + 1) * spans + (kb >> 2));
                    }
                }
                __syncwarp();
                ++issued;
                if (++stage == kStages) {
                    stage = 0;
                    phase ^= 1;
                }
            }
        }
        if (lane == 0) {
            s_issued = issued;
            if (!ok) {
                bi::report_error(err, bi::kErrTimeout | bi::kWhereGemmFp8);
                s_timeout = 1;
            }
        }
    } else if (warp == 1) {
        if (leader) {  // the whole warp runs the loop, one lane issues
            const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_base, 0);
            const uint32_t ring = bi::smem_u32(smem);
            int stage = 0;
            uint32_t phase = 0;
            int acc = 0;             // accumulators in turn, 0 .. 2
            uint32_t acc_phase = 0;  // flips when the turn comes round
            int sf = 0;              // scale place, 0 .. 7
            int consumed = 0;
            bool ok = true;
            for (int tile = pair_id; tile < num_tiles && ok; tile += npairs) {
                uint32_t sfa = 0;
                int d[2] = {0, 0};
                int left = 0;  // k-blocks of the part still to come
                for (int kb = 0; kb < num_kb; ++kb) {
                    const bool first = left == 0;
                    if (first) left = min(part_blocks, num_kb - kb);
                    --left;
                    if (!__all_sync(0xffffffffu, bi::mbar_wait(&full[stage], phase))) {
                        ok = false;
                        break;
                    }
                    ++consumed;
                    bi::tc_fence_after();
                    const uint32_t sa = ring + stage * kStageBytes;
                    if ((kb & 3) == 0) {
                        // The place was last read by MMAs of 8 tiles of scales ago.
                        // They are done: this stage's load waited for the MMAs of
                        // kStages < 8 k-blocks ago, and tiles are a k-block apart at least.
                        sfa = tmem + pair::kScaleCol + 16 * sf;
                        sf = (sf + 1) & 7;
                        const uint64_t s = scale_desc(ring + kStages * kStageBytes +
                                                      stage * pair::kScaleBytes);
                        if (bi::elect_one()) {
                            bi::tc_cp_scales_pair(sfa, s);
                            bi::tc_cp_scales_pair(sfa + 4, s + (kTile >> 4));
                            bi::tc_cp_scales_pair(sfa + 8, s + (2 * kTile >> 4));
                        }
                        __syncwarp();
                    }
                    const uint32_t idesc = with_byte(pair::kIdesc, kb & 3);
                    const uint64_t da = operand_desc(sa), db = operand_desc(sa + kABytes);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if (first) {
                            if (!__all_sync(0xffffffffu, bi::mbar_wait(&tempty[acc], acc_phase ^ 1))) {
                                ok = false;
                                break;
                            }
                            bi::tc_fence_after();
                            d[h] = acc;
                            if (++acc == 3) {
                                acc = 0;
                                acc_phase ^= 1;
                            }
                        }
                        if (bi::elect_one()) {
#pragma unroll
                            for (int k = 0; k < BK / 32; ++k)  // 32 bytes of K a step
                                bi::tc_mma_mxf8_pair(tmem + 128 * d[h], da + 2 * k,
                                                     db + (h * 64 * BK >> 4) + 2 * k, idesc, sfa,
                                                     sfa + 4 + 4 * h, (!first || k != 0) ? 1u : 0u);
                            if (left == 0)  // the half's part is complete in both CTAs
                                bi::tc_commit_pair_multicast(&tfull[d[h]], 0x3);
                            if (h == 1)  // the stage is free in both CTAs
                                bi::tc_commit_pair_multicast(&empty[stage], 0x3);
                        }
                        __syncwarp();
                    }
                    if (!ok) break;
                    if (++stage == kStages) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
            }
            if (bi::elect_one()) {
                s_consumed = consumed;
                if (!ok) {
                    bi::report_error(err, bi::kErrTimeout | bi::kWhereGemmFp8);
                    s_timeout = 1;
                }
                if (s_timeout && consumed > 0) {
                    // what was issued may still read shared memory and write TMEM: a
                    // bounded wait for it before both are freed
                    bi::tc_commit_pair_multicast(drain, 0x1);
                    bi::mbar_wait_for(drain, 0, bi::kDrainNs);
                }
            }
            __syncwarp();
        }
    }
    } else {
        bi::more_registers<pair::kManyRegs>();
        // epilogue warps 4..11: lane quarter warp % 4 of this CTA's 128 rows, and
        // 64 of either half's 128 columns
        const int quarter = warp & 3;
        const int c = (warp - 4) >> 2;
        const int num_parts = (num_kb + part_blocks - 1) / part_blocks;
        int acc = 0;
        uint32_t acc_phase = 0;
        int turn = 0, out_buf = 0;
        bool ok = true;  // of the whole warp; a warp that gave up still meets its partner
        const uint32_t taddr0 =
            tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + 64 * c;
        for (int tile = pair_id; tile < num_tiles; tile += npairs, turn ^= 1) {
            float sum[2][64];  // from -0 on: -0 + x is x, whatever its sign
#pragma unroll
            for (int i = 0; i < 64; ++i) sum[0][i] = sum[1][i] = -0.f;
#pragma unroll 1
            for (int p = 0; p < num_parts; ++p) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (ok) {
                        ok = __all_sync(0xffffffffu, bi::mbar_wait(&tfull[acc], acc_phase));
                        if (!ok && lane == 0) {
                            bi::report_error(err, bi::kErrTimeout | bi::kWhereGemmFp8);
                            s_timeout = 1;
                        }
                    }
                    if (ok) {
                        bi::tc_fence_after();
                        const uint32_t taddr = taddr0 + 128 * acc;
                        uint32_t r[2][32];
                        bi::tmem_ld_32x32b_x32(taddr, r[0]);
                        bi::tmem_ld_32x32b_x32(taddr + 32, r[1]);
                        bi::tmem_ld_wait();
                        bi::tc_fence_before();
                        __syncwarp();
                        if (lane == 0)
                            bi::mbar_arrive_cluster_relaxed(bi::mapa_shared(bi::smem_u32(&tempty[acc]), 0));
#pragma unroll
                        for (int i = 0; i < 64; ++i)
                            sum[h][i] = __fadd_rn(sum[h][i], __uint_as_float(r[i >> 5][i & 31]));
                    }
                    if (++acc == 3) {
                        acc = 0;
                        acc_phase ^= 1;
                    }
                }
            }
            int mb, nb;  // not before the sums are there: every register counts in that loop
            tile_coords(tile, num_m, num_n, group_m, mb, nb);
            const int in_tile = quarter * 32 + lane;
            const int row = mb * pair::BMP + static_cast<int>(rank) * 128 + in_tile;
            if constexpr (!kSwiGLU) {
                // 32 rows x 32 columns at a time through shared memory (64-byte rows,
                // swizzled: no bank conflicts) and out by TMA, which clips them to y.  A
                // lane storing its own row's 16 bytes at a time costs a cycle of the
                // store path for each of a warp's 32 rows: 6900 cycles a tile.
                if (!ok) continue;
                const int row0 = row - lane;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int col = nb * pair::BN + 128 * (q >> 1) + 64 * c + 32 * (q & 1);
                    if (row0 >= M || col >= N) continue;  // the whole warp
                    uint8_t* buf = smem_out + ((warp - 4) * pair::kOutBufs + out_buf) * pair::kOutBytes;
                    if (++out_buf == pair::kOutBufs) out_buf = 0;
                    if (bi::elect_one()) bi::tma_store_wait_read<pair::kOutBufs - 1>();
                    __syncwarp();
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        *reinterpret_cast<uint4*>(buf + lane * 64 + ((v ^ ((lane >> 1) & 3)) << 4)) =
                            pack8(&sum[q >> 1][32 * (q & 1) + 8 * v]);
                    bi::fence_proxy_async_smem();
                    __syncwarp();
                    if (bi::elect_one()) bi::tma_store_2d(&tmap_y, buf, col, row0);
                }
            } else {
                // 16 accumulator columns are 8 gate values and the 8 matching up values;
                // the tile's 256 columns are one block of 128 outputs of a row
                uint32_t top = 0;  // outputs take the places of the sums they are made of
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        // past F there are no W rows, and what stands for their scales may
                        // be NaN
                        const bool in = 2 * (nb * 128 + 64 * h + 32 * c + 8 * g) < N;
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const float v = bi::swiglu(sum[h][16 * g + e], sum[h][16 * g + 8 + e]);
                            sum[h][8 * g + e] = v;
                            if (in) top = max(top, __float_as_uint(v) & 0x7fffffffu);
                        }
                    }
                s_amax[turn][c][in_tile] = top;
                // the two warps that share these rows (one barrier a lane quarter); the
                // next tile writes the other buffer, and the one after it is behind the
                // next meeting
                asm volatile("bar.sync %0, 64;" ::"r"(1 + quarter) : "memory");
                top = max(top, s_amax[turn][c ^ 1][in_tile]);
                if (!ok || row >= M) continue;
                const uint32_t byte = bi_fp8::scale_byte(top);
                const float inv = bi_fp8::inverse_scale(byte);
                uint8_t* hr = static_cast<uint8_t*>(out.y) + static_cast<int64_t>(row) * out.ld;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int col = nb * 128 + 64 * h + 32 * c;
#pragma unroll
                    for (int v = 0; v < 2; ++v) {
                        uint32_t o[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float* f = &sum[h][16 * v + 4 * e];
                            o[e] = bi_fp8::codes4(__fmul_rn(f[0], inv), __fmul_rn(f[1], inv),
                                                  __fmul_rn(f[2], inv), __fmul_rn(f[3], inv));
                        }
                        if (2 * (col + 16 * v) < N)  // whole groups of 16 outputs
                            *reinterpret_cast<uint4*>(hr + col + 16 * v) = make_uint4(o[0], o[1], o[2], o[3]);
                    }
                }
                if (c == 0)
                    out.scales[bi_fp8::scale_word(row, nb >> 2, out.spans) + (nb & 3)] =
                        static_cast<uint8_t>(byte);
            }
        }
    }

    if (!kSwiGLU && warp >= 4 && bi::elect_one()) bi::tma_store_wait_all();
    __syncthreads();
    if (s_timeout && leader && threadIdx.x == 0) {
        // loads issued but never seen to land (at most one ring's worth): a bounded
        // wait for each, on barriers that count both CTAs' bytes
        for (int i = s_consumed; i < s_issued; ++i)
            bi::mbar_wait_for(&full[i % kStages], (i / kStages) & 1, bi::kDrainNs);
    }
    bi::tc_fence_before();
    bi::cluster_sync();  // both CTAs past their last TMEM access and remote arrive
    if (warp == 1) {
        bi::tc_fence_after();
        bi::tmem_dealloc_pair(tmem_base, pair::kTmemCols);
    }
}

// ----------------------------------------------------------- few rows ----
// NT: rows of x per CTA (the MMA's N); WT: tiles of 128 W rows per CTA (the MMA's
// M): one, or two where a block of 128 SwiGLU outputs needs 256 W rows; STAGES: k-blocks
// in flight per CTA.
template <int NT, int WT, int STAGES>
struct PartsShape {
    static constexpr int kWBytes = WT * 128 * BK;
    static constexpr int kStageBytes = kWBytes + NT * BK;
    static constexpr int kScaleBytes = (WT + 1) * kTile;
    static constexpr int kStages = STAGES;
    static constexpr int kUsedBytes = kStages * (kStageBytes + kScaleBytes) + 1024 + 256;
    static constexpr int kPartialBytes = WT * 128 * NT * 4;
    static_assert(kPartialBytes <= kStages * kStageBytes, "partials lie in the ring");
    // Tensor memory: the sums, then places for scales.  A place is used again kPlaces
    // tiles of scales (4 k-blocks each) later, and a stage's load has waited for the MMAs
    // of kStages k-blocks ago.
    static constexpr uint32_t kScaleCol = WT * NT;
    static constexpr uint32_t kPlaceCols = 4 * (WT + 1);
    static constexpr uint32_t kPlaces = kStages > 5 ? 4 : 2;
    static_assert(4 * kPlaces >= kStages + 3, "scale places");
    static constexpr uint32_t kCols = kScaleCol + kPlaces * kPlaceCols;
    static constexpr uint32_t kTmemCols =
        kCols <= 32 ? 32 : kCols <= 64 ? 64 : kCols <= 128 ? 128 : kCols <= 256 ? 256 : 512;
    // An SM must not hold more of this file's CTAs than its 512 columns of tensor
    // memory serve: were a cluster's CTA to wait for columns that another cluster holds,
    // the two could wait for each other.  So a CTA takes 1/543 of an SM's shared memory
    // for each of its columns at least, and the next multiple of 32 above 512 is 544.
    static constexpr int kShareBytes = (kTmemCols * (228 * 1024) + 542) / 543 - 1024;
    static constexpr int kSmemBytes = kUsedBytes > kShareBytes ? kUsedBytes : kShareBytes;
};

template <int NT, bool kSwiGLU, int STAGES>
__global__ void __launch_bounds__(192)
    gemm_fp8_parts_kernel(const __grid_constant__ CUtensorMap tmap_x,
                          const __grid_constant__ CUtensorMap tmap_w,
                          const __grid_constant__ CUtensorMap tmap_xs,
                          const __grid_constant__ CUtensorMap tmap_ws, Out out, int M, int N, int K,
                          int part_blocks, bool prefetch, uint32_t* err) {
    constexpr int WT = kSwiGLU ? 2 : 1;
    using S = PartsShape<NT, WT, STAGES>;
    constexpr int kStages = S::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t* smem_scales = smem + kStages * S::kStageBytes;
    uint64_t* full = reinterpret_cast<uint64_t*>(smem_scales + kStages * S::kScaleBytes);
    uint64_t* empty = full + kStages;
    uint64_t* tfull = empty + kStages;
    uint64_t* drain = tfull + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    float* partial = reinterpret_cast<float*>(smem);  // [NT][WT * 128], over the ring
    __shared__ int s_timeout, s_issued, s_consumed;

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
    const int lane = threadIdx.x & 31;
    const int rank = blockIdx.x;  // the cluster is the grid's x: one CTA a part
    const int nparts = gridDim.x;
    const int m0 = blockIdx.y * NT;
    const int n0 = blockIdx.z * (WT * 128);
    const int num_kb = (K + BK - 1) / BK;
    const int spans = (num_kb + 3) >> 2;
    const int kb0 = rank * part_blocks;
    const int nkb = min(part_blocks, num_kb - kb0);

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            bi::mbar_init(&full[i], 1);
            bi::mbar_init(&empty[i], 1);
        }
        bi::mbar_init(tfull, 1);
        bi::mbar_init(drain, 1);
        bi::fence_mbar_init();
        s_timeout = 0;
        s_issued = 0;
        s_consumed = 0;
        bi::tma_prefetch_desc(&tmap_x);
        bi::tma_prefetch_desc(&tmap_w);
        bi::tma_prefetch_desc(&tmap_xs);
        bi::tma_prefetch_desc(&tmap_ws);
    }
    if (warp == 1) {
        bi::tmem_alloc(tmem_slot, S::kTmemCols);
        bi::tmem_relinquish();
    }
    if (warp == 0) {
        // the weight may start on its way to L2 while the previous kernel, which as a
        // rule makes x, still runs (N = K = 4096, one row, after another such call: 6.3 ->
        // 5.9 us); no use to CTAs that start when others end
        if (prefetch && bi::elect_one())
            for (int i = 0; i < nkb; ++i)
                for (int t = 0; t < WT; ++t)
                    bi::tma_prefetch_2d(&tmap_w, (kb0 + i) * BK, n0 + 128 * t);
        __syncwarp();
    }
    bi::tc_fence_before();
    __syncthreads();
    bi::tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    bi::launch_dependents();
    bi::grid_dependency_wait();  // nothing global is read or written before the previous kernel ends

    if (warp == 0) {  // the whole warp runs the loop, one lane issues
        int stage = 0;
        uint32_t phase = 0;
        int issued = 0;
        bool ok = true;
        for (; issued < nkb; ++issued) {
            if (!__all_sync(0xffffffffu, bi::mbar_wait(&empty[stage], phase ^ 1))) {
                ok = false;
                break;
            }
            const int kb = kb0 + issued;
            const bool scales = (issued & 3) == 0;  // parts start on whole spans
            uint8_t* sw = smem + stage * S::kStageBytes;
            if (bi::elect_one()) {
                bi::mbar_arrive_expect_tx(&full[stage],
                                          S::kStageBytes + (scales ? S::kScaleBytes : 0));
#pragma unroll
                for (int t = 0; t < WT; ++t)
                    bi::tma_load_2d(sw + t * 128 * BK, &tmap_w, &full[stage], kb * BK, n0 + 128 * t);
                bi::tma_load_2d(sw + S::kWBytes, &tmap_x, &full[stage], kb * BK, m0);
                if (scales) {
                    uint8_t* sf = smem_scales + stage * S::kScaleBytes;
#pragma unroll
                    for (int t = 0; t < WT; ++t)
                        bi::tma_load_2d(sf + t * kTile, &tmap_ws, &full[stage], 0,
                                        (n0 / 128 + t) * spans + (kb >> 2));
                    // NT < 128 only where one tile holds all rows, so a tile's rows start
                    // where its scales do
                    bi::tma_load_2d(sf + WT * kTile, &tmap_xs, &full[stage], 0,
                                    (m0 / 128) * spans + (kb >> 2));
                }
            }
            __syncwarp();
            if (++stage == kStages) {
                stage = 0;
                phase ^= 1;
            }
        }
        if (lane == 0) {
            s_issued = issued;
            if (!ok) {
                bi::report_error(err, bi::kErrTimeout | bi::kWhereGemmFp8);
                s_timeout = 1;
            }
        }
    } else if (warp == 1) {  // the whole warp runs the loop, one lane issues
        const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_base, 0);
        const uint32_t ring = bi::smem_u32(smem);
        uint32_t sfw = 0;
        int stage = 0;
        uint32_t phase = 0;
        int i = 0;
        bool ok = true;
        for (; i < nkb; ++i) {
            if (!__all_sync(0xffffffffu, bi::mbar_wait(&full[stage], phase))) {
                ok = false;
                break;
            }
            bi::tc_fence_after();
            const uint32_t idesc = with_byte(mx_idesc(128, NT), i & 3);
            const uint32_t sw = ring + stage * S::kStageBytes;
            const uint64_t dw = operand_desc(sw), dx = operand_desc(sw + S::kWBytes);
            const uint64_t s = scale_desc(ring + kStages * S::kStageBytes + stage * S::kScaleBytes);
            if ((i & 3) == 0) sfw = tmem + S::kScaleCol + S::kPlaceCols * ((i >> 2) % S::kPlaces);
            if (bi::elect_one()) {
                if ((i & 3) == 0) {
#pragma unroll
                    for (int t = 0; t <= WT; ++t) bi::tc_cp_scales(sfw + 4 * t, s + (t * kTile >> 4));
                }
#pragma unroll
                for (int t = 0; t < WT; ++t)
#pragma unroll
                    for (int k = 0; k < BK / 32; ++k)  // 32 bytes of K a step
                        bi::tc_mma_mxf8(tmem + t * NT, dw + (t * 128 * BK >> 4) + 2 * k, dx + 2 * k,
                                        idesc, sfw + 4 * t, sfw + 4 * WT, (i | k) != 0 ? 1u : 0u);
                bi::tc_commit(&empty[stage]);
                if (i + 1 == nkb) bi::tc_commit(tfull);
            }
            __syncwarp();
            if (++stage == kStages) {
                stage = 0;
                phase ^= 1;
            }
        }
        if (bi::elect_one()) {
            s_consumed = i;
            if (!ok) {
                bi::report_error(err, bi::kErrTimeout | bi::kWhereGemmFp8);
                s_timeout = 1;
                if (i > 0) {
                    bi::tc_commit(drain);
                    bi::mbar_wait_for(drain, 0, bi::kDrainNs);
                }
            }
        }
        __syncwarp();
    } else {
        // warps 2..5: W rows quarter * 32 + lane of each W tile, all NT rows of x
        const int quarter = warp & 3;
        const bool ok = __all_sync(0xffffffffu, bi::mbar_wait(tfull, 0));
        if (!ok && lane == 0) {
            bi::report_error(err, bi::kErrTimeout | bi::kWhereGemmFp8);
            s_timeout = 1;
        }
        bi::tc_fence_after();
        const int rows = min(NT, M - m0);
        if (ok) {
#pragma unroll
            for (int t = 0; t < WT; ++t) {
                float* to = partial + t * 128 + quarter * 32 + lane;
                for (int m = 0; m < rows; m += 16) {
                    uint32_t r[16];
                    bi::tmem_ld_32x32b_x16(
                        tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + t * NT + m, r);
                    bi::tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 16; ++e) to[(m + e) * (WT * 128)] = __uint_as_float(r[e]);
                }
            }
        }
    }
    __syncthreads();
    if (s_timeout) {
        // copies in flight first (they land in the ring), then NaN where the sums would be
        if (threadIdx.x == 0)
            for (int i = s_consumed; i < s_issued; ++i)
                bi::mbar_wait_for(&full[i % kStages], (i / kStages) & 1, bi::kDrainNs);
        __syncthreads();
        for (int i = threadIdx.x; i < NT * WT * 128; i += 192) partial[i] = __uint_as_float(0x7FC00000u);
    }
    bi::tc_fence_before();
    bi::cluster_sync();  // all parts' sums are in place
    if (warp == 1) {
        bi::tc_fence_after();
        bi::tmem_dealloc(tmem_base, S::kTmemCols);
    }

    // the parts' sums, ascending, the outputs dealt out over the cluster's CTAs
    const int rows = min(NT, M - m0);
    const uint32_t base = bi::smem_u32(partial);
    if constexpr (!kSwiGLU) {
        const int items = rows * 32;  // four outputs each
        for (int i = rank * 192 + threadIdx.x; i < items; i += nparts * 192) {
            const int m = i >> 5, n = n0 + 4 * (i & 31);
            float4 v[8];
#pragma unroll
            for (int p = 0; p < 8; ++p)
                if (p < nparts) v[p] = bi::ld_cluster_f4(bi::mapa_shared(base + 16 * i, p));
            float4 s = v[0];
#pragma unroll
            for (int p = 1; p < 8; ++p)
                if (p < nparts) {
                    s.x = __fadd_rn(s.x, v[p].x);
                    s.y = __fadd_rn(s.y, v[p].y);
                    s.z = __fadd_rn(s.z, v[p].z);
                    s.w = __fadd_rn(s.w, v[p].w);
                }
            if (n < N)
                *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(out.y) +
                                          static_cast<int64_t>(m0 + m) * out.ld + n) =
                    make_uint2(bi::pack_bf16x2(s.x, s.y), bi::pack_bf16x2(s.z, s.w));
        }
    } else {
        // a warp folds one row's 256 columns: lane l the outputs 4l .. 4l + 3 of the
        // block, whose gate and up columns lie 8 apart in a group of 16
        const int nb = blockIdx.z;
        for (int m = rank * 6 + warp; m < rows; m += nparts * 6) {
            const uint32_t at = base + 4 * (m * 256 + (lane >> 1) * 16 + (lane & 1) * 4);
            float4 v[8], w[8];
#pragma unroll
            for (int p = 0; p < 8; ++p)
                if (p < nparts) {
                    const uint32_t a = bi::mapa_shared(at, p);
                    v[p] = bi::ld_cluster_f4(a);
                    w[p] = bi::ld_cluster_f4(a + 32);
                }
            float4 g = v[0], u = w[0];
#pragma unroll
            for (int p = 1; p < 8; ++p)
                if (p < nparts) {
                    g.x = __fadd_rn(g.x, v[p].x);
                    g.y = __fadd_rn(g.y, v[p].y);
                    g.z = __fadd_rn(g.z, v[p].z);
                    g.w = __fadd_rn(g.w, v[p].w);
                    u.x = __fadd_rn(u.x, w[p].x);
                    u.y = __fadd_rn(u.y, w[p].y);
                    u.z = __fadd_rn(u.z, w[p].z);
                    u.w = __fadd_rn(u.w, w[p].w);
                }
            const float h0 = bi::swiglu(g.x, u.x), h1 = bi::swiglu(g.y, u.y);
            const float h2 = bi::swiglu(g.z, u.z), h3 = bi::swiglu(g.w, u.w);
            uint32_t top = max(max(__float_as_uint(h0) & 0x7fffffffu, __float_as_uint(h1) & 0x7fffffffu),
                               max(__float_as_uint(h2) & 0x7fffffffu, __float_as_uint(h3) & 0x7fffffffu));
            const int col = nb * 128 + 4 * lane;
            if (2 * col >= N) top = 0;  // past F: no W rows, and perhaps NaN for their scales
            top = __reduce_max_sync(0xffffffffu, top);
            const uint32_t byte = bi_fp8::scale_byte(top);
            const float inv = bi_fp8::inverse_scale(byte);
            const int64_t row = m0 + m;
            if (2 * col < N)
                *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(out.y) + row * out.ld + col) =
                    bi_fp8::codes4(__fmul_rn(h0, inv), __fmul_rn(h1, inv), __fmul_rn(h2, inv),
                                   __fmul_rn(h3, inv));
            if (lane == 0)
                out.scales[bi_fp8::scale_word(row, nb >> 2, out.spans) + (nb & 3)] =
                    static_cast<uint8_t>(byte);
        }
    }
    __syncwarp();
    bi::cluster_sync_relaxed();  // no CTA leaves while another reads its sums
}

// ------------------------------------------------------------- launches ----
struct Call {
    const void *x, *xs, *W, *Ws;
    int32_t M, N, K;  // N: rows of W
    int64_t ld_x, ld_w;
    Out out;
    cudaStream_t stream;
};

bool encode(const Call& c, uint32_t x_rows, uint32_t w_rows, CUtensorMap (&t)[4]) {
    const uint64_t spans = bi_fp8::spans_of(c.K);
    return bi::encode_byte_map_2d(&t[0], c.x, c.K, c.M, c.ld_x, x_rows) == CUDA_SUCCESS &&
           bi::encode_byte_map_2d(&t[1], c.W, c.K, c.N, c.ld_w, w_rows) == CUDA_SUCCESS &&
           bi::encode_scale_map(&t[2], c.xs, (c.M + 127) / 128 * spans) == CUDA_SUCCESS &&
           bi::encode_scale_map(&t[3], c.Ws, (c.N + 127) / 128 * spans) == CUDA_SUCCESS;
}

template <bool kSwiGLU>
bi_status launch_pair(const Call& c) {
    static std::atomic<bool> set[64] = {};
    if (!bi::allow_smem(gemm_fp8_pair_kernel<kSwiGLU>, pair::kSmemBytes, set)) return BI_ERR_CUDA;
    const int sms = bi::sm_count();
    if (sms < 2) return BI_ERR_CUDA;
    CUtensorMap t[4];
    if (!encode(c, 128, 64, t)) return BI_ERR_CUDA;
    CUtensorMap ty = t[0];  // not read where the output is 8 bits
    if (!kSwiGLU && bi::encode_out_map(&ty, c.out.y, c.N, c.M, c.out.ld * 2) != CUDA_SUCCESS)
        return BI_ERR_CUDA;
    const int num_m = (c.M + pair::BMP - 1) / pair::BMP;
    const int64_t tiles = static_cast<int64_t>(num_m) * ((c.N + pair::BN - 1) / pair::BN);
    if (tiles > 0x7fffffffLL) return BI_ERR_UNSUPPORTED_SHAPE;
    const int pairs = static_cast<int>(std::min<int64_t>(tiles, sms / 2));
    // at most about 48 MB of x per group of M-tiles, as bi_gemm
    const int64_t slab = static_cast<int64_t>(pair::BMP) * c.K;
    const int64_t budget = int64_t{48} << 20;
    int group_m = num_m;
    if (slab * num_m > budget) group_m = static_cast<int>(std::max<int64_t>(1, budget / slab));
    return bi::launch_pdl(gemm_fp8_pair_kernel<kSwiGLU>, dim3(2 * pairs), dim3(pair::kThreads),
                          pair::kSmemBytes, c.stream, t[0], t[1], t[2], t[3], ty, c.out, c.M, c.N, c.K,
                          parts_of(c.K).blocks, group_m, bi::device_error_word()) == cudaSuccess
               ? BI_OK
               : BI_ERR_CUDA;
}

template <int NT, bool kSwiGLU, int STAGES>
bi_status launch_parts(const Call& c, bool prefetch) {
    using S = PartsShape<NT, kSwiGLU ? 2 : 1, STAGES>;
    static std::atomic<bool> set[64] = {};
    if (!bi::allow_smem(gemm_fp8_parts_kernel<NT, kSwiGLU, STAGES>, S::kSmemBytes, set))
        return BI_ERR_CUDA;
    CUtensorMap t[4];
    if (!encode(c, NT, 128, t)) return BI_ERR_CUDA;
    const Parts p = parts_of(c.K);
    const int rows = kSwiGLU ? 256 : 128;
    const dim3 grid(p.count, (c.M + NT - 1) / NT, (c.N + rows - 1) / rows);
    return bi::launch_pdl_cluster(gemm_fp8_parts_kernel<NT, kSwiGLU, STAGES>, p.count, grid,
                                  dim3(192), S::kSmemBytes, c.stream, t[0], t[1], t[2], t[3], c.out,
                                  c.M, c.N, c.K, p.blocks, prefetch, bi::device_error_word()) ==
                   cudaSuccess
               ? BI_OK
               : BI_ERR_CUDA;
}

// Stages by the launch's CTAs: one, two or three CTAs an SM, the fewest that hold the
// launch at once (a CTA then has the most loads in flight), else three.
template <int NT, bool kSwiGLU, int ONE, int TWO, int THREE>
bi_status launch_parts(const Call& c) {
    const int rows = kSwiGLU ? 256 : 128;
    const int64_t ctas = static_cast<int64_t>(parts_of(c.K).count) * ((c.M + NT - 1) / NT) *
                         ((c.N + rows - 1) / rows);
    const int sms = bi::sm_count();
    if (ctas <= sms) return launch_parts<NT, kSwiGLU, ONE>(c, true);
    if (ctas <= 2 * sms) return launch_parts<NT, kSwiGLU, TWO>(c, true);
    return launch_parts<NT, kSwiGLU, THREE>(c, false);
}

// Which kernel: a schedule choice, the bits are the same.  Up to 32 rows the parts
// kernel (17 rows, K = 4096: N = 4096 6.3 us against 15, N = 24576 21.4 against 29.7).  Beyond, its
// time goes with its 128 x 128 tiles, that of the other with its waves of 256 x 256
// tiles over the CTA pairs, and the two cross at about a pair's worth of tiles a wave:
// K = 4096, N = 4096 8.6 against 15.5 us at 128 rows and 11.0 against 15.5 at 200 (64
// tiles), 18.6 against 15.7 at 300 (96); N = 24576 35.6 against 30.1 at 128 rows (192 tiles,
// two waves); K = 12288, N = 4096 25.6 against 34.1 at 200 rows, 37.1 against 34.3 at 300.
template <bool kSwiGLU>
bi_status launch_gemm(const Call& c) {
    const int sms = bi::sm_count();
    if (sms < 2) return BI_ERR_CUDA;
    const int64_t small_m = (c.M + 127) / 128, small_n = (c.N + 127) / 128;
    const int64_t large = static_cast<int64_t>((c.M + 255) / 256) * ((c.N + 255) / 256);
    const int64_t waves = (large + sms / 2 - 1) / (sms / 2);
    if ((c.M <= 32 || small_m * small_n <= waves * (sms / 2)) && small_m <= 65535 && small_n <= 65535) {
        constexpr bool g = kSwiGLU;
        if (c.M <= 16) return g ? launch_parts<16, g, 6, 3, 2>(c) : launch_parts<16, g, 8, 4, 3>(c);
        if (c.M <= 32) return g ? launch_parts<32, g, 5, 2, 2>(c) : launch_parts<32, g, 8, 4, 3>(c);
        if (c.M <= 64) return g ? launch_parts<64, g, 4, 2, 2>(c) : launch_parts<64, g, 8, 4, 4>(c);
        return g ? launch_parts<128, g, 4, 4, 4>(c) : launch_parts<128, g, 6, 3, 3>(c);
    }
    return launch_pair<kSwiGLU>(c);
}

bi_status check(const Call& c, int n_step) {
    if (c.M < 0) return BI_ERR_INVALID_ARG;
    if (c.N < n_step || c.N % n_step || c.K < 16 || (c.K & 15)) return BI_ERR_UNSUPPORTED_SHAPE;
    if (c.M > 0x7fffffff - pair::BMP || c.N > 0x7fffffff - pair::BN || c.K > 0x7fffffff - 512)
        return BI_ERR_UNSUPPORTED_SHAPE;  // row, column and byte indices stay in int
    const int64_t spans = bi_fp8::spans_of(c.K);
    if ((c.M + 255) / 128 * spans > 0x7fffffffLL || (c.N + 255) / 128 * spans > 0x7fffffffLL)
        return BI_ERR_UNSUPPORTED_SHAPE;
    if (c.ld_x < c.K || c.ld_w < c.K) return BI_ERR_INVALID_ARG;
    if ((c.ld_x & 15) || (c.ld_w & 15)) return BI_ERR_MISALIGNED;
    return BI_OK;
}

}  // namespace

extern "C" bi_status bi_gemm_fp8(const void* x, const void* x_scales, const void* W,
                                 const void* W_scales, void* y, int32_t M, int32_t N, int32_t K,
                                 int64_t ld_x, int64_t ld_w, int64_t ld_y, cudaStream_t stream) {
    const Call c{x, x_scales, W, W_scales, M, N, K, ld_x, ld_w, {y, ld_y, nullptr, 0}, stream};
    const bi_status st = check(c, 8);
    if (st != BI_OK) return st;
    if (ld_y < N) return BI_ERR_INVALID_ARG;
    if (ld_y & 7) return BI_ERR_MISALIGNED;
    if (M == 0) return BI_OK;
    if (!x || !x_scales || !W || !W_scales || !y) return BI_ERR_INVALID_ARG;
    if (!bi::aligned16(x) || !bi::aligned16(x_scales) || !bi::aligned16(W) ||
        !bi::aligned16(W_scales) || !bi::aligned16(y))
        return BI_ERR_MISALIGNED;
    return launch_gemm<false>(c);
}

extern "C" bi_status bi_gemm_fp8_swiglu(const void* x, const void* x_scales, const void* W_gu,
                                        const void* W_gu_scales, void* h, void* h_scales, int32_t M,
                                        int32_t F, int32_t K, int64_t ld_x, int64_t ld_w,
                                        int64_t ld_h, cudaStream_t stream) {
    if (F < 16 || F > (0x7fffffff >> 1)) return BI_ERR_UNSUPPORTED_SHAPE;
    const Call c{x, x_scales, W_gu, W_gu_scales, M, 2 * F, K, ld_x, ld_w,
                 {h, ld_h, static_cast<uint8_t*>(h_scales), bi_fp8::spans_of(F)}, stream};
    const bi_status st = check(c, 32);
    if (st != BI_OK) return st;
    if (ld_h < F) return BI_ERR_INVALID_ARG;
    if (ld_h & 15) return BI_ERR_MISALIGNED;
    if (M == 0) return BI_OK;
    if (!x || !x_scales || !W_gu || !W_gu_scales || !h || !h_scales) return BI_ERR_INVALID_ARG;
    if (!bi::aligned16(x) || !bi::aligned16(x_scales) || !bi::aligned16(W_gu) ||
        !bi::aligned16(W_gu_scales) || !bi::aligned16(h) || !bi::aligned16(h_scales))
        return BI_ERR_MISALIGNED;
    return launch_gemm<true>(c);
}
