// bi_gemm_fp8, bi_gemm_fp8_swiglu: y = x . W^T of two 8-bit matrices (fp8.cuh)
// on tcgen05 tensor cores, the scales applied by the MMA itself.
//
// Arithmetic, the same for every M ("Defeating Nondeterminism in LLM Inference:
// The Core Role of Batch Invariance", section "2. Batch-Invariant Matrix
// Multiplication": the reduction order must not follow the batch size).  K is cut
// into at most 8 parts of 1024 values or more, by K alone (parts_of).  A
// part's sum is one fp32 tensor-memory accumulator: its blocks of 128 ascending,
// each as four MMAs of depth 32 whose products carry the two scales (powers of
// two, so scaling rounds nothing).  The parts' sums are then added in ascending
// order in fp32.  The page warns against split-K because a split that follows the
// batch changes the order; this one is part of the definition, as the attention's
// 256-token chunks are, so a call may compute the parts on one SM after another
// or on several at once:
//   many rows   gemm_fp8_pair_kernel: tiles of 256 rows on CTA pairs, a part's
//               accumulator drained into registers while the next part runs;
//   few rows    gemm_fp8_parts_kernel: a cluster of CTAs, one part each, whose sums
//               meet through distributed shared memory.  The weight is what such
//               a call has to read, and the parts are what spreads it over all SMs;
//   few rows, many of W   gemm_fp8_whole_kernel: a CTA an SM, all parts in turn.
// All give an output the same bits: the same MMA depth, kind and order, with the
// operands' roles swapped in the last two (tests compare them, adversarial inputs
// included).  launch_gemm has the rule and what it was measured with.
//
// Measured, weights cold: 8192 rows 3.1 to 3.5 PFLOP/s (N = 4096, K = 12288 236 us, N =
// 24576, K = 4096 475 us), where the board's power holds the clock at 1.7 to 1.8 GHz and a k-block
// takes 578 cycles against the MMAs' 512: its 33152 bytes come into each SM at 57 a cycle.  One
// row, N = 24576, K = 4096 18.2 us, K = 12288, N = 4096 10.0 us, 5.6 and 5.1 TB/s of weights and
// scales: what is left are the starts and ends of the CTAs, 2 to 3 us a call that nothing overlaps.
//
// Registers spilled (counted by local loads and stores over sizes of K): none in a loop over
// k-blocks.  Pair with 128 columns, once a tile; with 256, two loads an epilogue warp and part;
// whole with 128 rows three loads and a store a warp and part, with SwiGLU one load.
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
// H: halves of 128 columns in a tile.  Two as a rule; one where that keeps more pairs
// busy, at the price of reading x twice as often (each SM then takes 24 KB in the time of
// 256 cycles' MMAs, more than the 64 bytes a cycle it can).
// The 8-bit output leaves from registers, so SwiGLU has room for one more stage.
template <int H, bool kSwiGLU>
struct PairShape {
    static constexpr int BMP = 256;  // tile rows of the pair; 128 per CTA
    static constexpr int BN = 128 * H;
    static constexpr int kStages = H == 1 ? 7 : kSwiGLU ? 6 : 5;
    static constexpr int kABytes = 128 * BK;
    static constexpr int kStageBytes = kABytes + H * 64 * BK;  // 128 rows of x, 64 of each half's W
    static constexpr int kScaleBytes = (1 + H) * kTile;
    static constexpr int kEpiWarps = 8;
    static constexpr int kThreads = 128 + 32 * kEpiWarps;
    // Registers a thread: 168 at launch (three warps share a sub-partition's 16384).  The
    // epilogue holds 128 sums and loads 64 columns at once; the other four warps give
    // theirs up for that.
    static constexpr int kFewRegs = 56, kManyRegs = 224;
    static_assert(128 * kFewRegs + 32 * kEpiWarps * kManyRegs <= kThreads * 168, "registers");
    // Tensor memory: three accumulators of 128 columns, and 8 places of 16 columns
    // for scales.  The tile's column halves are accumulators of their own, taken in turn out
    // of three, so that a half's MMAs of the next part need not wait for the other half to
    // be drained; two accumulators of 256 columns would leave no room for the scales.
    static constexpr uint32_t kTmemCols = 512;
    static constexpr uint32_t kScaleCol = 384;
    static_assert(kStages < 8, "scale places");
    static constexpr int kOutBytes = 32 * 64;  // a warp's 32 rows x 32 bf16 columns on their way out
    static constexpr int kOutBufs = kSwiGLU ? 0 : 3;  // of them in turn
    static constexpr int kOutOffset = (kStages * (kStageBytes + kScaleBytes) + 1023) / 1024 * 1024;
    static constexpr int kSmemBytes = kOutOffset + kEpiWarps * kOutBufs * kOutBytes + 1024 + 256;
    static constexpr uint32_t kIdesc = mx_idesc(BMP, 128);
};

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

template <bool kSwiGLU, int H>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(PairShape<H, kSwiGLU>::kThreads, 1)
    gemm_fp8_pair_kernel(const __grid_constant__ CUtensorMap tmap_x,
                         const __grid_constant__ CUtensorMap tmap_w,
                         const __grid_constant__ CUtensorMap tmap_xs,
                         const __grid_constant__ CUtensorMap tmap_ws,
                         const __grid_constant__ CUtensorMap tmap_y, Out out, int M, int N, int K,
                         int part_blocks, int group_m, uint32_t* err) {
    static_assert(!kSwiGLU || H == 2, "a block of 128 outputs takes 256 W rows");
    using S = PairShape<H, kSwiGLU>;
    constexpr int kStages = S::kStages, kABytes = S::kABytes, kStageBytes = S::kStageBytes;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t* smem_scales = smem + kStages * kStageBytes;
    uint8_t* smem_out = smem + S::kOutOffset;
    uint64_t* full = reinterpret_cast<uint64_t*>(smem_out + S::kEpiWarps * S::kOutBufs *
                                                                S::kOutBytes);
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
    const int num_m = (M + S::BMP - 1) / S::BMP;
    const int num_n = (N + S::BN - 1) / S::BN;
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
            bi::mbar_init(&tempty[i], 2 * S::kEpiWarps);  // both CTAs' (leader's copy used)
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
        bi::tmem_alloc_pair(tmem_slot, S::kTmemCols);
        bi::tmem_relinquish_pair();
    }
    if (warp == 0) {
        // the ring's first stages of the weight start on their way to L2 while the previous
        // kernel still runs, once for all the pairs that share them (a decoder layer's chain
        // of calls, 300 rows 100.1 -> 99.1 us, 511 rows 102.0 -> 100.9; four rings' worth: 100.2, 102.1)
        int mb, nb;
        tile_coords(pair_id, num_m, num_n, group_m, mb, nb);
        if (mb == 0 && bi::elect_one())
            for (int i = 0; i < min(num_kb, kStages); ++i)
#pragma unroll
                for (int h = 0; h < H; ++h)
                    bi::tma_prefetch_2d(&tmap_w, i * BK, nb * S::BN + static_cast<int>(rank) * 64 + 128 * h);
        __syncwarp();
    }
    bi::tc_fence_before();
    bi::cluster_sync();  // both CTAs' barriers exist before either signals the other
    bi::tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    bi::launch_dependents();
    bi::grid_dependency_wait();  // nothing global is touched before the previous kernel ends

    if (warp < 4) {
        bi::fewer_registers<S::kFewRegs>();
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
                const int w_row = nb * S::BN + static_cast<int>(rank) * 64;
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
                                &full[stage], 2 * (kStageBytes + (scales ? S::kScaleBytes : 0)));
                        bi::tma_load_2d_pair(sa, &tmap_x, bar, kb * BK, m_tile * 128);
                        // a half's 128 W rows come half from each CTA (its share of B)
#pragma unroll
                        for (int h = 0; h < H; ++h)
                            bi::tma_load_2d_pair(sa + kABytes + h * 64 * BK, &tmap_w, bar, kb * BK,
                                                 w_row + 128 * h);
                        if (scales) {
                            uint8_t* sf = smem_scales + stage * S::kScaleBytes;
                            bi::tma_load_2d_pair(sf, &tmap_xs, bar, 0, m_tile * spans + (kb >> 2));
#pragma unroll
                            for (int h = 0; h < H; ++h)
                                bi::tma_load_2d_pair(sf + (1 + h) * kTile, &tmap_ws, bar, 0,
                                                     (H * nb + h) * spans + (kb >> 2));
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
                    int d[H] = {};
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
                            sfa = tmem + S::kScaleCol + 16 * sf;
                            sf = (sf + 1) & 7;
                            const uint64_t s = scale_desc(ring + kStages * kStageBytes +
                                                          stage * S::kScaleBytes);
                            if (bi::elect_one()) {
#pragma unroll
                                for (int i = 0; i < 1 + H; ++i)
                                    bi::tc_cp_scales_pair(sfa + 4 * i, s + (i * kTile >> 4));
                            }
                            __syncwarp();
                        }
                        const uint32_t idesc = with_byte(S::kIdesc, kb & 3);
                        const uint64_t da = operand_desc(sa), db = operand_desc(sa + kABytes);
#pragma unroll
                        for (int h = 0; h < H; ++h) {
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
                                if (h == H - 1)  // the stage is free in both CTAs
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
        bi::more_registers<S::kManyRegs>();
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
            float sum[H][64];  // from -0 on: -0 + x is x, whatever its sign
#pragma unroll
            for (int h = 0; h < H; ++h)
#pragma unroll
                for (int i = 0; i < 64; ++i) sum[h][i] = -0.f;
#pragma unroll 1
            for (int p = 0; p < num_parts; ++p) {
#pragma unroll
                for (int h = 0; h < H; ++h) {
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
            const int row = mb * S::BMP + static_cast<int>(rank) * 128 + in_tile;
            if constexpr (!kSwiGLU) {
                // 32 rows x 32 columns at a time through shared memory (64-byte rows,
                // swizzled: no bank conflicts) and out by TMA, which clips them to y.  A
                // lane storing its own row's 16 bytes at a time costs a cycle of the
                // store path for each of a warp's 32 rows: 6900 cycles a tile.
                if (!ok) continue;
                const int row0 = row - lane;
#pragma unroll
                for (int q = 0; q < 2 * H; ++q) {
                    const int col = nb * S::BN + 128 * (q >> 1) + 64 * c + 32 * (q & 1);
                    if (row0 >= M || col >= N) continue;  // the whole warp
                    uint8_t* buf = smem_out + ((warp - 4) * S::kOutBufs + out_buf) * S::kOutBytes;
                    if (++out_buf == S::kOutBufs) out_buf = 0;
                    if (bi::elect_one()) bi::tma_store_wait_read<S::kOutBufs - 1>();
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
                for (int h = 0; h < H; ++h)
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
                for (int h = 0; h < H; ++h) {
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
        bi::tmem_dealloc_pair(tmem_base, S::kTmemCols);
    }
}

// ----------------------------------------------------------- few rows ----
// The scales of k-blocks kb .. kb + 3 of 128 rows.  Past the last of a matrix' tiles
// (where it has no rows, and its codes are zeros) the last one's.
__device__ __forceinline__ void load_scales(uint8_t* dst, const uint8_t* scales, int tile, int rows,
                                            int kb, int spans, uint64_t* bar) {
    tile = min(tile, (rows - 1) >> 7);
    bi::bulk_load(dst, scales + (static_cast<int64_t>(tile) * spans + (kb >> 2)) * kTile, kTile, bar);
}

// NT: rows of x per CTA (the MMA's N); WT: tiles of 128 W rows per CTA (the MMA's
// M): one, or two where a block of 128 SwiGLU outputs needs 256 W rows or half the CTAs
// are more than the SMs hold at once; STAGES: k-blocks in flight per CTA.
template <int NT, int WT, int STAGES>
struct PartsShape {
    static constexpr int kWBytes = WT * 128 * BK;
    static constexpr int kStageBytes = kWBytes + NT * BK;
    static constexpr int kScaleBytes = (WT + 1) * kTile;
    static constexpr int kStages = STAGES;
    // Scales serve four k-blocks.  Their slot is loaded again for the next four when a
    // stage is free whose MMAs, kStages k-blocks ago, came after the slot's copy.
    static constexpr int kSlots = (kStages + 3) / 4;
    static constexpr int kScaleOffset = kStages * kStageBytes;
    static constexpr int kBarOffset = kScaleOffset + kSlots * kScaleBytes;
    static constexpr int kRecvOffset = kBarOffset + 256;
    // How the parts' sums meet.  Few sums a CTA sends to the CTA that puts the row
    // together, into memory kept for that: one way, and no barrier (one row, N = K = 4096:
    // 5.9 -> 5.7 us, K = 12288, 17 rows: 11.0 -> 10.5).  Many would take the place of one more
    // CTA on the SM (N = 6144, 128 rows: 18.2 us against 11.8; SwiGLU of F = 12288, 17 rows:
    // 25.0 against 20.0); they are left in the ring, which is done with, for the others to
    // read.
    static constexpr bool kSend = WT == 1 ? NT <= 64 : NT <= 16;
    static int recv_bytes(int rows, int parts) {
        return kSend ? (rows + parts - 1) / parts * parts * WT * 128 * 4 : 0;
    }
    static constexpr int kMostRecv = kSend ? (NT + 7) * WT * 128 * 4 : 0;
    static_assert(kSend || NT * WT * 128 * 4 <= kScaleOffset, "sums lie in the ring");
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
    static int smem_bytes(int rows, int parts) {
        return std::max(kShareBytes, kRecvOffset + recv_bytes(rows, parts) + 1024);
    }
    static constexpr int kMostBytes =
        std::max(kShareBytes, std::min(227 * 1024, kRecvOffset + kMostRecv + 1024));
};

// Output rows l < rows out of their sums: fold(l, n) gives four neighbouring values of the
// CTA's WT * 128 columns, row_of(l) the row of the output, n0 the first column's W row.
template <bool kSwiGLU, int WT, int THREADS, typename Fold, typename RowOf>
__device__ __forceinline__ void put_rows(const Out& out, const Fold& fold, int rows,
                                         const RowOf& row_of, int n0, int N) {
    if constexpr (!kSwiGLU) {
        constexpr int kFours = WT * 32;
        for (int i = threadIdx.x; i < rows * kFours; i += THREADS) {
            const int l = i / kFours, n = 4 * (i % kFours);
            const float4 s = fold(l, n);
            if (n0 + n < N)
                *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(out.y) +
                                          static_cast<int64_t>(row_of(l)) * out.ld + n0 + n) =
                    make_uint2(bi::pack_bf16x2(s.x, s.y), bi::pack_bf16x2(s.z, s.w));
        }
    } else {
        // a warp takes one row's 256 columns, a block of 128 outputs: lane i the outputs
        // 4i .. 4i + 3, whose gate and up columns lie 8 apart in a group of 16
        static_assert(WT == 2, "a whole block of outputs");
        const int lane = threadIdx.x & 31;
        const int col = n0 / 2 + 4 * lane;
        for (int l = threadIdx.x >> 5; l < rows; l += THREADS / 32) {
            const int at = (lane >> 1) * 16 + (lane & 1) * 4;
            const float4 g = fold(l, at), u = fold(l, at + 8);
            const float h0 = bi::swiglu(g.x, u.x), h1 = bi::swiglu(g.y, u.y);
            const float h2 = bi::swiglu(g.z, u.z), h3 = bi::swiglu(g.w, u.w);
            uint32_t top = max(max(__float_as_uint(h0) & 0x7fffffffu, __float_as_uint(h1) & 0x7fffffffu),
                               max(__float_as_uint(h2) & 0x7fffffffu, __float_as_uint(h3) & 0x7fffffffu));
            if (2 * col >= N) top = 0;  // past F: no W rows, and perhaps NaN for their scales
            top = __reduce_max_sync(0xffffffffu, top);
            const uint32_t byte = bi_fp8::scale_byte(top);
            const float inv = bi_fp8::inverse_scale(byte);
            const int64_t row = row_of(l);
            if (2 * col < N)
                *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(out.y) + row * out.ld + col) =
                    bi_fp8::codes4(__fmul_rn(h0, inv), __fmul_rn(h1, inv), __fmul_rn(h2, inv),
                                   __fmul_rn(h3, inv));
            if (lane == 0)
                out.scales[bi_fp8::scale_word(row, n0 >> 10, out.spans) + ((n0 >> 8) & 3)] =
                    static_cast<uint8_t>(byte);
        }
    }
}

template <int NT, int WT, bool kSwiGLU, int STAGES>
__global__ void __launch_bounds__(192)
    gemm_fp8_parts_kernel(const __grid_constant__ CUtensorMap tmap_x,
                          const __grid_constant__ CUtensorMap tmap_w,
                          const uint8_t* __restrict__ x_scales,
                          const uint8_t* __restrict__ w_scales, Out out, int M, int N, int K,
                          int part_blocks, bool prefetch, uint32_t* err) {
    using S = PartsShape<NT, WT, STAGES>;
    constexpr int kStages = S::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t* smem_scales = smem + S::kScaleOffset;
    // sums received [own rows][parts][WT * 128], or left for the others [rows][WT * 128]
    float* sums = reinterpret_cast<float*>(smem + (S::kSend ? S::kRecvOffset : 0));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + S::kBarOffset);
    uint64_t* empty = full + kStages;
    uint64_t* tfull = empty + kStages;
    uint64_t* rfull = tfull + 1;  // all sums of this CTA's rows have arrived
    uint64_t* drain = rfull + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
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
    const int rows = min(NT, M - m0);
    // row m of the tile is put together by CTA m % nparts, as its row m / nparts
    const int own_rows = (rows - rank + nparts - 1) / nparts;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            bi::mbar_init(&full[i], 1);
            bi::mbar_init(&empty[i], 1);
        }
        bi::mbar_init(tfull, 1);
        bi::mbar_init(rfull, 1);
        bi::mbar_init(drain, 1);
        bi::fence_mbar_init();
        if (S::kSend) bi::mbar_arrive_expect_tx(rfull, own_rows * nparts * WT * 512);
        s_timeout = 0;
        s_issued = 0;
        s_consumed = 0;
        bi::tma_prefetch_desc(&tmap_x);
        bi::tma_prefetch_desc(&tmap_w);
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
    bi::cluster_sync();  // every CTA's barriers exist before another's sums arrive
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
                    uint8_t* sf = smem_scales + (issued >> 2) % S::kSlots * S::kScaleBytes;
#pragma unroll
                    for (int t = 0; t < WT; ++t)
                        load_scales(sf + t * kTile, w_scales, n0 / 128 + t, N, kb, spans, &full[stage]);
                    // NT < 128 only where one tile holds all rows, so a tile's rows start
                    // where its scales do
                    load_scales(sf + WT * kTile, x_scales, m0 / 128, M, kb, spans, &full[stage]);
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
            const uint64_t s = scale_desc(ring + S::kScaleOffset + (i >> 2) % S::kSlots * S::kScaleBytes);
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
                                        idesc, sfw + 4 * t, sfw + 4 * WT,
                                        (i | k) != 0 ? 1u : 0u);
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
        // a part that gave up has NaN: nobody waits in vain, and nothing looks like a sum
        const uint32_t taddr = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16);
        const uint32_t to = bi::smem_u32(sums + quarter * 32 + lane), bar = bi::smem_u32(rfull);
#pragma unroll
        for (int t = 0; t < WT; ++t) {
            int owner = 0, local = 0;
            for (int m = 0; m < rows; m += 16) {
                uint32_t r[16];
                if (ok) {
                    bi::tmem_ld_32x32b_x16(taddr + t * NT + m, r);
                    bi::tmem_ld_wait();
                }
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const float v = __uint_as_float(ok ? r[e] : 0x7FC00000u);
                    if constexpr (S::kSend) {
                        if (m + e >= rows) break;
                        const uint32_t at = to + 4 * ((local * nparts + rank) * (WT * 128) + t * 128);
                        bi::st_async_f32(bi::mapa_shared(at, owner), v, bi::mapa_shared(bar, owner));
                        if (++owner == nparts) {
                            owner = 0;
                            ++local;
                        }
                    } else if (ok) {  // (the ring may still be written where it is not)
                        sums[(m + e) * (WT * 128) + t * 128 + quarter * 32 + lane] = v;
                    }
                }
            }
        }
    }
    __syncwarp();

    // the parts' sums of this CTA's rows, ascending
    bool arrived = true;
    if constexpr (S::kSend) {  // a peer that gives up does so within kWaitNs and then sends
        arrived = __all_sync(0xffffffffu, bi::mbar_wait_cluster(rfull, 0, 3 * bi::kWaitNs));
        if (!arrived && lane == 0) {
            bi::report_error(err, bi::kErrTimeout | bi::kWhereGemmFp8);
            s_timeout = 1;
        }
    } else {
        __syncthreads();
        if (s_timeout) {
            if (threadIdx.x == 0)  // copies in flight land in the ring
                for (int i = s_consumed; i < s_issued; ++i)
                    bi::mbar_wait_for(&full[i % kStages], (i / kStages) & 1, bi::kDrainNs);
            __syncthreads();
            for (int i = threadIdx.x; i < NT * WT * 128; i += 192) sums[i] = __uint_as_float(0x7FC00000u);
        }
        bi::cluster_sync();
    }
    const uint32_t sums_at = bi::smem_u32(sums);
    const auto fold = [&](int l, int n) {  // four neighbouring values of own row l
        float4 v[8];
#pragma unroll
        for (int p = 0; p < 8; ++p) {
            if (p >= nparts) continue;
            if constexpr (S::kSend)
                v[p] = *reinterpret_cast<const float4*>(sums + (l * nparts + p) * (WT * 128) + n);
            else
                v[p] = bi::ld_cluster_f4(
                    bi::mapa_shared(sums_at + 4 * ((l * nparts + rank) * (WT * 128) + n), p));
        }
        float4 s = v[0];
#pragma unroll
        for (int p = 1; p < 8; ++p) {
            if (p >= nparts) continue;
            s.x = __fadd_rn(s.x, v[p].x);
            s.y = __fadd_rn(s.y, v[p].y);
            s.z = __fadd_rn(s.z, v[p].z);
            s.w = __fadd_rn(s.w, v[p].w);
        }
        return s;
    };
    if (arrived)
        put_rows<kSwiGLU, WT, 192>(out, fold, own_rows, [&](int l) { return m0 + l * nparts + rank; },
                                   n0, N);
    bi::tc_fence_before();
    __syncthreads();
    if (S::kSend && s_timeout && threadIdx.x == 0)  // copies in flight
        for (int i = s_consumed; i < s_issued; ++i)
            bi::mbar_wait_for(&full[i % kStages], (i / kStages) & 1, bi::kDrainNs);
    if (warp == 1) {
        bi::tc_fence_after();
        bi::tmem_dealloc(tmem_base, S::kTmemCols);
    }
    __syncwarp();
    bi::cluster_sync_relaxed();  // no CTA leaves while sums are on their way to it, or read
}

// ------------------------------------ few rows, enough W rows for all SMs ----
// A CTA runs all of K for 256 W rows and the M <= NT rows of x, alone on its SM, the parts one
// after the other: no cluster, and the sums meet in registers as in the pair kernel (whose
// 256 rows of x would be mostly empty here).
template <int NT>
struct WholeShape {
    static constexpr int kStageBytes = 256 * BK + NT * BK;
    static constexpr int kScaleBytes = 3 * kTile;
    static constexpr int kStages = NT <= 32 ? 5 : 4;
    static constexpr int kScaleOffset = kStages * kStageBytes;
    static constexpr int kBarOffset = kScaleOffset + kStages * kScaleBytes;
    static constexpr int kSmemBytes = kBarOffset + 256 + 1024;
    static_assert(NT * 256 * 4 <= kScaleOffset, "sums lie in the ring at last");
    // Tensor memory: three accumulators of NT columns, taken in turn by the two W tiles of
    // every part (one is drained while the other's last k-block still runs), and 8 places
    // for scales: one is used again at least 8 k-blocks later, kStages < 8.
    static constexpr uint32_t kScaleCol = 384;
    static constexpr int kThreads = 320;
};

template <int NT, bool kSwiGLU>
__global__ void __launch_bounds__(WholeShape<NT>::kThreads, 1)
    gemm_fp8_whole_kernel(const __grid_constant__ CUtensorMap tmap_x,
                          const __grid_constant__ CUtensorMap tmap_w,
                          const uint8_t* __restrict__ x_scales,
                          const uint8_t* __restrict__ w_scales, Out out, int M, int N, int K,
                          int part_blocks, uint32_t* err) {
    using S = WholeShape<NT>;
    constexpr int kStages = S::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t* smem_scales = smem + S::kScaleOffset;
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + S::kBarOffset);
    uint64_t* empty = full + kStages;
    uint64_t* tfull = empty + kStages;
    uint64_t* tempty = tfull + 3;
    uint64_t* done = tempty + 3;  // every MMA has completed
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
    __shared__ int s_timeout, s_issued, s_consumed;

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
    const int lane = threadIdx.x & 31;
    const int n0 = blockIdx.x * 256;
    const int num_kb = (K + BK - 1) / BK;
    const int spans = (num_kb + 3) >> 2;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            bi::mbar_init(&full[i], 1);
            bi::mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 3; ++i) {
            bi::mbar_init(&tfull[i], 1);
            bi::mbar_init(&tempty[i], 4);
        }
        bi::mbar_init(done, 1);
        bi::fence_mbar_init();
        s_timeout = 0;
        s_issued = 0;
        s_consumed = 0;
        bi::tma_prefetch_desc(&tmap_x);
        bi::tma_prefetch_desc(&tmap_w);
    }
    if (warp == 1) {
        bi::tmem_alloc(tmem_slot, 512);
        bi::tmem_relinquish();
    }
    if (warp == 0) {
        // two rings of the weight start on their way to L2 while the previous kernel, which
        // as a rule makes x, still runs (a decoder layer's chain of calls, 24 rows 52.4 ->
        // 51.5 us, 128 rows 73.6 -> 71.0; all of the weight at once: 51.7 and 74.5)
        if (bi::elect_one())
            for (int i = 0; i < min(num_kb, 2 * kStages); ++i) {
                bi::tma_prefetch_2d(&tmap_w, i * BK, n0);
                bi::tma_prefetch_2d(&tmap_w, i * BK, n0 + 128);
            }
        __syncwarp();
    }
    bi::tc_fence_before();
    __syncthreads();
    bi::tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    bi::launch_dependents();
    bi::grid_dependency_wait();  // nothing global is touched before the previous kernel ends

    float sum[NT];  // epilogue warps; from -0 on: -0 + x is x, whatever its sign
    if (warp == 0) {  // the whole warp runs the loop, one lane issues
        int stage = 0;
        uint32_t phase = 0;
        int kb = 0;
        bool ok = true;
        for (; kb < num_kb; ++kb) {
            if (!__all_sync(0xffffffffu, bi::mbar_wait(&empty[stage], phase ^ 1))) {
                ok = false;
                break;
            }
            const bool scales = (kb & 3) == 0;
            uint8_t* sw = smem + stage * S::kStageBytes;
            if (bi::elect_one()) {
                bi::mbar_arrive_expect_tx(&full[stage],
                                          S::kStageBytes + (scales ? S::kScaleBytes : 0));
                bi::tma_load_2d(sw, &tmap_w, &full[stage], kb * BK, n0);
                bi::tma_load_2d(sw + 128 * BK, &tmap_w, &full[stage], kb * BK, n0 + 128);
                bi::tma_load_2d(sw + 256 * BK, &tmap_x, &full[stage], kb * BK, 0);
                if (scales) {
                    uint8_t* sf = smem_scales + stage * S::kScaleBytes;
                    load_scales(sf, w_scales, n0 / 128, N, kb, spans, &full[stage]);
                    load_scales(sf + kTile, w_scales, n0 / 128 + 1, N, kb, spans, &full[stage]);
                    load_scales(sf + 2 * kTile, x_scales, 0, M, kb, spans, &full[stage]);
                }
            }
            __syncwarp();
            if (++stage == kStages) {
                stage = 0;
                phase ^= 1;
            }
        }
        if (lane == 0) {
            s_issued = kb;
            if (!ok) {
                bi::report_error(err, bi::kErrTimeout | bi::kWhereGemmFp8);
                s_timeout = 1;
            }
        }
    } else if (warp == 1) {  // the whole warp runs the loop, one lane issues
        const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_base, 0);
        const uint32_t ring = bi::smem_u32(smem);
        uint32_t sf = 0;
        int stage = 0, acc = 0, left = 0, kb = 0;
        uint32_t phase = 0, acc_phase = 0;
        int d[2] = {0, 0};
        bool ok = true;
        for (; kb < num_kb && ok; ++kb) {
            const bool first = left == 0;
            if (first) left = min(part_blocks, num_kb - kb);
            --left;
            if (!__all_sync(0xffffffffu, bi::mbar_wait(&full[stage], phase))) {
                ok = false;
                break;
            }
            bi::tc_fence_after();
            const uint32_t sw = ring + stage * S::kStageBytes;
            const uint64_t dw = operand_desc(sw), dx = operand_desc(sw + 256 * BK);
            const uint32_t idesc = with_byte(mx_idesc(128, NT), kb & 3);
            if ((kb & 3) == 0) {
                sf = tmem + S::kScaleCol + 16 * ((kb >> 2) & 7);
                const uint64_t s = scale_desc(ring + S::kScaleOffset + stage * S::kScaleBytes);
                if (bi::elect_one()) {
#pragma unroll
                    for (int t = 0; t < 3; ++t) bi::tc_cp_scales(sf + 4 * t, s + (t * kTile >> 4));
                }
                __syncwarp();
            }
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                if (first) {
                    if (!__all_sync(0xffffffffu, bi::mbar_wait(&tempty[acc], acc_phase ^ 1))) {
                        ok = false;
                        break;
                    }
                    bi::tc_fence_after();
                    d[t] = acc;
                    if (++acc == 3) {
                        acc = 0;
                        acc_phase ^= 1;
                    }
                }
                if (bi::elect_one()) {
#pragma unroll
                    for (int k = 0; k < BK / 32; ++k)
                        bi::tc_mma_mxf8(tmem + d[t] * NT, dw + (t * 128 * BK >> 4) + 2 * k, dx + 2 * k,
                                        idesc, sf + 4 * t, sf + 8, (!first || k != 0) ? 1u : 0u);
                    if (left == 0) bi::tc_commit(&tfull[d[t]]);
                    if (t == 1) bi::tc_commit(&empty[stage]);
                    if (t == 1 && kb + 1 == num_kb) bi::tc_commit(done);
                }
                __syncwarp();
            }
            if (++stage == kStages) {
                stage = 0;
                phase ^= 1;
            }
        }
        if (bi::elect_one()) {
            s_consumed = kb;
            if (!ok) {
                bi::report_error(err, bi::kErrTimeout | bi::kWhereGemmFp8);
                s_timeout = 1;
                if (kb > 0) {  // a bounded wait for what was issued
                    bi::tc_commit(done);
                    bi::mbar_wait_for(done, 0, bi::kDrainNs);
                }
            }
        }
        __syncwarp();
    } else {
        // warps 2..5 tile 0, 6..9 tile 1: W rows quarter * 32 + lane, all rows of x
        const int quarter = warp & 3;
        const int t = (warp - 2) >> 2;
        const int num_parts = (num_kb + part_blocks - 1) / part_blocks;
        const uint32_t taddr = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16);
        int acc = t;
        uint32_t acc_phase = 0;
        bool ok = true;
#pragma unroll
        for (int i = 0; i < NT; ++i) sum[i] = -0.f;
#pragma unroll 1
        for (int p = 0; p < num_parts && ok; ++p) {
            ok = __all_sync(0xffffffffu, bi::mbar_wait(&tfull[acc], acc_phase));
            if (!ok) break;
            bi::tc_fence_after();
#pragma unroll
            for (int q = 0; q < NT / 16; ++q) {
                uint32_t r[16];
                bi::tmem_ld_32x32b_x16(taddr + acc * NT + 16 * q, r);
                bi::tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    sum[16 * q + i] = __fadd_rn(sum[16 * q + i], __uint_as_float(r[i]));
            }
            bi::tc_fence_before();
            __syncwarp();
            if (lane == 0) bi::mbar_arrive(&tempty[acc]);
            acc += 2;
            if (acc >= 3) {
                acc -= 3;
                acc_phase ^= 1;
            }
        }
        // the ring is free once the other tile's MMAs are done too
        if (ok) ok = __all_sync(0xffffffffu, bi::mbar_wait(done, 0));
        if (!ok && lane == 0) {
            bi::report_error(err, bi::kErrTimeout | bi::kWhereGemmFp8);
            s_timeout = 1;
        }
        if (ok) {
            float* to = reinterpret_cast<float*>(smem) + t * 128 + quarter * 32 + lane;
#pragma unroll
            for (int i = 0; i < NT; ++i)
                if (i < M) to[i * 256] = sum[i];
        }
        bi::tc_fence_before();
    }
    __syncthreads();
    if (s_timeout) {
        if (threadIdx.x == 0)  // copies in flight
            for (int i = s_consumed; i < s_issued; ++i)
                bi::mbar_wait_for(&full[i % kStages], (i / kStages) & 1, bi::kDrainNs);
        __syncthreads();
    } else {
        const float* sums = reinterpret_cast<const float*>(smem);
        put_rows<kSwiGLU, 2, S::kThreads>(
            out, [&](int l, int n) { return *reinterpret_cast<const float4*>(sums + l * 256 + n); },
            M, [](int l) { return l; }, n0, N);
    }
    if (warp == 1) {
        bi::tc_fence_after();
        bi::tmem_dealloc(tmem_base, 512);
    }
}

// ------------------------------------------------------------- launches ----
struct Call {
    const void *x, *xs, *W, *Ws;
    int32_t M, N, K;  // N: rows of W
    int64_t ld_x, ld_w;
    Out out;
    cudaStream_t stream;
    bi::Device dev;
};

bool encode(const Call& c, uint32_t x_rows, uint32_t w_rows, CUtensorMap& x, CUtensorMap& w) {
    return bi::encode_byte_map_2d(&x, c.x, c.K, c.M, c.ld_x, x_rows) == CUDA_SUCCESS &&
           bi::encode_byte_map_2d(&w, c.W, c.K, c.N, c.ld_w, w_rows) == CUDA_SUCCESS;
}

bool encode(const Call& c, uint32_t x_rows, uint32_t w_rows, CUtensorMap (&t)[4]) {
    const uint64_t spans = bi_fp8::spans_of(c.K);
    return encode(c, x_rows, w_rows, t[0], t[1]) &&
           bi::encode_scale_map(&t[2], c.xs, (c.M + 127) / 128 * spans) == CUDA_SUCCESS &&
           bi::encode_scale_map(&t[3], c.Ws, (c.N + 127) / 128 * spans) == CUDA_SUCCESS;
}

template <bool kSwiGLU, int H>
bi_status launch_pair(const Call& c, int sms) {
    using S = PairShape<H, kSwiGLU>;
    static std::atomic<bool> set[64] = {};
    if (!bi::allow_smem(gemm_fp8_pair_kernel<kSwiGLU, H>, S::kSmemBytes, set, c.dev.index)) return BI_ERR_CUDA;
    CUtensorMap t[4];
    if (!encode(c, 128, 64, t)) return BI_ERR_CUDA;
    CUtensorMap ty = t[0];  // not read where the output is 8 bits
    if (!kSwiGLU && bi::encode_out_map(&ty, c.out.y, c.N, c.M, c.out.ld * 2) != CUDA_SUCCESS)
        return BI_ERR_CUDA;
    const int num_m = (c.M + S::BMP - 1) / S::BMP;
    const int64_t tiles = static_cast<int64_t>(num_m) * ((c.N + S::BN - 1) / S::BN);
    if (tiles > 0x7fffffffLL) return BI_ERR_UNSUPPORTED_SHAPE;
    const int pairs = static_cast<int>(std::min<int64_t>(tiles, sms / 2));
    // at most about 48 MB of x per group of M-tiles, as bi_gemm
    const int64_t slab = static_cast<int64_t>(S::BMP) * c.K;
    const int64_t budget = int64_t{48} << 20;
    int group_m = num_m;
    if (slab * num_m > budget) group_m = static_cast<int>(std::max<int64_t>(1, budget / slab));
    return bi::launch_pdl(gemm_fp8_pair_kernel<kSwiGLU, H>, dim3(2 * pairs), dim3(S::kThreads),
                          S::kSmemBytes, c.stream, t[0], t[1], t[2], t[3], ty, c.out, c.M, c.N, c.K,
                          parts_of(c.K).blocks, group_m, c.dev.err) == cudaSuccess
               ? BI_OK
               : BI_ERR_CUDA;
}

struct PartsPlan {
    Parts parts;
    int64_t ctas;
    int rows;  // of the largest tile
};

// Asked about, never launched: of a kernel that uses tensor memory the runtime says that an
// SM holds one CTA, as if each took all of it.
__global__ void no_tensor_memory_kernel() {}

// How many clusters of the parts kernel the device holds at once.  A cluster lies in one of
// the chip's GPCs, whose SMs are not a multiple of every cluster's size: 8 parts, one CTA an
// SM, 120 CTAs of 152; two an SM, 288 of 304.
int clusters_at_once(int dev, int an_sm, int parts, int bytes) {
    constexpr int kMostAnSm = 16;  // at 32 columns of tensor memory a CTA, the least
    static std::atomic<int> known[64][kMostAnSm + 1][9] = {};  // the device's answer + 1
    if (an_sm > kMostAnSm) an_sm = kMostAnSm;
    std::atomic<int>& slot = known[dev][an_sm][parts];
    int clusters = slot.load(std::memory_order_relaxed) - 1;
    if (clusters >= 0) return clusters;
    static std::atomic<bool> set[64] = {};
    if (!bi::allow_smem(no_tensor_memory_kernel, 227 * 1024, set, dev)) return 0;
    clusters = bi::active_clusters(no_tensor_memory_kernel, parts, dim3(192), bytes);
    slot.store(clusters + 1, std::memory_order_relaxed);
    return clusters;
}

template <int NT, int WT, bool kSwiGLU, int STAGES>
bool at_once(const Call& c, const PartsPlan& p) {  // whether the SMs hold all CTAs at once
    using S = PartsShape<NT, WT, STAGES>;
    const int bytes = S::smem_bytes(p.rows, p.parts.count);
    const int an_sm = (228 * 1024) / (bytes + 1024 + 128);
    if (bytes > S::kMostBytes || int64_t{an_sm} * c.dev.sms < p.ctas) return false;
    return p.parts.count == 1 ||
           int64_t{clusters_at_once(c.dev.index, an_sm, p.parts.count, bytes)} * p.parts.count >= p.ctas;
}

template <int NT, int WT, bool kSwiGLU, int STAGES>
bi_status launch_parts(const Call& c, const PartsPlan& p, bool prefetch) {
    using S = PartsShape<NT, WT, STAGES>;
    static std::atomic<bool> set[64] = {};
    if (!bi::allow_smem(gemm_fp8_parts_kernel<NT, WT, kSwiGLU, STAGES>, S::kMostBytes, set, c.dev.index))
        return BI_ERR_CUDA;
    CUtensorMap x, w;
    if (!encode(c, NT, 128, x, w)) return BI_ERR_CUDA;
    constexpr int rows = 128 * WT;
    const dim3 grid(p.parts.count, (c.M + NT - 1) / NT, (c.N + rows - 1) / rows);
    return bi::launch_pdl_cluster(gemm_fp8_parts_kernel<NT, WT, kSwiGLU, STAGES>, p.parts.count, grid,
                                  dim3(192), S::smem_bytes(p.rows, p.parts.count), c.stream, x, w,
                                  static_cast<const uint8_t*>(c.xs),
                                  static_cast<const uint8_t*>(c.Ws), c.out, c.M, c.N, c.K, p.parts.blocks, prefetch,
                                  c.dev.err) == cudaSuccess
               ? BI_OK
               : BI_ERR_CUDA;
}

template <int NT, int WT>
PartsPlan plan_of(const Call& c) {
    const Parts parts = parts_of(c.K);
    return {parts,
            static_cast<int64_t>(parts.count) * ((c.M + NT - 1) / NT) * ((c.N + 128 * WT - 1) / (128 * WT)),
            std::min(NT, c.M)};
}

template <int NT, bool kSwiGLU>
bi_status launch_whole(const Call& c) {
    using S = WholeShape<NT>;
    static std::atomic<bool> set[64] = {};
    if (!bi::allow_smem(gemm_fp8_whole_kernel<NT, kSwiGLU>, S::kSmemBytes, set, c.dev.index)) return BI_ERR_CUDA;
    CUtensorMap x, w;
    if (!encode(c, NT, 128, x, w)) return BI_ERR_CUDA;
    const dim3 grid((c.N + 255) / 256);
    return bi::launch_pdl(gemm_fp8_whole_kernel<NT, kSwiGLU>, grid, dim3(S::kThreads), S::kSmemBytes,
                          c.stream, x, w, static_cast<const uint8_t*>(c.xs),
                          static_cast<const uint8_t*>(c.Ws), c.out, c.M, c.N, c.K,
                          parts_of(c.K).blocks, c.dev.err) == cudaSuccess
               ? BI_OK
               : BI_ERR_CUDA;
}

// What becomes of the kernel that a call's sizes choose: it is launched, or named
// (bi_gemm_fp8_form).
struct Launch {
    using Result = bi_status;
    template <bool g, int H>
    static bi_status pair(const Call& c) {
        return launch_pair<g, H>(c, c.dev.sms);
    }
    template <bool g, int NT>
    static bi_status whole(const Call& c) {
        return launch_whole<NT, g>(c);
    }
    template <bool g, int NT, int WT, int STAGES>
    static bi_status parts(const Call& c, const PartsPlan& p, bool prefetch) {
        return launch_parts<NT, WT, g, STAGES>(c, p, prefetch);
    }
};
struct Name {
    using Result = int32_t;
    template <bool g, int H>
    static int32_t pair(const Call&) {
        return 1000000 + 128 * H * 1000 + PairShape<H, g>::kStages;
    }
    template <bool g, int NT>
    static int32_t whole(const Call&) {
        return 2000000 + NT * 1000 + 200 + WholeShape<NT>::kStages;
    }
    template <bool g, int NT, int WT, int STAGES>
    static int32_t parts(const Call&, const PartsPlan&, bool) {
        return 3000000 + NT * 1000 + 100 * WT + STAGES;
    }
};

// The deepest ring (most loads in flight a CTA) with which the SMs hold the launch at
// once, else the shallowest (most CTAs, whose starts and ends overlap).  Which of them ask
// for the weight early was measured: three stages of 128 W rows, at once, N = 12288, one row
// 10.6 -> 9.8 us; two of 256, N = 24576 18.1 -> 18.6, which therefore do not.
template <typename Act, bool g, int NT, int WT, int DEEP, int MID, int SHALLOW>
typename Act::Result choose_ring(const Call& c) {
    const PartsPlan p = plan_of<NT, WT>(c);
    if (at_once<NT, WT, g, DEEP>(c, p)) return Act::template parts<g, NT, WT, DEEP>(c, p, true);
    if (at_once<NT, WT, g, MID>(c, p)) return Act::template parts<g, NT, WT, MID>(c, p, true);
    return Act::template parts<g, NT, WT, SHALLOW>(c, p, WT == 1 && at_once<NT, WT, g, SHALLOW>(c, p));
}

// Which kernel: a schedule choice, the bits are the same.  "At once": the SMs hold all CTAs of the
// launch.  "A CTA an SM": the blocks of 256 W rows are more than two fifths of the SMs, and no more
// than the SMs.
//   1 to 32 rows   parts, 128 W rows a CTA, if at once;
//                  else, up to 16 rows, parts with 256 W rows a CTA, if that is at once;
//                  else whole, if a CTA an SM;
//                  else parts, 128 W rows a CTA.
//     SwiGLU       parts has 256 W rows a CTA.  Up to 16 rows whole if a CTA an SM and parts is not at
//                  once; above 16 whole if a CTA an SM; else parts.
//   33 to 128      whole, if the blocks of 256 W rows are more than the pairs and no more than the SMs.
//   33 and up      parts, if its tiles of 64 rows x 128 W rows are no more than the pairs, and K has two
//                  parts (up to 64 rows) or four.
//     SwiGLU       parts, if its tiles of 128 rows x 128 W rows are no more than the pairs in as many
//                  waves as the pair kernel would take and its CTAs no more than the SMs, K as above.
//   the rest       pair (as more than 65535 tiles of 128 W rows or rows of x do: a grid's limit); without
//                  SwiGLU with tiles of 128 columns where a wave of them, 0.6 of the other's time, makes
//                  up for their number.
// Measured, us, K = 4096 unless said otherwise, as parts / whole / pair with tiles of 128 columns / of 256:
//   1 to 32 rows   N = 4096, 24 rows 6.2 / 14.6 / 11.0 / 15.0; N = 12288 10.4 / 15.9 / 21.9 / 19.8.
//     not at once  one row, parts of 128 / of 256 / whole: N = 16384 15.7 / 12.1 / 16.0, N = 24576 19.9 / 18.0 /
//                  19.4, N = K = 8192 15.8 / 11.9 / -; 17 rows, N = 16384 17.1 / 18.2 / 16.5.
//     a CTA an SM  N = 24576, 24 rows 22.1 / - / 20.3; 48 CTAs, N = 12288, 32 rows 15.3 / 16.4 / 16.1, K = 8192, one
//                  row 20.2 / 22.1 / 25.8.
//     SwiGLU       F = 12288, 4 rows, at once, 18.4 / whole 19.7, 8 rows, not, 23.5 / 19.6; above 16 rows the
//                  sums are pulled: F = 8192, 24 rows, at once, 19.0 / 17.1.
//   whole          N = 24576, 64 rows 29.2 / 21.2 / - / 28.8, 128 rows 35.1 / 24.8 / - / 29.9; but N = 12288, one
//                  wave of the pairs, 128 rows 22.2 / 20.5 / 18.1 / 17.1.
//   parts          N = 4096, 128 rows, 64 tiles, 8.8 / 19.7 / 10.6 / 15.6, 256 rows, 128, 11.6 / 19.3 / 10.6 /
//                  15.7; N = 8192, 48 rows, 64, 9.1 / 16.0 / 11.3 / 15.7, 128 rows, 128, 12.3 / 20.1 / 11.7 / 16.1;
//                  K = 12288, N = 4096, 128 rows 15.8 / 44.3 / 22.4 / 34.3.  Parts to spread: K = 1024, one, 48
//                  rows 6.4 / 6.8 / 5.9 / 7.6; K = 2048, two, 48 rows 6.1 / - / 7.5 / -, 96 rows 8.0 / - / 7.5 / -.
//     SwiGLU       F = 4096, 128 rows 14.9 / 21.6 / - / 16.2; K = 12288 46.6 / 46.4 / - / 35.6.
//   pair           N = 4096, 400 rows - / - / 11.0 / 15.8, one wave of either; 768 rows 16.9 / 16.4, two and
//                  one; N = 6144, 1024 rows 23.6 / 26.7, three and two; N = 8192 29.6 / 27.4, four and two.
template <typename Act, bool g>
typename Act::Result choose_few(const Call& c, bool whole) {  // up to 32 rows
    if constexpr (g) {
        if (c.M <= 16)
            return whole && !at_once<16, 2, true, 2>(c, plan_of<16, 2>(c)) ? Act::template whole<g, 16>(c)
                                                                           : choose_ring<Act, g, 16, 2, 5, 3, 2>(c);
        return whole ? Act::template whole<g, 32>(c) : choose_ring<Act, g, 32, 2, 4, 2, 2>(c);
    } else {
        if (c.M > 16)
            return whole && !at_once<32, 1, false, 3>(c, plan_of<32, 1>(c)) ? Act::template whole<g, 32>(c)
                                                                            : choose_ring<Act, g, 32, 1, 8, 4, 3>(c);
        if (!at_once<16, 1, false, 3>(c, plan_of<16, 1>(c))) {
            // no ring of five stages: an SM holds one such CTA, and what fits in one of 256 W rows an
            // SM has fitted above in two of 128
            if (at_once<16, 2, false, 2>(c, plan_of<16, 2>(c))) return choose_ring<Act, g, 16, 2, 3, 3, 2>(c);
            if (whole) return Act::template whole<g, 16>(c);
        }
        return choose_ring<Act, g, 16, 1, 8, 4, 3>(c);
    }
}

template <typename Act, bool g>
typename Act::Result choose(const Call& c) {
    const int sms = c.dev.sms;
    const int64_t pairs = sms / 2;
    const int64_t small_m = (c.M + 127) / 128, small_n = (c.N + 127) / 128;
    const int64_t large_m = (c.M + 255) / 256, large_n = (c.N + 255) / 256;
    const int64_t waves = (large_m * large_n + pairs - 1) / pairs;
    const int64_t half_waves = (large_m * small_n + pairs - 1) / pairs;
    const int parts = parts_of(c.K).count;
    const int64_t ctas = parts * small_m * (g ? large_n : small_n);
    if (c.M <= 32 && small_n <= 65535) {
        const bool whole = large_n * 5 > 2 * sms && large_n <= sms;
        return choose_few<Act, g>(c, whole);
    }
    if (c.M > 32 && c.M <= 128 && large_n > pairs && large_n <= sms)
        return c.M <= 64 ? Act::template whole<g, 64>(c) : Act::template whole<g, 128>(c);
    if (c.M > 32 && small_m <= 65535 && small_n <= 65535 && parts >= (c.M <= 64 ? 2 : 4) &&
        (g ? small_m * small_n <= waves * pairs && ctas <= sms
           : static_cast<int64_t>((c.M + 63) / 64) * small_n <= pairs)) {
        if constexpr (g)
            return c.M <= 64 ? choose_ring<Act, g, 64, 2, 4, 2, 2>(c) : choose_ring<Act, g, 128, 2, 4, 4, 4>(c);
        else
            return c.M <= 64 ? choose_ring<Act, g, 64, 1, 6, 3, 3>(c) : choose_ring<Act, g, 128, 1, 6, 3, 3>(c);
    }
    if constexpr (!g)
        if (5 * half_waves < 8 * waves) return Act::template pair<g, 1>(c);
    return Act::template pair<g, 2>(c);
}

template <bool kSwiGLU>
bi_status launch_gemm(Call& c) {
    c.dev = bi::current_device_state();
    if (c.dev.index < 0) return BI_ERR_CUDA;
    return choose<Launch, kSwiGLU>(c);
}

bi_status check(const Call& c, int n_step) {
    if (c.M < 0) return BI_ERR_INVALID_ARG;
    if (c.N < n_step || c.N % n_step || c.K < 16 || (c.K & 15)) return BI_ERR_UNSUPPORTED_SHAPE;
    if (c.M > 0x7fffffff - 256 || c.N > 0x7fffffff - 256 || c.K > 0x7fffffff - 512)
        return BI_ERR_UNSUPPORTED_SHAPE;  // row, column and byte indices stay in int
    const int64_t spans = bi_fp8::spans_of(c.K);
    if ((c.M + 255) / 128 * spans > 0x7fffffffLL || (c.N + 255) / 128 * spans > 0x7fffffffLL)
        return BI_ERR_UNSUPPORTED_SHAPE;
    if (c.ld_x < c.K || c.ld_w < c.K) return BI_ERR_INVALID_ARG;
    if ((c.ld_x & 15) || (c.ld_w & 15)) return BI_ERR_MISALIGNED;
    return BI_OK;
}

template <bool kSwiGLU>
int32_t form_of(Call& c) {
    if (check(c, kSwiGLU ? 32 : 8) != BI_OK || c.M == 0) return 0;
    c.dev = bi::current_device_state();
    return c.dev.index < 0 ? 0 : choose<Name, kSwiGLU>(c);
}

}  // namespace

extern "C" int32_t bi_gemm_fp8_form(int32_t M, int32_t N, int32_t K, int32_t swiglu) {
    Call c{};
    c.M = M, c.N = N, c.K = K;
    c.ld_x = c.ld_w = K;
    return swiglu ? form_of<true>(c) : form_of<false>(c);
}

extern "C" bi_status bi_gemm_fp8(const void* x, const void* x_scales, const void* W,
                                 const void* W_scales, void* y, int32_t M, int32_t N, int32_t K,
                                 int64_t ld_x, int64_t ld_w, int64_t ld_y, cudaStream_t stream) {
    Call c{x, x_scales, W, W_scales, M, N, K, ld_x, ld_w, {y, ld_y, nullptr, 0}, stream, {}};
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
    Call c{x, x_scales, W_gu, W_gu_scales, M, 2 * F, K, ld_x, ld_w,
                 {h, ld_h, static_cast<uint8_t*>(h_scales), bi_fp8::spans_of(F)}, stream, {}};
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
