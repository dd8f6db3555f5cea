// fp4_gemm.cuh -- W4A4 product for prompts on the 5th-generation tensor cores
// (sm_100a):
//   y[m][n] = gx * gw * sum_k (x[m][k] * sx[m][k / B]) * (w[n][k] * sw[n][k / B])
// with both operands block-scaled E2M1 (fp4.cuh): tcgen05.mma kind::mxf4 (MXFP4,
// B = 32, E8M0) or kind::mxf4nvf4 (NVFP4, B = 16, E4M3).  The tensor cores apply
// the block scales, so nothing is decoded: codes and scale tiles go from global to
// shared memory by TMA, scales from there to tensor memory by tcgen05.cp;
// accumulators are binary32 in tensor memory.  gx * gw is applied in the epilogue.
//
// A cluster of two CTAs works on one tile of 256 tokens x NT weight rows
// (cta_group::2): each CTA stages its 128 tokens and half of the weight rows, and
// holds its 128 tokens' accumulators.  One CTA alone would have to write and read
// 12 KB of shared memory per 128-cycle MMA step (128 x 256 x 64), above the 128
// bytes per cycle the memory gives; the pair moves 8 KB per CTA and step.
//
// Tensor memory: two accumulators of NT columns and the scales of one stage (the
// MMAs and scale copies of one thread run in order).  At NT = 256 two accumulators
// and the scales do not fit, so they share the middle columns: the epilogue
// drains those first, and the next tile's MMAs start when they are free.
//
// Warp roles (12 warps, both CTAs unless said): 0 and 10 TMA producers; 1 tensor-memory
// allocation, scale copies and MMAs (first CTA); 2-9 epilogue (warp w reads lanes
// 32 (w % 4) .. + 31, every second chunk of 64 columns); 11 waits for the MMA issuer
// (first CTA).  Every mbarrier wait is bounded (fp4_mma.cuh).
#pragma once

#include "fp4_mma.cuh"

namespace w4 {

namespace fgemm {

namespace pair {

constexpr int kEpiWarps = 8;
constexpr int kEpiWarp0 = 2;
constexpr int kXWarp = kEpiWarp0 + kEpiWarps;
constexpr int kWaitWarp = kXWarp + 1;
constexpr int kWarps = kWaitWarp + 1;
constexpr int kThreads = kWarps * 32;
constexpr int CHUNK = 64;                // accumulator columns per epilogue step
constexpr uint32_t kSmemBudget = 225 * 1024 - kEpiWarps * OUT_BYTES;

template <int FMT, int NT>
struct Config {
    static constexpr int ST = Scales<FMT>::TILES;
    // 128-row scale groups a tile of NT rows touches.  NT is a multiple of 64: a tile
    // starts on column 0 or 2 of its first group's scales (an MMA's scale address must
    // be a multiple of two columns).
    static constexpr int GB = (NT + 64) / 128;
    static constexpr uint32_t B_BYTES = NT / 2 * (BK / 2);
    static constexpr uint32_t SF_BYTES = SF_TILE * ST;                      // one group, one stage
    static constexpr uint32_t STAGE_BYTES = A_BYTES + B_BYTES + (1 + GB) * SF_BYTES;   // of one CTA
    static constexpr int STAGES = (int)(kSmemBudget / STAGE_BYTES) < 8 ? (int)(kSmemBudget / STAGE_BYTES) : 8;
    static constexpr uint32_t SF_COLS = 4 * ST * (1 + GB);
    static constexpr uint32_t SF_COL0 = 512 - SF_COLS;
    static constexpr uint32_t ACC1 = NT < SF_COL0 - NT ? NT : SF_COL0 - NT;  // first column of accumulator 1
    static constexpr int OVERLAP = NT - (int)ACC1;                           // columns the accumulators share
    static_assert(NT % 64 == 0 && NT >= 2 * CHUNK && NT <= 256 && STAGES >= 3 && OVERLAP <= CHUNK, "tile");
};

template <int FMT, int NT>
struct Shared {
    using C = Config<FMT, NT>;
    uint8_t a[C::STAGES][A_BYTES];                 // 1024-byte aligned (swizzle atoms)
    uint8_t b[C::STAGES][C::B_BYTES];
    uint8_t out[kEpiWarps][OUT_BYTES];             // 1024-byte aligned
    uint8_t sfa[C::STAGES][C::ST][SF_TILE];
    uint8_t sfb[C::STAGES][C::GB][C::ST][SF_TILE];
    uint64_t full[C::STAGES], empty[C::STAGES];    // full: the first CTA's, for both CTAs' loads
    uint64_t acc_full[2], acc_empty[2];            // acc_empty: the first CTA's, for both CTAs' epilogues
    uint64_t mma_done;
    uint32_t tmem_base;
    int abort;
};

struct Params {
    const float *gx, *gw;          // global scales (NVFP4) or null
    Output out;
    int K;
    int tiles_m, tiles_n, tiles_k; // tiles_k: scale tiles along K
    int early_w;                   // the weights may be read before the previous kernel has completed
};

// Arrives on the barrier at this offset in both CTAs once the MMAs and copies
// issued so far have completed.
__device__ __forceinline__ void commit_pair(uint64_t *bar) {
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
                 ::"r"(smem_addr(bar)), "h"((uint16_t)3) : "memory");
}

// 2-D TMA load into this CTA's shared memory, bytes counted on a barrier of either CTA of the pair.
__device__ __forceinline__ void tma_load_pair(void *dst, const CUtensorMap *map, int c0, int c1, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 "
        "[%0], [%1, {%2, %3}], [%4];"
        ::"r"(smem_addr(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar) : "memory");
}

// This shared-memory address in the first CTA of the cluster.
__device__ __forceinline__ uint32_t in_first_cta(const void *p) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(smem_addr(p)));
    return r;
}

__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

// This word in the other CTA of the pair.
__device__ __forceinline__ void store_in_other_cta(volatile int *p, int v, uint32_t rank) {
    asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, %1;\n\t"
                 "st.shared::cluster.b32 [a], %2;\n\t}"
                 ::"r"(smem_addr(const_cast<int *>(p))), "r"(rank ^ 1u), "r"(v) : "memory");
}

// TMA: y leaves as TMA boxes (its rows start and end on 16 bytes).
template <int FMT, int NT, bool TMA>
__global__ void __launch_bounds__(kThreads, 1)
    gemm_kernel(const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap wmap,
                const __grid_constant__ CUtensorMap sxmap, const __grid_constant__ CUtensorMap swmap,
                const __grid_constant__ CUtensorMap ymap, const __grid_constant__ Params p) {
    using S = Shared<FMT, NT>;
    using C = Config<FMT, NT>;
    constexpr int STAGES = C::STAGES;
    extern __shared__ uint8_t smem_raw[];
    S &sh = *reinterpret_cast<S *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int pair0 = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    const int KT = (p.K + BK - 1) / BK;
    const int ntiles = p.tiles_m * p.tiles_n;
    volatile int *abort = &sh.abort;
    const unsigned long long limit = g_wait_limit_ns;

    if (threadIdx.x == 0) {
        sh.abort = 0;
        for (int i = 0; i < STAGES; i++) {
            mbar_init(&sh.full[i], 1);
            mbar_init(&sh.empty[i], 1);
        }
        for (int i = 0; i < 2; i++) {
            mbar_init(&sh.acc_full[i], 1);
            mbar_init(&sh.acc_empty[i], 2 * kEpiWarps);
        }
        mbar_init(&sh.mma_done, 1);
        fence_mbar_init();
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(smem_addr(&sh.tmem_base)), "r"(512u));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, sh.tmem_base, 0);
    if (warp == 0 || warp == kXWarp) {
        // ------------------------------ TMA producers ------------------------------
        // Warp 0 loads w, warp kXWarp x (one warp for both: 8192 x 9728 x 2560 NVFP4 81.7
        // us, two 77.6 us).  With early_w the weights of the first stages are on
        // the way while the previous kernel (which makes x) still runs.
        const bool is_w = warp == 0;
        if (!is_w || !p.early_w) pdl_wait_prior_grid();
        int it = 0;
        bool stop = false;
        for (int t = pair0; t < ntiles && !stop; t += pairs) {
            const int m0 = (t % p.tiles_m) * 2 * BM + (int)rank * BM, tn = t / p.tiles_m;
            const int n0 = tn * NT + (int)rank * (NT / 2);
            for (int kt = 0; kt < KT; kt++, it++) {
                const int s = it % STAGES;
                // (a wait's limit is not to run while the previous kernel does)
                if (it == STAGES) pdl_wait_prior_grid();
                if (it >= STAGES) pipe_wait(&sh.empty[s], ((it / STAGES) - 1) & 1, abort, limit);
                // after an abort nothing more is loaded: the stage may not be free
                stop = __any_sync(0xFFFFFFFFu, *abort != 0);
                if (stop) break;
                if (elect_one()) {
                    const uint32_t full = in_first_cta(&sh.full[s]);
                    // scale tiles are rows of 128 words; those past a row's last (read from the
                    // next group, or zeros past the end) are not used
                    if (is_w) {
                        if (rank == 0) mbar_arrive_expect_tx(&sh.full[s], 2 * C::STAGE_BYTES);
                        tma_load_pair(sh.b[s], &wmap, kt * (BK / 2), n0, full);
#pragma unroll
                        for (int g = 0; g < C::GB; g++)
                            tma_load_pair(sh.sfb[s][g], &swmap, 0, (tn * NT / 128 + g) * p.tiles_k + kt * C::ST, full);
                    } else {
                        tma_load_pair(sh.a[s], &xmap, kt * (BK / 2), m0, full);
                        tma_load_pair(sh.sfa[s], &sxmap, 0, (m0 / 128) * p.tiles_k + kt * C::ST, full);
                    }
                }
            }
        }
        // (work of no more stages than the ring holds comes here without having waited)
        pdl_wait_prior_grid();
        // no load may land and no commit arrive after this CTA has left: the first CTA
        // waits for both CTAs' loads, each for the MMAs' arrivals on its own barriers,
        // and both meet in the cluster barrier at the end
        if (rank == 0 && is_w) {
            // (after an abort a stage may lack the loads the other CTA or warp did not issue:
            // settle() at the end takes this wait's place)
            for (int i = max(0, it - STAGES); i < it && !*abort; i++)
                if (!mbar_wait_bounded(&sh.full[i % STAGES], (uint32_t)((i / STAGES) & 1))) *abort = 1;
        }
        for (int i = max(0, it - STAGES); i < it; i++)
            pipe_wait(&sh.empty[i % STAGES], (i / STAGES) & 1, abort, limit);
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------- MMA issuer -------------------------------
        // Warp kWaitWarp does its mbarrier waits and meets it at named barrier 1 once per
        // stage (an accumulator's wait comes before its tile's first stage): with one warp
        // that waits and issues, 2048 x 9728 x 2560 took 25.1 / 27.0 us (MXFP4 / NVFP4),
        // so 23.2 / 24.1.
        //
        // After an abort it issues on stages that hold anything, but frees none: the abort
        // flag is one CTA's, and freed stages would have the second CTA go on loading, with
        // bytes counted on barriers that the first no longer arms.  A barrier holds less than
        // 2^20 such bytes (27 fills of an NVFP4 stage of 256 rows); as it is, a stage is
        // filled at most once more: 2 STAGE_BYTES.  (The flag is read ahead of the issue and
        // used behind it: 512 x 2560 x 9728 MXFP4 10.8 -> 10.9 us, longer products as before;
        // a barrier that also reduces a flag of the waiter 11.0.)
        if (rank == 0) {
            int it = 0, lt = 0;
            const int steps = (p.K + 63) / 64;
            const uint32_t sfa = tmem + C::SF_COL0, sfb = sfa + 4 * C::ST;
            for (int t = pair0; t < ntiles; t += pairs, lt++) {
                const uint32_t acc = tmem + (lt & 1 ? C::ACC1 : 0u);
                const uint32_t shift = (uint32_t)(((t / p.tiles_m) * NT % 128) / 32);
                for (int kt = 0; kt < KT; kt++, it++) {
                    const int s = it % STAGES;
                    named_barrier_sync(1, 64);
                    const bool aborted = *abort != 0;   // set before the waiter's wait returned, if that expired
                    tc_fence_after();
                    if (elect_one()) {
                        const uint32_t a = codes_desc(smem_addr(sh.a[s])), b = codes_desc(smem_addr(sh.b[s]));
                        const uint32_t fa = scale_desc(smem_addr(sh.sfa[s])), fb = scale_desc(smem_addr(sh.sfb[s]));
#pragma unroll
                        for (int c = 0; c < C::ST; c++) {
                            copy_scales<2>(sfa + 4 * c, fa + c * (SF_TILE / 16));
#pragma unroll
                            for (int g = 0; g < C::GB; g++)
                                copy_scales<2>(sfb + 4 * (c * C::GB + g), fb + (g * C::ST + c) * (SF_TILE / 16));
                        }
#pragma unroll
                        for (int j = 0; j < BK / 64; j++) {
                            const int c = j / Scales<FMT>::STEPS_PER_TILE;
                            if (kt * (BK / 64) + j < steps)
                                mma_fp4<FMT, 2>(acc, a + 2 * j, b + 2 * j, idesc<FMT>(2 * BM, NT) | scale_ids<FMT>(j),
                                                sfa + 4 * c, sfb + 4 * c * C::GB + shift, (kt | j) ? 1u : 0u);
                        }
                        if (!aborted) commit_pair(&sh.empty[s]);
                        if (kt == KT - 1) commit_pair(&sh.acc_full[lt & 1]);
                    }
                    __syncwarp();
                }
            }
            // tensor memory is released after the cluster barrier: every MMA and copy
            // issued must have completed by then (also after an abort)
            if (elect_one())
                asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];"
                             ::"r"(smem_addr(&sh.mma_done)) : "memory");
            __syncwarp();
            if (!mbar_wait_bounded(&sh.mma_done, 0)) *abort = 1;
        }
        __syncwarp();
    } else if (warp == kWaitWarp) {
        // ------------------- waits on behalf of the MMA issuer -------------------
        if (rank == 0) {
            pdl_wait_prior_grid();   // a wait's limit is not to run while the previous kernel does
            int it = 0, lt = 0;
            for (int t = pair0; t < ntiles; t += pairs, lt++) {
                if (C::OVERLAP > 0) {   // the columns shared with the previous tile's accumulator are drained
                    if (lt >= 1) pipe_wait(&sh.acc_empty[(lt - 1) & 1], ((lt - 1) >> 1) & 1, abort, limit);
                } else {                // this accumulator is
                    if (lt >= 2) pipe_wait(&sh.acc_empty[lt & 1], ((lt >> 1) - 1) & 1, abort, limit);
                }
                for (int kt = 0; kt < KT; kt++, it++) {
                    // on expiry (abort) both warps still meet
                    pipe_wait(&sh.full[it % STAGES], (it / STAGES) & 1, abort, limit);
                    __syncwarp();
                    named_barrier_sync(1, 64);
                }
            }
        }
        __syncwarp();
    } else {
        // -------------------------------- epilogue --------------------------------
        const int q = warp & 3, half = (warp - kEpiWarp0) >> 2;
        pdl_wait_prior_grid();   // y and the global scales belong to the previous kernel until then
        const Factor fac(p.gx, p.gw);
        int lt = 0;
        for (int t = pair0; t < ntiles; t += pairs, lt++) {
            const int b = lt & 1;
            const int m0 = (t % p.tiles_m) * 2 * BM + (int)rank * BM + q * 32;
            const int n0 = (t / p.tiles_m) * NT;
            // on expiry (abort) the accumulator is garbage, but the warp stays together
            pipe_wait(&sh.acc_full[b], (lt >> 1) & 1, abort, limit);
            __syncwarp();
            tc_fence_after();
            const uint32_t acc = tmem + ((uint32_t)(q * 32) << 16) + (b ? C::ACC1 : 0u);
            const uint32_t empty = in_first_cta(&sh.acc_empty[b]);
            // shared columns first: the last of accumulator 0, the first of accumulator 1
#pragma unroll 1
            for (int i = half; i < NT / CHUNK; i += 2) {
                const int c = b ? i : NT / CHUNK - 1 - i;
                float v[CHUNK];
                tmem_ld64(acc + (uint32_t)(c * CHUNK), v);
                if (C::OVERLAP > 0 ? i == half : i + 2 >= NT / CHUNK) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) arrive_cluster(empty);
                }
                apply_factor(fac, v);
                store_rows<TMA>(p.out, &ymap, sh.out[warp - kEpiWarp0], m0, n0 + c * CHUNK, v);
            }
        }
        if (TMA) store_rows_done();
        __syncwarp();
    }

    tc_fence_before();
    __syncthreads();
    // After an abort in either CTA no barrier tells when the loads into both, which count on
    // the first's barriers, and the arrivals of commits have landed: neither leaves before
    // they must have.
    if (threadIdx.x == 0 && *abort) store_in_other_cta(abort, 1, rank);
    __syncwarp();
    cluster_sync();
    if (*abort) {
        if (threadIdx.x == 0) settle();
        __syncthreads();
        cluster_sync();
    }
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u));
    }
}

}  // namespace pair

}  // namespace fgemm

}  // namespace w4
