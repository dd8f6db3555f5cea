// fp4_skinny.cuh -- W4A4 product with one CTA per tile (sm_100a): few tokens.
// (see fp4_mma.cuh for the instructions both product kernels use)
//
// Tile: 128 rows of w (the operand A, tensor-memory lanes) x NT tokens (B) x 256 k
// per stage: no work is wasted on missing tokens, and the lanes of an epilogue
// store run along a row of y.
//
// Warp roles (6 warps): 0 TMA producer; 1 tensor-memory allocation, scale copies
// and MMAs (one lane); 2-5 epilogue (warp w reads lanes 32 (w % 4) .. + 31).
// Persistent CTAs, one per SM; two accumulators, so the epilogue of a tile
// overlaps the next tile's MMAs.  Every mbarrier wait is bounded (common.cuh).
#pragma once

#include "fp4_mma.cuh"

namespace w4 {

namespace fgemm {

namespace skinny {

constexpr int STAGES = 4;
constexpr int kWarps = 6;
constexpr int kThreads = kWarps * 32;
constexpr int kEpiWarps = 4;

template <int FMT, int NT>
struct Config {
    static constexpr int ST = Scales<FMT>::TILES;
    static constexpr int GB = (NT + 127) / 128;                 // 128-row groups of a B tile
    static constexpr uint32_t B_BYTES = NT * (BK / 2);
    static constexpr uint32_t SF_COLS = 4 * ST * (1 + GB);      // tensor-memory columns of a stage's scales
    static constexpr uint32_t ACC_COLS = NT < 32 ? 32 : NT;
    static constexpr uint32_t SF_COL0 = 2 * ACC_COLS;
    static constexpr uint32_t TMEM_COLS = pow2_at_least(SF_COL0 + SF_COLS);
    static_assert(TMEM_COLS <= 512, "tensor memory");
};

template <int FMT, int NT>
struct Shared {
    using C = Config<FMT, NT>;
    uint8_t a[STAGES][A_BYTES];                              // 1024-byte aligned (swizzle atoms)
    uint8_t b[STAGES][C::B_BYTES];
    uint8_t sfa[STAGES][C::ST][SF_TILE];
    uint8_t sfb[STAGES][C::GB][C::ST][SF_TILE];
    uint64_t full[STAGES], empty[STAGES];
    uint64_t acc_full[2], acc_empty[2];
    uint64_t mma_done;
    uint32_t tmem_base;
    int abort;
};

struct Params {
    const uint8_t *sfa, *sfb;      // scale tiles of A and B
    const float *ga, *gb;          // global scales (NVFP4) or null
    void *y;
    long long ldy;
    int rows_a, rows_b, K;
    int tiles_a, tiles_b, tiles_k; // tiles_k: scale tiles along K
    int out_type;
    int early_w;                   // the weights may be read before the previous kernel has completed
};

template <int FMT, int NT>
__global__ void __launch_bounds__(kThreads, 1) gemm_kernel(const __grid_constant__ CUtensorMap amap,
                                                            const __grid_constant__ CUtensorMap bmap,
                                                            const __grid_constant__ Params p) {
    using S = Shared<FMT, NT>;
    using C = Config<FMT, NT>;
    extern __shared__ uint8_t smem_raw[];
    S &sh = *reinterpret_cast<S *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int KT = (p.K + BK - 1) / BK;
    const int ntiles = p.tiles_a * p.tiles_b;
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
            mbar_init(&sh.acc_empty[i], kEpiWarps);
        }
        mbar_init(&sh.mma_done, 1);
        fence_mbar_init();
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(smem_addr(&sh.tmem_base)), "r"(C::TMEM_COLS));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, sh.tmem_base, 0);
    // x may be the previous kernel's output (programmatic dependent launch)
    pdl_wait_prior_grid();

    if (warp == 0) {
        // ------------------------------ TMA producer ------------------------------
        int it = 0;
        bool stop = false;
        for (int t = blockIdx.x; t < ntiles && !stop; t += gridDim.x) {
            const int ta = t % p.tiles_a, tb = t / p.tiles_a;
            const int groups_b = min(C::GB, (p.rows_b + 127) / 128 - tb * NT / 128);
            for (int kt = 0; kt < KT; kt++, it++) {
                const int s = it % STAGES;
                if (it >= STAGES) pipe_wait(&sh.empty[s], ((it / STAGES) - 1) & 1, abort, limit);
                // after an abort nothing more is loaded: the stage may not be free
                stop = __any_sync(0xFFFFFFFFu, *abort != 0);
                if (stop) break;
                // scale tiles that exist in this stage (the last one of a row may be cut)
                const int nt = min(C::ST, p.tiles_k - kt * C::ST);
                if (elect_one()) {
                    mbar_arrive_expect_tx(&sh.full[s],
                                          A_BYTES + C::B_BYTES + (uint32_t)(nt * (1 + groups_b)) * SF_TILE);
                    tma_load_2d(sh.a[s], &amap, kt * (BK / 2), ta * BM, &sh.full[s]);
                    tma_load_2d(sh.b[s], &bmap, kt * (BK / 2), tb * NT, &sh.full[s]);
                    bulk_load(sh.sfa[s], p.sfa + ((size_t)ta * p.tiles_k + kt * C::ST) * SF_TILE,
                              (uint32_t)nt * SF_TILE, &sh.full[s]);
                    for (int g = 0; g < groups_b; g++)
                        bulk_load(sh.sfb[s][g],
                                  p.sfb + ((size_t)(tb * NT / 128 + g) * p.tiles_k + kt * C::ST) * SF_TILE,
                                  (uint32_t)nt * SF_TILE, &sh.full[s]);
                }
            }
        }
        drain_ring(sh.full, STAGES, it);
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------- MMA issuer -------------------------------
        int it = 0, lt = 0;
        bool stop = false;
        const int steps = (p.K + 63) / 64;
        for (int t = blockIdx.x; t < ntiles && !stop; t += gridDim.x, lt++) {
            const uint32_t acc = tmem + (uint32_t)(lt & 1) * C::ACC_COLS;
            if (lt >= 2) pipe_wait(&sh.acc_empty[lt & 1], ((lt >> 1) - 1) & 1, abort, limit);
            for (int kt = 0; kt < KT; kt++, it++) {
                const int s = it % STAGES;
                pipe_wait(&sh.full[s], (it / STAGES) & 1, abort, limit);
                stop = __any_sync(0xFFFFFFFFu, *abort != 0);
                if (stop) break;
                tc_fence_after();
                if (elect_one()) {
                    const uint32_t sfa = tmem + C::SF_COL0, sfb = sfa + 4 * C::ST;
                    const uint32_t a = codes_desc(smem_addr(sh.a[s])), b = codes_desc(smem_addr(sh.b[s]));
                    const uint32_t fa = scale_desc(smem_addr(sh.sfa[s])), fb = scale_desc(smem_addr(sh.sfb[s]));
#pragma unroll
                    for (int c = 0; c < C::ST; c++) {
                        if (kt * C::ST + c < p.tiles_k) {
                            copy_scales<1>(sfa + 4 * c, fa + c * (SF_TILE / 16));
#pragma unroll
                            for (int g = 0; g < C::GB; g++)
                                copy_scales<1>(sfb + 4 * (c * C::GB + g), fb + (g * C::ST + c) * (SF_TILE / 16));
                        }
                    }
#pragma unroll
                    for (int j = 0; j < BK / 64; j++) {
                        const int c = j / Scales<FMT>::STEPS_PER_TILE;
                        if (kt * (BK / 64) + j < steps)
                            mma_fp4<FMT, 1>(acc, a + 2 * j, b + 2 * j, idesc<FMT>(BM, NT) | scale_ids<FMT>(j),
                                            sfa + 4 * c, sfb + 4 * c * C::GB, (kt | j) ? 1u : 0u);
                    }
                    mma_commit(&sh.empty[s]);
                    if (kt == KT - 1) mma_commit(&sh.acc_full[lt & 1]);
                }
                __syncwarp();
            }
        }
        // tensor memory is released after the final barrier: every MMA and copy
        // issued must have completed by then (also after an abort)
        if (elect_one()) mma_commit(&sh.mma_done);
        __syncwarp();
        mbar_wait_bounded(&sh.mma_done, 0);
        __syncwarp();
    } else {
        // -------------------------------- epilogue --------------------------------
        const int q = warp & 3;
        const Factor fac(p.ga, p.gb);
        int lt = 0;
        for (int t = blockIdx.x; t < ntiles; t += gridDim.x, lt++) {
            const int b = lt & 1;
            const int n = (t % p.tiles_a) * BM + q * 32 + lane;    // this lane's row of w
            // on expiry (abort) the accumulator is garbage, but the warp stays together
            pipe_wait(&sh.acc_full[b], (lt >> 1) & 1, abort, limit);
            __syncwarp();
            tc_fence_after();
            for (int c = 0; c < NT / 16; c++) {
                uint32_t r[16];
                W4_FP4_TMEM_LD16(tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(b * C::ACC_COLS + c * 16), r);
                asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
                float v[16];
#pragma unroll
                for (int j = 0; j < 16; j++) v[j] = __uint_as_float(r[j]);
                apply_factor(fac, v);
                if (n >= p.rows_a) continue;
                const int m0 = (t / p.tiles_a) * NT + c * 16, count = min(16, p.rows_b - m0);
#pragma unroll
                for (int j = 0; j < 16; j++) {
                    if (j >= count) break;
                    const size_t i = (size_t)(m0 + j) * p.ldy + n;
                    if (p.out_type == OUT_F32) reinterpret_cast<float *>(p.y)[i] = v[j];
                    else reinterpret_cast<uint16_t *>(p.y)[i] = (uint16_t)pack16(v[j], v[j], p.out_type);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.acc_empty[b]);
        }
        __syncwarp();
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::TMEM_COLS));
    }
}

}  // namespace skinny

}  // namespace fgemm

}  // namespace w4
