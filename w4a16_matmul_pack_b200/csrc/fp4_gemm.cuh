// fp4_gemm.cuh -- W4A4 product on the 5th-generation tensor cores (sm_100a):
//   y[m][n] = gx * gw * sum_k (x[m][k] * sx[m][k / B]) * (w[n][k] * sw[n][k / B])
// with both operands block-scaled E2M1 (fp4.cuh): tcgen05.mma kind::mxf4 (MXFP4,
// B = 32, E8M0) or kind::mxf4nvf4 (NVFP4, B = 16, E4M3).  The tensor cores apply
// the block scales, so nothing is decoded: codes go from global to shared memory
// by TMA, scale tiles (512 bytes, 128 rows x 4 scales) by bulk copies and from
// there to tensor memory by tcgen05.cp; accumulators are binary32 in tensor
// memory.  gx * gw is applied in the epilogue.
//
// Tile: 128 rows of the operand A (tensor-memory lanes) x NT rows of B x 256 k
// per stage.  SWAP = false (prompts): A is x, so a thread of the epilogue holds
// part of an output row.  SWAP = true (few tokens): A is w, so that 128 x NT
// wastes no work on missing tokens; lanes then run along n.
//
// Warp roles (6 warps): 0 TMA producer; 1 tensor-memory allocation, scale copies
// and MMAs (one lane); 2-5 epilogue (warp w reads lanes 32 (w % 4) .. + 31).
// Persistent CTAs, one per SM; two accumulators, so the epilogue of a tile
// overlaps the next tile's MMAs.  Every mbarrier wait is bounded (common.cuh).
#pragma once

#include "fp4.cuh"

namespace w4 {

namespace fgemm {

constexpr int BM = 128;
constexpr int BK = 256;                 // k per stage: one 128-byte swizzle row of codes
constexpr int STAGES = 4;
constexpr int kWarps = 6;
constexpr int kThreads = kWarps * 32;
constexpr int kEpiWarps = 4;
constexpr uint32_t A_BYTES = BM * (BK / 2);

enum { OUT_BF16 = W4_TYPE_BF16, OUT_F16 = W4_TYPE_F16, OUT_F32 = W4_TYPE_F32 };

template <int FMT> struct Scales;
// TILES scale tiles along K per stage; STEP_TILES(j): the tile of MMA step j (64 k)
template <> struct Scales<W4_FMT_MXFP4> { static constexpr int TILES = 2, STEPS_PER_TILE = 2; };
template <> struct Scales<W4_FMT_NVFP4> { static constexpr int TILES = 4, STEPS_PER_TILE = 1; };

constexpr uint32_t pow2_at_least(uint32_t v) {
    uint32_t p = 32;
    while (p < v) p *= 2;
    return p;
}

template <int FMT, int NT>
struct Config {
    static constexpr int ST = Scales<FMT>::TILES;
    static constexpr int GB = (NT + 127) / 128;                 // 128-row groups of a B tile
    static constexpr uint32_t B_BYTES = NT * (BK / 2);
    static constexpr uint32_t SF_TILE = 512;
    static constexpr uint32_t SF_COLS = 4 * ST * (1 + GB);      // tensor-memory columns of a stage's scales
    static constexpr uint32_t ACC_COLS = NT < 32 ? 32 : NT;
    static constexpr uint32_t SF_COL0 = 2 * ACC_COLS;
    static constexpr uint32_t TMEM_COLS = pow2_at_least(SF_COL0 + STAGES * SF_COLS);
    static_assert(TMEM_COLS <= 512, "tensor memory");
    // Instruction descriptor: A and B E2M1 (bits 7-9, 10-11), N >> 3 at bit 17,
    // scale type at bit 23 (1: E8M0, 0: E4M3), M >> 7 at bit 27, both K-major.
    // The scale ids (bits 4-5 of B, 29-30 of A) select the bytes of a scale word.
    static constexpr uint32_t IDESC = (1u << 7) | (1u << 10) | ((uint32_t)(NT >> 3) << 17) |
                                      ((FMT == W4_FMT_MXFP4 ? 1u : 0u) << 23) | ((uint32_t)(BM >> 7) << 27);
};

template <int FMT, int NT>
struct Shared {
    using C = Config<FMT, NT>;
    uint8_t a[STAGES][A_BYTES];                              // 1024-byte aligned (swizzle atoms)
    uint8_t b[STAGES][C::B_BYTES];
    uint8_t sfa[STAGES][C::ST][C::SF_TILE];
    uint8_t sfb[STAGES][C::ST][C::GB][C::SF_TILE];
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

__device__ __forceinline__ uint64_t sw128_desc(uint32_t saddr) {
    uint64_t d = (uint64_t)((saddr & 0x3FFFFu) >> 4);
    d |= (uint64_t)1 << 16;            // leading byte offset (unused for this layout)
    d |= (uint64_t)(1024 >> 4) << 32;  // stride byte offset: 8-row atoms
    d |= (uint64_t)1 << 46;            // version
    d |= (uint64_t)2 << 61;            // SWIZZLE_128B
    return d;
}

// A scale tile: 32 rows of 16 bytes, no swizzle, 8-row groups 128 bytes apart.
__device__ __forceinline__ uint64_t scale_desc(uint32_t saddr) {
    uint64_t d = (uint64_t)((saddr & 0x3FFFFu) >> 4);
    d |= (uint64_t)(128 >> 4) << 16;
    d |= (uint64_t)(128 >> 4) << 32;
    d |= (uint64_t)1 << 46;
    return d;
}

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

__device__ __forceinline__ void copy_scales(uint32_t tmem, uint64_t desc) {
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
}

template <int FMT>
__device__ __forceinline__ void mma_fp4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                        uint32_t accumulate) {
    if constexpr (FMT == W4_FMT_MXFP4)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}"
            ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate) : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}"
            ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate) : "memory");
}

__device__ __forceinline__ void mma_commit(uint64_t *bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];"
                 ::"r"(smem_addr(bar)) : "memory");
}

__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 ::"r"(smem_addr(dst)), "l"(src), "r"(bytes), "r"(smem_addr(bar)) : "memory");
}

#define W4_FP4_TMEM_LD16(taddr, v)                                                                          \
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 "                                                  \
                 "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"                           \
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),       \
                   "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),   \
                   "=r"(v[14]), "=r"(v[15])                                                                  \
                 : "r"(taddr))

// gx * gw: one binary32 factor when it is a normal number or zero, else applied
// in binary64 per value (the factor may leave binary32's range when the result
// does not).
struct Factor {
    float f;
    double d;
    bool wide;
    __device__ __forceinline__ Factor(const float *ga, const float *gb) {
        d = (ga ? (double)__ldg(ga) : 1.0) * (gb ? (double)__ldg(gb) : 1.0);
        f = (float)d;
        const double m = fabs(d);
        wide = !(d == 0.0 || (m >= 0x1p-126 && m < 0x1p128));
    }
    __device__ __forceinline__ float apply(float acc) const {
        return wide ? (float)((double)acc * d) : acc * f;
    }
};

__device__ __forceinline__ void store_one(void *y, size_t i, float v, int type) {
    if (type == OUT_BF16) reinterpret_cast<__nv_bfloat16 *>(y)[i] = __float2bfloat16_rn(v);
    else if (type == OUT_F16) reinterpret_cast<__half *>(y)[i] = __float2half_rn(v);
    else reinterpret_cast<float *>(y)[i] = v;
}

template <int FMT, int NT, bool SWAP>
__global__ void __launch_bounds__(kThreads, 1) gemm_kernel(const __grid_constant__ CUtensorMap amap,
                                                            const __grid_constant__ CUtensorMap bmap, const Params p) {
    using S = Shared<FMT, NT>;
    using C = Config<FMT, NT>;
    extern __shared__ uint8_t smem_raw[];
    S &sh = *reinterpret_cast<S *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int KT = (p.K + BK - 1) / BK;
    const int ntiles = p.tiles_a * p.tiles_b;
    volatile int *abort = &sh.abort;

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
    const uint32_t tmem = sh.tmem_base;
    // x may be the previous kernel's output (programmatic dependent launch)
    pdl_wait_prior_grid();

    if (warp == 0) {
        // ------------------------------ TMA producer ------------------------------
        if (lane == 0) {
            int it = 0;
            for (int t = blockIdx.x; t < ntiles && !*abort; t += gridDim.x) {
                const int ta = t % p.tiles_a, tb = t / p.tiles_a;
                const int groups_b = min(C::GB, (p.rows_b + 127) / 128 - tb * NT / 128);
                for (int kt = 0; kt < KT; kt++, it++) {
                    const int s = it % STAGES;
                    if (it >= STAGES) mbar_wait(&sh.empty[s], ((it / STAGES) - 1) & 1, abort);
                    if (*abort) break;
                    // scale tiles that exist in this stage (the last one of a row may be cut)
                    const int nt = min(C::ST, p.tiles_k - kt * C::ST);
                    mbar_arrive_expect_tx(&sh.full[s],
                                          A_BYTES + C::B_BYTES + (uint32_t)(nt * (1 + groups_b)) * C::SF_TILE);
                    tma_load_2d(sh.a[s], &amap, kt * (BK / 2), ta * BM, &sh.full[s]);
                    tma_load_2d(sh.b[s], &bmap, kt * (BK / 2), tb * NT, &sh.full[s]);
                    bulk_load(sh.sfa[s], p.sfa + ((size_t)ta * p.tiles_k + kt * C::ST) * C::SF_TILE,
                              (uint32_t)nt * C::SF_TILE, &sh.full[s]);
                    for (int g = 0; g < groups_b; g++)
                        for (int c = 0; c < nt; c++)
                            bulk_load(sh.sfb[s][c][g],
                                      p.sfb + ((size_t)(tb * NT / 128 + g) * p.tiles_k + kt * C::ST + c) * C::SF_TILE,
                                      C::SF_TILE, &sh.full[s]);
                }
            }
            drain_ring(sh.full, STAGES, it);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------- MMA issuer -------------------------------
        if (lane == 0) {
            int it = 0, lt = 0;
            const int steps = (p.K + 63) / 64;
            for (int t = blockIdx.x; t < ntiles; t += gridDim.x, lt++) {
                const int b = lt & 1;
                const uint32_t acc = tmem + (uint32_t)b * C::ACC_COLS;
                // a B tile narrower than 128 rows starts inside its scale tile
                const uint32_t sfb_shift = (uint32_t)(((t / p.tiles_a) * NT % 128) / 32);
                if (lt >= 2) mbar_wait(&sh.acc_empty[b], ((lt >> 1) - 1) & 1, abort);
                tc_fence_after();
                for (int kt = 0; kt < KT; kt++, it++) {
                    const int s = it % STAGES;
                    mbar_wait(&sh.full[s], (it / STAGES) & 1, abort);
                    if (*abort) break;
                    tc_fence_after();
                    // the stage's own scale columns: free once the stage is (its MMAs have completed)
                    const uint32_t sfa = tmem + C::SF_COL0 + (uint32_t)s * C::SF_COLS, sfb = sfa + 4 * C::ST;
                    const uint32_t a0 = smem_addr(sh.a[s]), b0 = smem_addr(sh.b[s]);
                    for (int c = 0; c < C::ST; c++) {
                        if (kt * C::ST + c >= p.tiles_k) break;
                        copy_scales(sfa + 4 * c, scale_desc(smem_addr(sh.sfa[s][c])));
                        for (int g = 0; g < C::GB; g++)
                            copy_scales(sfb + 4 * (c * C::GB + g), scale_desc(smem_addr(sh.sfb[s][c][g])));
                    }
#pragma unroll
                    for (int j = 0; j < BK / 64; j++) {
                        if (kt * (BK / 64) + j >= steps) break;
                        const int c = j / Scales<FMT>::STEPS_PER_TILE;
                        const uint32_t id = Scales<FMT>::STEPS_PER_TILE == 2 ? (uint32_t)(j & 1) * 2u : 0u;
                        mma_fp4<FMT>(acc, sw128_desc(a0 + 32 * j), sw128_desc(b0 + 32 * j),
                                     C::IDESC | (id << 4) | (id << 29), sfa + 4 * c, sfb + 4 * c * C::GB + sfb_shift,
                                     (kt | j) ? 1u : 0u);
                    }
                    mma_commit(&sh.empty[s]);
                }
                if (*abort) break;
                mma_commit(&sh.acc_full[b]);
            }
            // tensor memory is released after the final barrier: every MMA and copy
            // this thread issued must have completed by then (also after an abort)
            mma_commit(&sh.mma_done);
            mbar_wait_bounded(&sh.mma_done, 0);
        }
        __syncwarp();
    } else {
        // -------------------------------- epilogue --------------------------------
        const int q = warp & 3;
        const Factor fac(p.ga, p.gb);
        int lt = 0;
        for (int t = blockIdx.x; t < ntiles; t += gridDim.x, lt++) {
            const int b = lt & 1;
            const int ra = (t % p.tiles_a) * BM + q * 32 + lane;   // this lane's row of A
            const int rb0 = (t / p.tiles_a) * NT;
            // on expiry (abort) the accumulator is garbage, but the warp stays together
            mbar_wait(&sh.acc_full[b], (lt >> 1) & 1, abort);
            __syncwarp();
            tc_fence_after();
            for (int c = 0; c < NT / 16; c++) {
                uint32_t v[16];
                W4_FP4_TMEM_LD16(tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(b * C::ACC_COLS + c * 16), v);
                asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
                for (int j = 0; j < 16; j++) {
                    const int rb = rb0 + c * 16 + j;
                    if (ra < p.rows_a && rb < p.rows_b) {
                        const size_t i = SWAP ? (size_t)rb * p.ldy + ra : (size_t)ra * p.ldy + rb;
                        store_one(p.y, i, fac.apply(__uint_as_float(v[j])), p.out_type);
                    }
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

}  // namespace fgemm

}  // namespace w4
