// fp4_skinny.cuh -- W4A4 product for few tokens and for small outputs (sm_100a),
// one CTA per tile and slice of K (fp4_gemm.cuh: the instructions and the formula).
//
// Tile: 128 rows of w (the operand A, tensor-memory lanes) x NT tokens (B) x 256 k
// per stage: no work is wasted on missing tokens, and the lanes of an epilogue
// store run along a row of y.  Such a product streams weights: what counts is how
// many SMs load at once and how soon the first byte arrives.
//   - A few tiles do not fill the GPU, so the K of a tile is shared out to the S CTAs
//     of a cluster.  Each sends the partial sums of NT / S tokens to each of the others
//     through distributed shared memory and adds those of its own tokens in the order
//     of the slices (deterministic, no workspace).
//   - With W4_LAUNCH_PDL the first stages' weights are on their way while the previous
//     kernel (the norm that makes x) still runs.
//   - Up to 16 tokens are quantised here (T: the type of x): every CTA needs a slice of x
//     small enough to encode while its weights arrive.  One token, 2560 x 9728 MXFP4: 6.0
//     us, as two launches 6.6; nine tokens, 9728 x 2560 NVFP4 (two divisions per 16
//     values, in every CTA): 8.6 us, as two launches 7.4, but the second launch costs the
//     host 3.7 us.
//
// Warp roles: 0 TMA producer; 1 tensor-memory allocation, scale copies and MMAs; 2-5
// epilogue (warp w reads lanes 32 (w % 4) .. + 31); with x to quantise 2-7 do that
// first (one token MXFP4 / nine NVFP4 as above: four warps 5.9 / 9.2 us, six 6.0 / 8.8,
// twelve 6.6 / 8.7, before the last steps).  Every mbarrier wait is bounded (fp4_mma.cuh).
#pragma once

#include "fp4_mma.cuh"

namespace w4 {

namespace fgemm {

namespace skinny {

constexpr int kEpiWarp0 = 2, kEpiWarps = 4;
constexpr int kMaxSplit = 8;
constexpr int kQuantWarps = 6;   // warps kEpiWarp0 on

struct Quantised {};   // T of an x that is 4-bit already
template <typename T> constexpr bool kFused = true;
template <> constexpr bool kFused<Quantised> = false;
template <typename T> constexpr int kThreads = 32 * (kEpiWarp0 + (kFused<T> ? kQuantWarps : kEpiWarps));

template <int FMT, int NT>
struct Config {
    static constexpr int ST = Scales<FMT>::TILES;
    static constexpr uint32_t B_BYTES = NT * (BK / 2);
    static constexpr uint32_t STAGE_BYTES = A_BYTES + B_BYTES + 2 * ST * SF_TILE;
    static constexpr uint32_t RED_BYTES = NT * BM * 4;                      // partial sums of NT / S tokens x S slices
    // two CTAs per SM where the partial sums are small
    static constexpr uint32_t BUDGET = NT <= 32 ? 112 * 1024 : 224 * 1024;
    static constexpr int STAGES = (int)((BUDGET - RED_BYTES - 2048) / STAGE_BYTES) < 8
                                      ? (int)((BUDGET - RED_BYTES - 2048) / STAGE_BYTES) : 8;
    static constexpr uint32_t SF_COLS = 4 * ST * 2;                         // scales of w and of x, one stage
    static constexpr uint32_t ACC_COLS = NT < 32 ? 32 : NT;
    static constexpr uint32_t TMEM_COLS = pow2_at_least(ACC_COLS + SF_COLS);
    static_assert(NT % 16 == 0 && NT <= 128 && STAGES >= 3 && TMEM_COLS <= 512, "tile");
};

template <int FMT, int NT>
struct Shared {
    using C = Config<FMT, NT>;
    uint8_t a[C::STAGES][A_BYTES];                 // 1024-byte aligned (swizzle atoms)
    uint8_t b[C::STAGES][C::B_BYTES];
    uint8_t sfa[C::STAGES][C::ST][SF_TILE];
    uint8_t sfb[C::STAGES][C::ST][SF_TILE];
    float red[NT * BM];                            // [slice][token of this CTA][row of w]
    uint64_t full[C::STAGES], empty[C::STAGES];
    uint64_t acc_full, mma_done;
    uint32_t tmem_base;
    int abort;
};

struct Params {
    const uint8_t *sfw, *sfx;      // scale tiles
    const float *gw, *gx;          // global scales (NVFP4) or null
    void *y;
    long long ldy;
    int N, M, K;
    int tiles_n, tiles_k;          // tiles_k: scale tiles along K
    int splits;                    // CTAs of a cluster: slices of K
    int out_type;
    int early_w;                   // the weights may be read before the previous kernel has completed
    const void *x;                 // x to quantise: rows ldx values apart
    long long ldx;
    int ceil_rule;
    int *d_status;
    uint32_t inv_m;                // ceil(2^32 / M) (M > 1): (i * inv_m) >> 32 = i / M below 2^28
};

// The first `count` of n values of consecutive tokens, one column of y per lane.
template <int n>
__device__ __forceinline__ void store_column(const Params &p, int m, int col, int count, const float (&v)[n]) {
    const size_t at = (size_t)m * p.ldy + col;
    if (p.out_type == OUT_F32) {
        float *o = reinterpret_cast<float *>(p.y) + at;
#pragma unroll
        for (int j = 0; j < n; j++, o += p.ldy)
            if (j < count) *o = v[j];
    } else {
        uint16_t *o = reinterpret_cast<uint16_t *>(p.y) + at;
#pragma unroll
        for (int j = 0; j < n; j += 2) {
            const uint32_t w = pack16(v[j], v[j + 1 < n ? j + 1 : j], p.out_type);
            if (j < count) *o = (uint16_t)w;
            o += p.ldy;
            if (j + 1 < count) *o = (uint16_t)(w >> 16);
            o += p.ldy;
        }
    }
}

// Tokens first .. first + own - 1 of column n0 + row: the slices' partial sums in order.
template <int n>
__device__ __forceinline__ void add_slices(const Params &p, const Factor &fac, const float *red, int own, int first,
                                           int n0, int row) {
#pragma unroll 1
    for (int i = 0; i < own && first + i < p.M; i += n) {
        float v[n];
#pragma unroll
        for (int j = 0; j < n; j++) v[j] = red[(i + j) * BM + row];
#pragma unroll 1
        for (int k = 1; k < p.splits; k++)
#pragma unroll
            for (int j = 0; j < n; j++) v[j] += red[(k * own + i + j) * BM + row];
        apply_factor(fac, v);
        store_column(p, first + i, n0 + row, p.M - first - i, v);
    }
}

// Codes and scales of this CTA's tokens for the k of its stages, written where TMA would
// have put them: rows of 128 bytes with the 128-byte swizzle, scale tiles; as many
// stages at once as the ring holds.
template <typename T, int FMT, int NT>
__device__ __forceinline__ void quantize_stages(const Params &p, Shared<FMT, NT> &sh, int k0, int stages, int warp,
                                                int lane, volatile int *abort, unsigned long long limit) {
    constexpr int STAGES = Config<FMT, NT>::STAGES, WORDS = 8 * sizeof(T), NB = 32 / fp4::Format<FMT>::BLOCK;
    const int zero = fp4::wait_prior_grid_zero();
    const float g = FMT == W4_FMT_NVFP4 ? fp4::load_scalar(p.gx + zero) : 1.0f;
    const T *x = reinterpret_cast<const T *>(p.x) + zero;
    for (int b0 = 0; b0 < stages; b0 += STAGES) {
        const int batch = min(STAGES, stages - b0), units = batch * p.M * 8;
        if (b0 > 0) {
            for (int s = 0; s < batch; s++) pipe_wait(&sh.empty[s], ((b0 / STAGES) - 1) & 1, abort, limit);
            if (__any_sync(0xFFFFFFFFu, *abort != 0)) break;
        }
        for (int i0 = (warp - kEpiWarp0) * 32; i0 < units; i0 += kQuantWarps * 32) {
            // (a division by M here costs 0.1 to 0.3 us of a call)
            const int i = i0 + lane, u = lane & 7, j = i >> 3;
            const int s = p.M == 1 ? j : (int)__umulhi((uint32_t)j, p.inv_m), row = j - s * p.M;
            const int k = (k0 + b0 + s) * BK + u * 32;
            uint32_t w[WORDS], c[4];
            if (i < units && k < p.K) {
                const uint32_t *src = reinterpret_cast<const uint32_t *>(x + (long long)row * p.ldx + k);
#pragma unroll
                for (int j = 0; j < WORDS; j += 4) fp4::load_words<4>(src + j, w + j);
            } else {
#pragma unroll
                for (int j = 0; j < WORDS; j++) w[j] = 0u;
            }
            bool bad;
            const uint32_t word = fp4::quantize32<T, FMT>(w, g, p.ceil_rule, c, bad);
            if (i >= units) continue;
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};"
                         ::"r"(smem_addr(sh.b[s]) + (uint32_t)(row * 128 + ((u ^ (row & 7)) * 16))),
                         "r"(c[0]), "r"(c[1]), "r"(c[2]), "r"(c[3]) : "memory");
            if (u * NB % 4 == 0)
                asm volatile("st.shared.b32 [%0], %1;"
                             ::"r"(smem_addr(sh.sfb[s][u * NB / 4]) + (uint32_t)(row * 16)), "r"(word) : "memory");
            if (bad) fp4::report_nonfinite(p.d_status);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0)
            for (int s = 0; s < batch; s++) mbar_arrive(&sh.full[s]);
    }
    __syncwarp();
}

// T: Quantised (x by TMA) or the type of an x of at most 16 tokens to quantise.
template <int FMT, int NT, typename T>
__global__ void __launch_bounds__(kThreads<T>, 2) gemm_kernel(const __grid_constant__ CUtensorMap wmap,
                                                         const __grid_constant__ CUtensorMap xmap,
                                                         const __grid_constant__ Params p) {
    using S = Shared<FMT, NT>;
    using C = Config<FMT, NT>;
    constexpr int STAGES = C::STAGES;
    extern __shared__ uint8_t smem_raw[];
    S &sh = *reinterpret_cast<S *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int tile = blockIdx.x / p.splits, slice = blockIdx.x % p.splits;
    const int n0 = (tile % p.tiles_n) * BM, m0 = (tile / p.tiles_n) * NT;
    // stages of this slice: the first KT % splits slices take one more
    const int KT = (p.K + BK - 1) / BK;
    const int k0 = slice * (KT / p.splits) + min(slice, KT % p.splits);
    const int k1 = k0 + KT / p.splits + (slice < KT % p.splits ? 1 : 0);
    volatile int *abort = &sh.abort;
    const unsigned long long limit = g_wait_limit_ns;

    if (threadIdx.x == 0) {
        sh.abort = 0;
        for (int i = 0; i < STAGES; i++) {
            mbar_init(&sh.full[i], kFused<T> ? 1 + kQuantWarps : 1);
            mbar_init(&sh.empty[i], 1);
        }
        mbar_init(&sh.acc_full, 1);
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
    // (first half of a cluster barrier: a CTA's shared memory is written by others once
    // it is known to run)
    if (p.splits > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, sh.tmem_base, 0);

    if (warp == 0) {
        // ------------------------------ TMA producer ------------------------------
        // scale tiles that exist in a stage (the last stage of a row may be cut)
        auto tiles = [&](int kt) { return min(C::ST, p.tiles_k - kt * C::ST); };
        auto load_w = [&](int kt, int s) {
            mbar_arrive_expect_tx(&sh.full[s], A_BYTES + (uint32_t)tiles(kt) * SF_TILE +
                                                   (kFused<T> ? 0u : C::B_BYTES + (uint32_t)tiles(kt) * SF_TILE));
            tma_load_2d(sh.a[s], &wmap, kt * (BK / 2), n0, &sh.full[s]);
            bulk_load(sh.sfa[s], p.sfw + ((size_t)(n0 / 128) * p.tiles_k + kt * C::ST) * SF_TILE,
                      (uint32_t)tiles(kt) * SF_TILE, &sh.full[s]);
        };
        auto load_x = [&](int kt, int s) {
            tma_load_2d(sh.b[s], &xmap, kt * (BK / 2), m0, &sh.full[s]);
            bulk_load(sh.sfb[s], p.sfx + ((size_t)(m0 / 128) * p.tiles_k + kt * C::ST) * SF_TILE,
                      (uint32_t)tiles(kt) * SF_TILE, &sh.full[s]);
        };
        const int first = p.early_w ? min(k1 - k0, STAGES) : 0;
        for (int i = 0; i < first; i++)
            if (elect_one()) load_w(k0 + i, i);
        pdl_wait_prior_grid();   // x may be the previous kernel's output
        if (!kFused<T>)
            for (int i = 0; i < first; i++)
                if (elect_one()) load_x(k0 + i, i);
        int it = first;
        for (; it < k1 - k0; it++) {
            const int s = it % STAGES;
            if (it >= STAGES) pipe_wait(&sh.empty[s], ((it / STAGES) - 1) & 1, abort, limit);
            // after an abort nothing more is loaded: the stage may not be free
            if (__any_sync(0xFFFFFFFFu, *abort != 0)) break;
            if (elect_one()) {
                load_w(k0 + it, s);
                if (!kFused<T>) load_x(k0 + it, s);
            }
        }
        // no load may land after the CTA has left (after an abort a stage may lack x that was
        // not quantised: one full wait, and what was issued has landed)
        for (int i = max(0, it - STAGES); i < it; i++)
            if (!mbar_wait_bounded(&sh.full[i % STAGES], (uint32_t)((i / STAGES) & 1))) break;
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------- MMA issuer -------------------------------
        pdl_wait_prior_grid();   // a wait's limit is not to run while the previous kernel does
        const int steps = (p.K + 63) / 64;
        const uint32_t sfa = tmem + C::ACC_COLS, sfb = sfa + 4 * C::ST;
        for (int it = 0; it < k1 - k0; it++) {
            const int s = it % STAGES, kt = k0 + it;
            pipe_wait(&sh.full[s], (it / STAGES) & 1, abort, limit);
            if (__any_sync(0xFFFFFFFFu, *abort != 0)) break;
            tc_fence_after();
            if (elect_one()) {
                const uint32_t a = codes_desc(smem_addr(sh.a[s])), b = codes_desc(smem_addr(sh.b[s]));
                const uint32_t fa = scale_desc(smem_addr(sh.sfa[s])), fb = scale_desc(smem_addr(sh.sfb[s]));
#pragma unroll
                for (int c = 0; c < C::ST; c++) {
                    if (kt * C::ST + c < p.tiles_k) {
                        copy_scales<1>(sfa + 4 * c, fa + c * (SF_TILE / 16));
                        copy_scales<1>(sfb + 4 * c, fb + c * (SF_TILE / 16));
                    }
                }
#pragma unroll
                for (int j = 0; j < BK / 64; j++) {
                    const int c = j / Scales<FMT>::STEPS_PER_TILE;
                    if (kt * (BK / 64) + j < steps)
                        mma_fp4<FMT, 1>(tmem, a + 2 * j, b + 2 * j, idesc<FMT>(BM, NT) | scale_ids<FMT>(j),
                                        sfa + 4 * c, sfb + 4 * c, (it | j) ? 1u : 0u);
                }
                mma_commit(&sh.empty[s]);
                if (it == k1 - k0 - 1) mma_commit(&sh.acc_full);
            }
            __syncwarp();
        }
        // tensor memory is released after the final barrier: every MMA and copy
        // issued must have completed by then (also after an abort)
        if (elect_one()) mma_commit(&sh.mma_done);
        __syncwarp();
        mbar_wait_bounded(&sh.mma_done, 0);
        __syncwarp();
    } else if constexpr (kFused<T>) {
        quantize_stages<T, FMT, NT>(p, sh, k0, k1 - k0, warp, lane, abort, limit);
    }

    // -------------------------------- epilogue --------------------------------
    const int q = warp & 3, row = q * 32 + lane;            // row of w in the tile
    const int own = NT / p.splits;                          // tokens a CTA of the cluster adds up (a power of two)
    if (p.splits > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    const bool epilogue = warp >= kEpiWarp0 && warp < kEpiWarp0 + kEpiWarps;
    if (epilogue) {
        pdl_wait_prior_grid();                              // y and the global scales belong to it until then
        // on expiry (abort) the accumulator is garbage, but the warp stays together
        pipe_wait(&sh.acc_full, 0, abort, limit);
        __syncwarp();
        tc_fence_after();
        const Factor fac(p.gw, p.gx);
        const int n = n0 + row, shift = 31 - __clz(own);
#pragma unroll 1
        for (int c = 0; c < NT / 16 && m0 + c * 16 < p.M; c++) {
            uint32_t r[16];
            W4_FP4_TMEM_LD16(tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(c * 16), r);
            asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
            if (p.splits > 1) {
#pragma unroll
                for (int j = 0; j < 16; j++) {
                    const int m = c * 16 + j, to = m >> shift;   // the CTA that adds token m
                    const uint32_t here = smem_addr(sh.red) + 4u * (uint32_t)((slice * own + m - (to << shift)) * BM + row);
                    uint32_t there;
                    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(here), "r"(to));
                    asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(there), "r"(r[j]) : "memory");
                }
            } else if (n < p.N) {
                float v[16];
#pragma unroll
                for (int j = 0; j < 16; j++) v[j] = __uint_as_float(r[j]);
                apply_factor(fac, v);
                store_column(p, m0 + c * 16, n, p.M - m0 - c * 16, v);
            }
        }
    }
    if (p.splits > 1) {
        // all partial sums are in place; after this no CTA touches another's shared memory
        asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
        if (epilogue && n0 + row < p.N) {
            const Factor fac(p.gw, p.gx);
            const int first = m0 + slice * own;
            if (own >= 8) add_slices<8>(p, fac, sh.red, own, first, n0, row);
            else add_slices<2>(p, fac, sh.red, own, first, n0, row);
        }
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
