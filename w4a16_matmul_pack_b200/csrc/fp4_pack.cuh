// fp4_pack.cuh -- passes over a matrix that quantise it to a 4-bit operand, decode
// one, or lay out its scales (fp4.cuh; sm_100a, CUDA cores).
#pragma once

#include "fp4.cuh"

namespace w4 {

namespace fp4 {

// One lane per 32 values, per_row lanes per row (K / 32 and up to three more, whose
// scales are the padding of the last word).  A lane of eight values (as the norms
// write) would spend as many instructions on its block's scale and its addresses as on
// its values, and the pass was bound by them: 16 per value, 18 us for 2048 x 9728 BF16
// where memory needs 8.
template <typename T, int FMT, bool WIDE>
__global__ void __launch_bounds__(256) quantize_kernel(const T *__restrict__ x, long long ldx, int rows, int per_row,
                                                       const Out o) {
    // in this order: what the next kernel may read early is then complete
    const int zero = wait_prior_grid_zero();
    pdl_allow_dependents();
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x + zero;
    const long long row = i < 0x80000000ll ? (long long)((uint32_t)i / (uint32_t)per_row) : i / per_row;
    const int u = (int)(i - row * per_row);
    const bool active = row < rows && u * 32 < o.K;
    constexpr int WORDS = 8 * sizeof(T), LOAD = WIDE ? 8 : 4;
    uint32_t w[WORDS];
    const float g = FMT == W4_FMT_NVFP4 ? load_scalar(o.global_scale) : 1.0f;
    if (active) {
        const T *p = x + row * ldx + (long long)u * 32;
#pragma unroll
        for (int j = 0; j < WORDS; j += LOAD) load_words<LOAD>(reinterpret_cast<const uint32_t *>(p) + j, w + j);
    } else {
#pragma unroll
        for (int j = 0; j < WORDS; j++) w[j] = 0u;
    }
    constexpr int NB = 32 / Format<FMT>::BLOCK;
    uint32_t c[4];
    bool bad;
    const uint32_t word = quantize32<T, FMT>(w, g, o.ceil_rule, c, bad);
    if (row >= rows) return;
    if (active) store_words<4>(o.codes + row * (o.K / 2) + (long long)u * 16, c);
    if (u * NB % 4 == 0 && u * NB / 4 < o.tiles_k)
        *reinterpret_cast<uint32_t *>(o.scales + scale_word_offset((int)row, u * NB / 4, o.tiles_k)) = word;
    if (bad) report_nonfinite(o.d_status);
}

// E8M0 byte -> binary32 (0xFF: NaN).
__device__ __forceinline__ float e8m0_to_f32(uint32_t b) {
    return __uint_as_float(b == 0u ? 0x00400000u : b == 0xFFu ? 0x7FC00000u : b << 23);
}

// The values codes and scales stand for: e2m1 * s (exact in binary32), times g,
// rounded to T.  One lane per 32 values, as quantize_kernel.
template <typename T, int FMT, bool WIDE>
__global__ void __launch_bounds__(256) dequantize_kernel(const uint8_t *__restrict__ codes,
                                                         const uint8_t *__restrict__ scales,
                                                         const float *__restrict__ gscale, int rows, int K, int tiles_k,
                                                         int per_row, T *__restrict__ out, long long ldo) {
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x + wait_prior_grid_zero();
    const long long row = i < 0x80000000ll ? (long long)((uint32_t)i / (uint32_t)per_row) : i / per_row;
    const int u = (int)(i - row * per_row);
    if (row >= rows || u * 32 >= K) return;
    constexpr int NB = 32 / Format<FMT>::BLOCK, WORDS = 8 * sizeof(T), STORE = WIDE ? 8 : 4;
    uint32_t c[4];
    load_words<4>(codes + row * (K / 2) + (long long)u * 16, c);
    const uint8_t *sp = scales + scale_word_offset((int)row, u * NB / 4, tiles_k) + (u * NB) % 4;
    const float g = FMT == W4_FMT_NVFP4 ? load_scalar(gscale) : 1.0f;
    uint32_t w[WORDS];
#pragma unroll
    for (int e = 0; e < 4; e++) {
        const uint32_t b = sp[e * NB / 4];
        const float s = FMT == W4_FMT_MXFP4 ? e8m0_to_f32(b) : e4m3_to_f32(b);
        uint32_t h[4];
        e2m1x8_to_f16x2(c[e], h);
#pragma unroll
        for (int j = 0; j < 4; j++) {
            float2 f = __fmul2_rn(__half22float2(*reinterpret_cast<const __half2 *>(&h[j])), make_float2(s, s));
            if (FMT == W4_FMT_NVFP4) f = __fmul2_rn(f, make_float2(g, g));
            if constexpr (sizeof(T) == 4) {
                w[8 * e + 2 * j] = __float_as_uint(f.x), w[8 * e + 2 * j + 1] = __float_as_uint(f.y);
            } else if constexpr (kIsHalf<T>) {
                const __half2 r = __float22half2_rn(f);
                w[4 * e + j] = *reinterpret_cast<const uint32_t *>(&r);
            } else {
                const __nv_bfloat162 r = __float22bfloat162_rn(f);
                w[4 * e + j] = *reinterpret_cast<const uint32_t *>(&r);
            }
        }
    }
    uint32_t *p = reinterpret_cast<uint32_t *>(out + row * ldo + (long long)u * 32);
#pragma unroll
    for (int j = 0; j < WORDS; j += STORE) store_words<STORE>(p + j, w + j);
}

// Row-major scales [rows][per_row] -> tiles (zero padding past per_row in the
// last word of a row).
__global__ void __launch_bounds__(256) tile_scales_kernel(const uint8_t *__restrict__ src, int rows, int per_row,
                                                          int tiles_k, uint8_t *__restrict__ dst) {
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x + wait_prior_grid_zero();
    const long long row = i / tiles_k;
    if (row >= rows) return;
    const int word = (int)(i - row * tiles_k);
    const uint8_t *p = src + row * per_row + word * 4;
    uint32_t w = 0;
#pragma unroll
    for (int j = 0; j < 4; j++)
        if (word * 4 + j < per_row) w |= (uint32_t)p[j] << (8 * j);
    *reinterpret_cast<uint32_t *>(dst + scale_word_offset((int)row, word, tiles_k)) = w;
}

}  // namespace fp4

}  // namespace w4
