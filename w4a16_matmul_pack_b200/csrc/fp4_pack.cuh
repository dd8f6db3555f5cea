// fp4_pack.cuh -- passes over a matrix that quantise it to a 4-bit operand, decode
// one, or lay out its scales (fp4.cuh; sm_100a, CUDA cores).
#pragma once

#include "fp4.cuh"

namespace w4 {

namespace fp4 {

// 32 or 16 consecutive bytes.
template <int WORDS>
__device__ __forceinline__ void load_words(const void *p, uint32_t *w) {
    if constexpr (WORDS == 8)
        asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                     : "l"(p));
    else
        asm volatile("ld.global.nc.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "l"(p));
}
template <int WORDS>
__device__ __forceinline__ void store_words(void *p, const uint32_t *w) {
    if constexpr (WORDS == 8)
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                     ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
    else
        asm volatile("st.global.v4.b32 [%0], {%1, %2, %3, %4};"
                     ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]) : "memory");
}

// Largest magnitude of n words of T, as binary32 bits.
template <typename T>
__device__ __forceinline__ uint32_t absmax_words(const uint32_t *w, int n) {
    uint32_t m = 0;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < n; i++) m = max(m, w[i] & 0x7FFFFFFFu);
        return m;
    } else {
#pragma unroll
        for (int i = 0; i < n; i++) m = __vmaxu2(m, w[i] & 0x7FFF7FFFu);
        m = max(m & 0xFFFFu, m >> 16);
        if constexpr (sizeof(T) == 2 && !kIsHalf<T>)
            return m << 16;
        else
            return __float_as_uint(__half2float(__ushort_as_half((unsigned short)m))) & 0x7FFFFFFFu;
    }
}

// Eight values from the words at w.
template <typename T>
__device__ __forceinline__ void values8(const uint32_t *w, float (&v)[8]) {
#pragma unroll
    for (int j = 0; j < 8; j++) {
        if constexpr (sizeof(T) == 4) v[j] = __uint_as_float(w[j]);
        else if constexpr (!kIsHalf<T>) v[j] = j % 2 ? bf16_hi(w[j / 2]) : bf16_lo(w[j / 2]);
        else {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[j / 2]));
            v[j] = j % 2 ? f.y : f.x;
        }
    }
}

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
    constexpr int NB = 32 / Format<FMT>::BLOCK, BW = WORDS / NB;   // blocks of the lane, words of a block
    const int lane = threadIdx.x & 31;
    uint32_t word = 0, c[4];
    bool bad = false;
#pragma unroll
    for (int b = 0; b < NB; b++) {
        const uint32_t amax = absmax_words<T>(w + b * BW, BW);
        float f;
        word |= block_scale<FMT>(amax, g, o.ceil_rule, f) << (8 * ((NB * lane + b) & 3));
        bad = bad || amax >= 0x7F800000u;
#pragma unroll
        for (int e = 0; e < 4 / NB; e++) {
            float v[8];
            values8<T>(w + b * BW + e * (WORDS / 4), v);
            c[b * (4 / NB) + e] = amax >= 0x7F800000u ? 0u : pack_e2m1x8(v, f);
        }
    }
    word |= __shfl_xor_sync(0xFFFFFFFFu, word, 1);
    if (NB == 1) word |= __shfl_xor_sync(0xFFFFFFFFu, word, 2);
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
