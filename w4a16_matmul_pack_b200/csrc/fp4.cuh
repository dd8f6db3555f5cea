// fp4.cuh -- block-scaled 4-bit operands of the W4A4 product: formats, scale
// layout, and the encoder of one block (sm_100a, CUDA cores).
//
// MXFP4: E2M1 codes, one power of two (E8M0) per 32 values along K,
//   e = floor(log2 amax) - 2 (OCP Microscaling Formats 1.0, section 6.3), or with
//   W4_MX_SCALE_CEIL the smallest e with amax <= 6 * 2^e; x * 2^-e is exact, so
//   each code is rounded once.
// NVFP4 ("EdgeRock-4B-NVFP4" card, intro): E2M1 codes, one E4M3 scale per 16
//   values, one given binary32 global scale g: s = E4M3(amax / 6 / g),
//   code = E2M1(x * RN(1 / (s * g))).  One reciprocal per block instead of the
//   weight packer's division per value: the encoder is a pass over memory, and
//   sixteen divisions cost more than its loads.
//
// Scales are kept as the tensor cores read them (w4_fp4 in include/w4a16.h):
// tiles of 128 rows x 4 scales, 512 bytes, row r at byte (r % 32) * 16 +
// (r / 32) * 4.  A tile is one bulk copy to shared memory and one tcgen05.cp to
// tensor memory; from row-major scales the product would have to move every
// 4-byte word by itself.
#pragma once

#include "common.cuh"

namespace w4 {

namespace fp4 {

// Waits for the previous kernel on the stream and returns 0, which every address read
// after it is to contain: loads marked read-only, and assembly that is not volatile,
// may otherwise be moved up past the wait.
__device__ __forceinline__ int wait_prior_grid_zero() {
    int zero;
    pdl_wait_prior_grid();
    asm volatile("mov.b32 %0, 0;" : "=r"(zero) :: "memory");
    return zero;
}

// One float, read where the program says.
__device__ __forceinline__ float load_scalar(const float *p) {
    float v;
    asm volatile("ld.global.f32 %0, [%1];" : "=f"(v) : "l"(p) : "memory");
    return v;
}

constexpr int kUnit = 8;   // values of a lane of the norms: 16 bytes of a 16-bit type, 4 bytes of codes

template <typename T> constexpr bool kIsHalf = false;
template <> constexpr bool kIsHalf<__half> = true;

template <int FMT> struct Format;
// BLOCK values per scale; a scale word (4 scales) covers WORD_UNITS lanes
template <> struct Format<W4_FMT_MXFP4> { static constexpr int BLOCK = 32, WORD_UNITS = 16; };
template <> struct Format<W4_FMT_NVFP4> { static constexpr int BLOCK = 16, WORD_UNITS = 8; };

// Scale tiles along K.
__host__ __device__ inline int scale_tiles_k(int fmt, int K) {
    return fmt == W4_FMT_MXFP4 ? (K + 127) / 128 : (K + 63) / 64;
}

// Byte offset of the 4-scale word `word` (along K) of row `row`.
__device__ __forceinline__ size_t scale_word_offset(int row, int word, int tiles_k) {
    return ((size_t)(row >> 7) * tiles_k + word) * 512 + (size_t)((row & 31) * 16 + ((row >> 5) & 3) * 4);
}

// Largest magnitude of eight values as bits: unsigned order is the order of
// magnitudes, with Inf and NaN above every finite value.
__device__ __forceinline__ uint32_t absmax_bits(const float (&v)[8]) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; j++) m = max(m, __float_as_uint(v[j]) & 0x7FFFFFFFu);
    return m;
}

// Where a quantiser writes.
struct Out {
    uint8_t *codes;
    uint8_t *scales;
    const float *global_scale;   // NVFP4
    int *d_status;
    int K, tiles_k, ceil_rule;
};

// Eight values times f as E2M1 codes, nearest even, saturating (value 2j in the
// low nibble of byte j).  The conversion keeps the sign of values that round to
// zero; NaN does not come here.
__device__ __forceinline__ uint32_t pack_e2m1x8(const float (&v)[8], float f) {
    float2 q[4];
#pragma unroll
    for (int j = 0; j < 4; j++) q[j] = __fmul2_rn(make_float2(v[2 * j], v[2 * j + 1]), make_float2(f, f));
    uint32_t c;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(c)
        : "f"(q[0].x), "f"(q[0].y), "f"(q[1].x), "f"(q[1].y), "f"(q[2].x), "f"(q[2].y), "f"(q[3].x), "f"(q[3].y));
    return c;
}

// The scale of a block whose largest magnitude has the bits `amax`: its byte, and the
// factor its values are multiplied by before they are rounded to codes.  A block that
// holds Inf or NaN gets the scale type's NaN, so that every value it stands for, and
// every product with it, is NaN; its codes are zero.
template <int FMT>
__device__ __forceinline__ uint32_t block_scale(uint32_t amax, float g, bool ceil_rule, float &f) {
    uint32_t byte;
    if constexpr (FMT == W4_FMT_MXFP4) {
        // the bias of binary32 and of E8M0 is the same: 2^(e - 2) is byte e - 2
        const int up = (ceil_rule && (amax & 0x7FFFFFu) > 0x400000u) ? 1 : 0;
        byte = (uint32_t)max((int)(amax >> 23) - 2 + up, 0);
        f = __uint_as_float((254u - byte) << 23);
        if (amax >= 0x7F800000u) byte = 0xFFu, f = 0.0f;
    } else {
        const float t = __fdiv_rn(__fdiv_rn(__uint_as_float(amax), 6.0f), g);
        byte = g > 0.0f ? f32_to_e4m3(t) : (g != g ? 0x7Fu : 0u);
        f = __frcp_rn(__fmul_rn(e4m3_to_f32(byte), g));
        // s * g == 0, or too small for a binary32 reciprocal: a block of zeros
        if (!(fabsf(f) <= 3.4028234e38f) && byte != 0x7Fu) byte = 0u, f = 0.0f;
        if (amax >= 0x7F800000u || byte == 0x7Fu) byte = 0x7Fu, f = 0.0f;
    }
    return byte;
}

__device__ __forceinline__ void report_nonfinite(int *d_status) {
    record_error(W4_ERR_NONFINITE);
    if (d_status) *d_status = W4_ERR_NONFINITE;
}

// Unit `u` (values 8u .. 8u+7) of row `row`, one lane each, the lanes of a warp
// holding consecutive units from a multiple of 32: block maxima by shuffles, the
// codes as one 4-byte store per lane, four scales as one 4-byte store by the
// first lane of their lanes.  Lanes past the row's end pass active = false,
// amax = 0 (their scales are the zero padding of the last word) and take part.
template <int FMT>
__device__ __forceinline__ void store_unit(const Out &o, int row, int u, bool active, const float (&v)[8],
                                           uint32_t amax, float g) {
    const int lane = threadIdx.x & 31;
    constexpr int BU = Format<FMT>::BLOCK / kUnit;   // lanes of a block
    amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
    if (BU == 4) amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
    float f;
    const uint32_t byte = block_scale<FMT>(amax, g, o.ceil_rule, f);
    uint32_t word = byte << (8 * ((lane / BU) & 3));
    word |= __shfl_xor_sync(0xFFFFFFFFu, word, BU);
    word |= __shfl_xor_sync(0xFFFFFFFFu, word, 2 * BU);
    if (!active) return;
    const bool bad = amax >= 0x7F800000u;
    const uint32_t c = bad ? 0u : pack_e2m1x8(v, f);
    *reinterpret_cast<uint32_t *>(o.codes + (size_t)row * (o.K / 2) + (size_t)u * 4) = c;
    constexpr int WU = Format<FMT>::WORD_UNITS;
    if (u % WU == 0) *reinterpret_cast<uint32_t *>(o.scales + scale_word_offset(row, u / WU, o.tiles_k)) = word;
    if (bad) report_nonfinite(o.d_status);
}

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

// 32 values of a row (in the words w; zeros past the row's end) as codes, and the
// 4-scale word they belong to, complete in every lane of its lanes: four lanes with
// consecutive 32 values for MXFP4, two for NVFP4, from a multiple of that many.
template <typename T, int FMT>
__device__ __forceinline__ uint32_t quantize32(const uint32_t *w, float g, bool ceil_rule, uint32_t (&c)[4], bool &bad) {
    constexpr int WORDS = 8 * sizeof(T), NB = 32 / Format<FMT>::BLOCK, BW = WORDS / NB;   // blocks, words of a block
    const int lane = threadIdx.x & 31;
    uint32_t word = 0;
    bad = false;
#pragma unroll
    for (int b = 0; b < NB; b++) {
        const uint32_t amax = absmax_words<T>(w + b * BW, BW);
        float f;
        word |= block_scale<FMT>(amax, g, ceil_rule, f) << (8 * ((NB * lane + b) & 3));
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
    return word;
}

}  // namespace fp4

}  // namespace w4
