// fp4.cuh -- block-scaled 4-bit operands of the W4A4 product (sm_100a, CUDA
// cores): quantise, decode, lay out scales.
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

constexpr int kUnit = 8;   // values of one lane: 16 bytes of a 16-bit type, 4 bytes of codes

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

// Eight consecutive values (16-byte aligned) as binary32, and the bits of their
// largest magnitude: unsigned order is the order of magnitudes, with Inf and NaN
// above every finite value.
template <typename T>
__device__ __forceinline__ void load8(const T *p, float (&v)[8], uint32_t &amax);

template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16 *p, float (&v)[8], uint32_t &amax) {
    const uint4 r = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 4; j++) {
        v[2 * j] = bf16_lo(w[j]);
        v[2 * j + 1] = bf16_hi(w[j]);
        m = __vmaxu2(m, w[j] & 0x7FFF7FFFu);
    }
    amax = max(m & 0xFFFFu, m >> 16) << 16;
}

template <>
__device__ __forceinline__ void load8<__half>(const __half *p, float (&v)[8], uint32_t &amax) {
    const uint4 r = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 4; j++) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[j]));
        v[2 * j] = f.x;
        v[2 * j + 1] = f.y;
        m = __vmaxu2(m, w[j] & 0x7FFF7FFFu);
    }
    amax = __float_as_uint(__half2float(__ushort_as_half((unsigned short)max(m & 0xFFFFu, m >> 16)))) & 0x7FFFFFFFu;
}

__device__ __forceinline__ uint32_t absmax_bits(const float (&v)[8]) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; j++) m = max(m, __float_as_uint(v[j]) & 0x7FFFFFFFu);
    return m;
}

template <>
__device__ __forceinline__ void load8<float>(const float *p, float (&v)[8], uint32_t &amax) {
    const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    amax = absmax_bits(v);
}

// Where a quantiser writes.
struct Out {
    uint8_t *codes;
    uint8_t *scales;
    const float *global_scale;   // NVFP4
    int *d_status;
    int K, tiles_k, ceil_rule;
};

__device__ __forceinline__ uint32_t pack_e2m1x8(const float (&v)[8], float f) {
    uint32_t c = 0;
#pragma unroll
    for (int j = 0; j < 4; j++) c |= f32x2_to_e2m1x2(v[2 * j] * f, v[2 * j + 1] * f) << (8 * j);
    return c;
}

// Unit `u` (values 8u .. 8u+7) of row `row`, one lane each, the lanes of a warp
// holding consecutive units from a multiple of 32: block maxima by shuffles, the
// codes as one 4-byte store per lane, four scales as one 4-byte store by the
// first lane of their lanes.  Lanes past the row's end pass active = false,
// amax = 0 (their scales are the zero padding of the last word) and take part.
// A block that holds Inf or NaN gets the scale type's NaN, so that every value
// it stands for, and every product with it, is NaN.
template <int FMT>
__device__ __forceinline__ void store_unit(const Out &o, int row, int u, bool active, const float (&v)[8],
                                           uint32_t amax, float g) {
    const int lane = threadIdx.x & 31;
    uint32_t byte, word;
    float f;
    bool bad;
    if constexpr (FMT == W4_FMT_MXFP4) {
        amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
        amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
        bad = amax >= 0x7F800000u;
        // the bias of binary32 and of E8M0 is the same: 2^(e - 2) is byte e - 2
        const int up = (o.ceil_rule && (amax & 0x7FFFFFu) > 0x400000u) ? 1 : 0;
        byte = (uint32_t)max((int)(amax >> 23) - 2 + up, 0);
        f = __uint_as_float((254u - byte) << 23);
        if (bad) byte = 0xFFu;
        word = byte << (8 * ((lane >> 2) & 3));
        word |= __shfl_xor_sync(0xFFFFFFFFu, word, 4);
        word |= __shfl_xor_sync(0xFFFFFFFFu, word, 8);
    } else {
        amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
        bad = amax >= 0x7F800000u;
        const float t = __fdiv_rn(__fdiv_rn(__uint_as_float(amax), 6.0f), g);
        byte = g > 0.0f ? f32_to_e4m3(t) : (g != g ? 0x7Fu : 0u);
        f = __frcp_rn(__fmul_rn(e4m3_to_f32(byte), g));
        // s * g == 0, or too small for a binary32 reciprocal: a block of zeros
        if (!(f <= 3.4028234e38f) && byte != 0x7Fu) byte = 0u, f = 0.0f;
        if (bad) byte = 0x7Fu;
        word = byte << (8 * ((lane >> 1) & 3));
        word |= __shfl_xor_sync(0xFFFFFFFFu, word, 2);
        word |= __shfl_xor_sync(0xFFFFFFFFu, word, 4);
    }
    if (!active) return;
    const uint32_t c = bad ? 0u : pack_e2m1x8(v, f);
    *reinterpret_cast<uint32_t *>(o.codes + (size_t)row * (o.K / 2) + (size_t)u * 4) = c;
    constexpr int WU = Format<FMT>::WORD_UNITS;
    if (u % WU == 0) *reinterpret_cast<uint32_t *>(o.scales + scale_word_offset(row, u / WU, o.tiles_k)) = word;
    if (bad) {
        record_error(W4_ERR_NONFINITE);
        if (o.d_status) *o.d_status = W4_ERR_NONFINITE;
    }
}

// One warp per 256 values of a row.  Bound by memory: the values read once,
// codes and scales written once.
template <typename T, int FMT>
__global__ void __launch_bounds__(256) quantize_kernel(const T *__restrict__ x, long long ldx, int rows, int pieces,
                                                       const Out o) {
    pdl_allow_dependents();
    const long long task = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    const long long row = task / pieces;
    if (row >= rows) return;
    const int u = (int)(task - row * pieces) * 32 + (threadIdx.x & 31);
    const bool active = u < o.K / kUnit;
    float v[8] = {};
    uint32_t amax = 0;
    if (active) load8<T>(x + row * ldx + (long long)u * kUnit, v, amax);
    const float g = FMT == W4_FMT_NVFP4 ? __ldg(o.global_scale) : 1.0f;
    store_unit<FMT>(o, (int)row, u, active, v, amax, g);
}

// E8M0 byte -> binary32 (0xFF: NaN).
__device__ __forceinline__ float e8m0_to_f32(uint32_t b) {
    return __uint_as_float(b == 0u ? 0x00400000u : b == 0xFFu ? 0x7FC00000u : b << 23);
}

__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; j++) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
        w[j] = *reinterpret_cast<const uint32_t *>(&b);
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(__half *p, const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; j++) {
        const __half2 b = __floats2half2_rn(v[2 * j], v[2 * j + 1]);
        w[j] = *reinterpret_cast<const uint32_t *>(&b);
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(float *p, const float (&v)[8]) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

// The values codes and scales stand for: e2m1 * s (exact in binary32), times g,
// rounded to T.
template <typename T, int FMT>
__global__ void __launch_bounds__(256) dequantize_kernel(const uint8_t *__restrict__ codes,
                                                         const uint8_t *__restrict__ scales,
                                                         const float *__restrict__ gscale, int rows, int K, int tiles_k,
                                                         int pieces, T *__restrict__ out, long long ldo) {
    const long long task = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    const long long row = task / pieces;
    if (row >= rows) return;
    const int u = (int)(task - row * pieces) * 32 + (threadIdx.x & 31);
    if (u >= K / kUnit) return;
    const uint32_t c = *reinterpret_cast<const uint32_t *>(codes + row * (K / 2) + (long long)u * 4);
    constexpr int WU = Format<FMT>::WORD_UNITS, BU = Format<FMT>::BLOCK / kUnit;
    const uint32_t b = scales[scale_word_offset((int)row, u / WU, tiles_k) + (u / BU) % 4];
    const float s = FMT == W4_FMT_MXFP4 ? e8m0_to_f32(b) : e4m3_to_f32(b);
    const float g = FMT == W4_FMT_NVFP4 ? __ldg(gscale) : 1.0f;
    uint32_t h[4];
    e2m1x8_to_f16x2(c, h);
    float v[8];
#pragma unroll
    for (int j = 0; j < 4; j++) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h[j]));
        v[2 * j] = f.x * s;
        v[2 * j + 1] = f.y * s;
        if (FMT == W4_FMT_NVFP4) v[2 * j] *= g, v[2 * j + 1] *= g;
    }
    store8(out + row * ldo + (long long)u * kUnit, v);
}

// Row-major scales [rows][per_row] -> tiles (zero padding past per_row in the
// last word of a row).
__global__ void __launch_bounds__(256) tile_scales_kernel(const uint8_t *__restrict__ src, int rows, int per_row,
                                                          int tiles_k, uint8_t *__restrict__ dst) {
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
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
