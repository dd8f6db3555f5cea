// fp4_mma.cuh -- what the two W4A4 product kernels share: formats, shared-memory
// and instruction descriptors, tcgen05 PTX, the epilogue's factor and stores.
#pragma once

#include "fp4.cuh"

namespace w4 {

namespace fgemm {

constexpr int BM = 128;                 // rows of A per CTA (tensor-memory lanes)
constexpr int BK = 256;                 // k per stage: one 128-byte swizzle row of codes
constexpr uint32_t A_BYTES = BM * (BK / 2);
constexpr uint32_t SF_TILE = 512;       // bytes of a scale tile

enum { OUT_BF16 = W4_TYPE_BF16, OUT_F16 = W4_TYPE_F16, OUT_F32 = W4_TYPE_F32 };

template <int FMT> struct Scales;
// TILES scale tiles along K per stage; STEPS_PER_TILE MMA steps (64 k) share one
template <> struct Scales<W4_FMT_MXFP4> { static constexpr int TILES = 2, STEPS_PER_TILE = 2; };
template <> struct Scales<W4_FMT_NVFP4> { static constexpr int TILES = 4, STEPS_PER_TILE = 1; };

constexpr uint32_t pow2_at_least(uint32_t v) {
    uint32_t p = 32;
    while (p < v) p *= 2;
    return p;
}

// Instruction descriptor: A and B E2M1 (bits 7-9, 10-11), N >> 3 at bit 17, scale
// type at bit 23 (1: E8M0, 0: E4M3), M >> 7 at bit 27, both K-major.  The scale
// ids (bits 4-5 of B, 29-30 of A) select the bytes of a scale word.
template <int FMT>
constexpr uint32_t idesc(int m, int n) {
    return (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | ((FMT == W4_FMT_MXFP4 ? 1u : 0u) << 23) |
           ((uint32_t)(m >> 7) << 27);
}
// The ids of MMA step j within its scale tile (MXFP4: two scales per step).
template <int FMT>
constexpr uint32_t scale_ids(int j) {
    return Scales<FMT>::STEPS_PER_TILE == 2 ? ((uint32_t)(j & 1) * 2u) * ((1u << 4) | (1u << 29)) : 0u;
}

// Shared-memory descriptors as two words.  The high words are constants: version 1
// (bit 46), the stride of 8-row groups, and the swizzle.
constexpr uint32_t kCodesDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);   // 128-byte rows, SWIZZLE_128B
constexpr uint32_t kScaleDescHi = (128u >> 4) | (1u << 14);                 // 16-byte rows, no swizzle

// The low word of the descriptor of a stage of codes / a scale tile at shared-memory
// address `saddr`; 64 k further on is + 2, one scale tile further on + SF_TILE / 16.
__device__ __forceinline__ uint32_t codes_desc(uint32_t saddr) { return ((saddr & 0x3FFFFu) >> 4) | (1u << 16); }
__device__ __forceinline__ uint32_t scale_desc(uint32_t saddr) { return ((saddr & 0x3FFFFu) >> 4) | (8u << 16); }

// One lane of a converged warp, the same one every time.  The loops around the
// tcgen05 and TMA instructions are run by the whole warp and only the instructions
// by this lane: then their operands are computed once per warp.  In code that one
// lane alone reaches, issuing them took longer than executing them (twelve scale
// copies and four 256 x 256 x 64 MMAs: 827 cycles, this way 513).
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
    return p != 0;
}

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// A scale tile from shared memory to four columns, the same for each quarter of the lanes.
template <int GROUP>
__device__ __forceinline__ void copy_scales(uint32_t tmem, uint32_t desc) {
    if constexpr (GROUP == 1)
        asm volatile("{\n\t.reg .b64 d;\n\tmov.b64 d, {%1, %2};\n\t"
                     "tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], d;\n\t}" ::"r"(tmem), "r"(desc), "n"(kScaleDescHi)
                     : "memory");
    else
        asm volatile("{\n\t.reg .b64 d;\n\tmov.b64 d, {%1, %2};\n\t"
                     "tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], d;\n\t}" ::"r"(tmem), "r"(desc), "n"(kScaleDescHi)
                     : "memory");
}

#define W4_FP4_MMA(group, kind)                                                                              \
    asm volatile(                                                                                            \
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tmov.b64 a, {%1, %7};\n\tmov.b64 b, {%2, %7};\n\t"            \
        "setp.ne.b32 p, %6, 0;\n\t"                                                                          \
        "tcgen05.mma.cta_group::" group "." kind " [%0], a, b, %3, [%4], [%5], p;\n\t}"                      \
        ::"r"(d), "r"(a), "r"(b), "r"(id), "r"(sfa), "r"(sfb), "r"(accumulate), "n"(kCodesDescHi) : "memory")

// D += A * B over 64 k; a, b: codes_desc words; sfa, sfb: scale columns.
template <int FMT, int GROUP>
__device__ __forceinline__ void mma_fp4(uint32_t d, uint32_t a, uint32_t b, uint32_t id, uint32_t sfa, uint32_t sfb,
                                        uint32_t accumulate) {
    if constexpr (FMT == W4_FMT_MXFP4 && GROUP == 1) W4_FP4_MMA("1", "kind::mxf4.block_scale.scale_vec::2X");
    if constexpr (FMT == W4_FMT_MXFP4 && GROUP == 2) W4_FP4_MMA("2", "kind::mxf4.block_scale.scale_vec::2X");
    if constexpr (FMT == W4_FMT_NVFP4 && GROUP == 1) W4_FP4_MMA("1", "kind::mxf4nvf4.block_scale.scale_vec::4X");
    if constexpr (FMT == W4_FMT_NVFP4 && GROUP == 2) W4_FP4_MMA("2", "kind::mxf4nvf4.block_scale.scale_vec::4X");
}
#undef W4_FP4_MMA

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

// mbar_wait (common.cuh) without a clock read on the way: reading the limit and the
// global timer takes longer than the waits of a running pipeline.  A wait that has
// to suspend tries kFastTries times (about 0.1 ms) before it goes by the clock; a
// limit below one suspension expires it at once, as there.
constexpr int kFastTries = 1024;
__device__ __forceinline__ bool pipe_wait(uint64_t *bar, uint32_t parity, volatile int *abort,
                                          unsigned long long limit) {
    if (mbar_test_wait(bar, parity)) return true;
    if (limit >= kSuspendNs) {
        for (int i = 0; i < kFastTries; i++) {
            if (mbar_try_wait(bar, parity)) return true;
            if (*abort) return false;
        }
    }
    return mbar_wait(bar, parity, abort);
}

// As long as a bounded wait (2 s): what is in flight when it begins has landed.
__device__ __forceinline__ void settle() {
    const unsigned long long t0 = global_ns();
    for (int i = 0; i < (1 << 26) && global_ns() - t0 < kWaitLimitNs; i++) __nanosleep(1000);
}

// gx * gw: one binary32 factor when it is a normal number or zero, else applied
// in binary64 per value (the factor may leave binary32's range when the result
// does not).
struct Factor {
    float f;
    double d;
    bool wide;
    __device__ __forceinline__ Factor(const float *ga, const float *gb) {
        d = (ga ? (double)fp4::load_scalar(ga) : 1.0) * (gb ? (double)fp4::load_scalar(gb) : 1.0);
        f = (float)d;
        const double m = fabs(d);
        wide = !(d == 0.0 || (m >= 0x1p-126 && m < 0x1p128));
    }
};

// 32 consecutive columns of this warp's 32 lanes.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
          "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]),
          "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]),
          "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(taddr));
}

// 64 columns of this warp's 32 lanes (one row of the output each, or one column of
// it transposed), times the factor.
__device__ __forceinline__ void tmem_ld64(uint32_t taddr, float (&v)[64]) {
    uint32_t a[32], b[32];
    tmem_ld32(taddr, a);
    tmem_ld32(taddr + 32, b);
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 32; i++) v[i] = __uint_as_float(a[i]), v[32 + i] = __uint_as_float(b[i]);
}

template <int n>
__device__ __forceinline__ void apply_factor(const Factor &f, float (&v)[n]) {
    if (f.wide) {
#pragma unroll
        for (int i = 0; i < n; i++) v[i] = (float)((double)v[i] * f.d);
    } else {
#pragma unroll
        for (int i = 0; i < n; i++) v[i] *= f.f;
    }
}

// Two values as 16-bit words of `type` (OUT_BF16 or OUT_F16).
__device__ __forceinline__ uint32_t pack16(float a, float b, int type) {
    if (type == OUT_BF16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// Where an epilogue writes y [rows][cols].
struct Output {
    void *y;
    long long ldy;
    int rows, cols, type;
};

constexpr uint32_t OUT_BYTES = 32 * 128;   // staging of one epilogue warp: 32 rows x 128 bytes

// `rows` rows of `width` (64 or 32) values of T from a staging buffer to y, whose rows start
// on any value.  Whole 16-byte pieces of y where a row has them, eight lanes a row; the up
// to 16 bytes before the first and after the last piece one value a lane.  `cols` < width:
// value by value.  (Value by value throughout, 2048 x 2560 x 9727 BF16 took 82 us; 9728
// takes 22.8 in MXFP4.)
template <typename T>
__device__ __forceinline__ void store_unaligned(const uint8_t *buf, T *dst, long long ldy, int rows, int cols) {
    constexpr int width = 128 / (int)sizeof(T), per = 16 / (int)sizeof(T);
    const int lane = threadIdx.x & 31, k = lane & 7;
    auto value = [&](int r, int c) {
        const int byte = c * (int)sizeof(T);
        return *reinterpret_cast<const T *>(buf + r * 128 + (((byte >> 4) ^ (r & 7)) * 16) + (byte & 15));
    };
    if (cols < width) {
        for (int r = 0; r < rows; r++)
            for (int c = lane; c < cols; c += 32) dst[(size_t)r * ldy + c] = value(r, c);
        return;
    }
#pragma unroll 2
    for (int r0 = 0; r0 < rows; r0 += 4) {
        const int r = r0 + (lane >> 3);
        if (r >= rows) continue;
        T *row = dst + (size_t)r * ldy;
        const int past = (int)((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));   // values since a piece began
        if (past == 0 || k > 0) {
            const int c = k * per - past;
            union { T v[per]; uint4 u; } q;
#pragma unroll
            for (int i = 0; i < per; i++) q.v[i] = value(r, c + i);
            *reinterpret_cast<uint4 *>(row + c) = q.u;
        }
        if (past && k < per) {   // tail: the last `past` values; head: the first per - past
            const int c = k < past ? width - past + k : k - past;
            row[c] = value(r, c);
        }
    }
}

// 32 rows x 64 columns of y at (row0, col0) from the lanes of a warp (lane = row).
// A lane's values are consecutive in a row of y, and the rows of a warp far apart:
// written straight from registers every store touches 32 rows (3.4 us for a 128 x 256
// tile); so the rows are gathered in shared memory (128 bytes each, 128-byte
// swizzle, no bank conflicts) and leave as one TMA box (TMA: y's rows start and end on
// 16 bytes, the unit boxes are clipped in) or in pieces.
template <bool TMA>
__device__ __forceinline__ void store_rows(const Output &o, const CUtensorMap *map, uint8_t *buf, int row0, int col0,
                                           const float (&v)[64]) {
    const int lane = threadIdx.x & 31;
    const bool f32 = o.type == OUT_F32;
    const uint32_t row = smem_addr(buf) + (uint32_t)lane * 128;
#pragma unroll
    for (int half = 0; half < 2; half++) {
        if (half == 1 && !f32) break;
        const int col = col0 + half * 32;
        if (row0 >= o.rows || col >= o.cols) break;
        // the previous box has been read
        if (TMA && elect_one()) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 8; j++) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; i++)
                w[i] = f32 ? __float_as_uint(v[half * 32 + 4 * j + i])
                           : pack16(v[8 * j + 2 * i], v[8 * j + 2 * i + 1], o.type);
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};"
                         ::"r"(row + (uint32_t)((j ^ (lane & 7)) * 16)), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                         : "memory");
        }
        if constexpr (TMA) {
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (elect_one())
                asm volatile(
                    "cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];\n\t"
                    "cp.async.bulk.commit_group;"
                    ::"l"(reinterpret_cast<uint64_t>(map)), "r"(col), "r"(row0), "r"(smem_addr(buf)) : "memory");
        } else {
            __syncwarp();
            const int rows = min(32, o.rows - row0), cols = o.cols - col;
            const size_t at = (size_t)row0 * o.ldy + col;
            if (f32) store_unaligned(buf, reinterpret_cast<uint32_t *>(o.y) + at, o.ldy, rows, cols);
            else store_unaligned(buf, reinterpret_cast<uint16_t *>(o.y) + at, o.ldy, rows, cols);
        }
    }
}

// Before the warp's staging buffer goes out of use: its boxes have been read.
__device__ __forceinline__ void store_rows_done() {
    if (elect_one()) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
    __syncwarp();
}

}  // namespace fgemm

}  // namespace w4
