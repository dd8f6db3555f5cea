// block_norm.cuh -- what stands between two blocks of a decoder, in one pass
// over memory (sm_100a, CUDA cores):
//   b  = y * rsqrt(mean(y^2) + eps) * (w_post + offset)      (or b = y)
//   h' = residual_scale * h + block_scale * act(gate) * b
//   z  = h' * rsqrt(mean(h'^2) + eps) * (w_pre + offset)
// h' is written in the inputs' type, z in that type or as the 4-bit operand of
// the next product (fp4.cuh).
//
// The row stays in registers from the first load to the last store: y, h and the
// gate are read once, h' and z written once, and both statistics are binary32
// sums (fixed order: lanes, warps).  z is formed from h' before h' is rounded to
// its stored type, and quantised before any rounding to 16 bits: the one
// rounding of each output is its own.
//
// One CTA of at most MAXT threads per row, PV units of eight values per thread.
// CTAs walk the rows: the weights (and a gate that serves every row) are loaded
// once per CTA, and the next row's y is on its way while this row is reduced.
#pragma once

#include "fp4.cuh"

namespace w4 {

namespace norm {

enum { GATE_NONE = 0, GATE_SIGMOID = 1, GATE_TANH = 2 };

constexpr int kMaxD = 32768;      // 1024 threads, four units each
constexpr int kMaxM = 1 << 30;    // a row and a grid's stride past the last fit an int

// How a row's values are shared out.
//   VECTOR    thread t, unit p: values 8 (p * threads + t) .. + 7, 16-byte accesses.
//   SCALAR    the same values, one by one (rows that do not start on 16 bytes, 4-bit z).
//   STRIDED   value j of unit p: (8 p + j) * threads + t, one by one and coalesced
//             (widths or strides that are no multiple of 16 bytes).
enum { VECTOR = 0, SCALAR = 1, STRIDED = 2 };

struct Args {
    const void *y, *h, *w_post, *w_pre, *gate;
    void *h_out, *z;
    long long ldy, ldh, ldgate, ldh_out, ldz;
    int M, D, gate_rows, gate_act;
    float inv_D, residual_scale, block_scale, eps, offset;
    fp4::Out q;   // 4-bit z
};

template <int MODE>
__device__ __forceinline__ int index(int p, int j) {
    return MODE == STRIDED ? (8 * p + j) * (int)blockDim.x + (int)threadIdx.x
                           : 8 * (p * (int)blockDim.x + (int)threadIdx.x) + j;
}

// Eight values as they are stored.
template <typename T> struct Raw { uint32_t w[2 * sizeof(T)]; };

template <typename T> __device__ __forceinline__ void unpack(const Raw<T> &r, float2 (&v)[4]);
template <> __device__ __forceinline__ void unpack<__nv_bfloat16>(const Raw<__nv_bfloat16> &r, float2 (&v)[4]) {
#pragma unroll
    for (int j = 0; j < 4; j++) v[j] = make_float2(bf16_lo(r.w[j]), bf16_hi(r.w[j]));
}
template <> __device__ __forceinline__ void unpack<__half>(const Raw<__half> &r, float2 (&v)[4]) {
#pragma unroll
    for (int j = 0; j < 4; j++) v[j] = __half22float2(*reinterpret_cast<const __half2 *>(&r.w[j]));
}
template <> __device__ __forceinline__ void unpack<float>(const Raw<float> &r, float2 (&v)[4]) {
#pragma unroll
    for (int j = 0; j < 4; j++) v[j] = make_float2(__uint_as_float(r.w[2 * j]), __uint_as_float(r.w[2 * j + 1]));
}

template <typename T> __device__ __forceinline__ void pack(const float2 (&v)[4], Raw<T> &r);
template <> __device__ __forceinline__ void pack<__nv_bfloat16>(const float2 (&v)[4], Raw<__nv_bfloat16> &r) {
#pragma unroll
    for (int j = 0; j < 4; j++) {
        const __nv_bfloat162 b = __float22bfloat162_rn(v[j]);
        r.w[j] = *reinterpret_cast<const uint32_t *>(&b);
    }
}
template <> __device__ __forceinline__ void pack<__half>(const float2 (&v)[4], Raw<__half> &r) {
#pragma unroll
    for (int j = 0; j < 4; j++) {
        const __half2 b = __float22half2_rn(v[j]);
        r.w[j] = *reinterpret_cast<const uint32_t *>(&b);
    }
}
template <> __device__ __forceinline__ void pack<float>(const float2 (&v)[4], Raw<float> &r) {
#pragma unroll
    for (int j = 0; j < 4; j++) r.w[2 * j] = __float_as_uint(v[j].x), r.w[2 * j + 1] = __float_as_uint(v[j].y);
}

// A load that the compiler may move past stores: no output overlaps what is still to
// be read (h_out may be h, z may be y, but every value is read before it is written,
// by the same thread).  Zeros where it is not taken.
__device__ __forceinline__ void load_if(bool take, const void *p, uint32_t *w) {
    asm("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
        "@q ld.global.v4.b32 {%0, %1, %2, %3}, [%4];\n\t}"
        : "=&r"(w[0]), "=&r"(w[1]), "=&r"(w[2]), "=&r"(w[3]) : "l"(p), "r"((int)take));
}

// Unit p of a row; values past D are zero.
template <typename T, int MODE>
__device__ __forceinline__ void load_unit(const void *base, long long offset, int p, int D, Raw<T> &r) {
    const T *row = reinterpret_cast<const T *>(base) + offset;
    constexpr int WORDS = 2 * sizeof(T);
    if constexpr (MODE == VECTOR) {
        const int i = index<MODE>(p, 0);
#pragma unroll
        for (int q = 0; q < WORDS; q += 4) load_if(i < D, reinterpret_cast<const uint32_t *>(row + i) + q, r.w + q);
    } else {
#pragma unroll
        for (int j = 0; j < 8; j++) {
            const int i = index<MODE>(p, j);
            if constexpr (sizeof(T) == 4) {
                r.w[j] = i < D ? reinterpret_cast<const uint32_t *>(row)[i] : 0u;
            } else {
                const uint32_t u = i < D ? reinterpret_cast<const uint16_t *>(row)[i] : 0u;
                r.w[j / 2] = j % 2 ? r.w[j / 2] | (u << 16) : u;
            }
        }
    }
}

template <typename T, int MODE>
__device__ __forceinline__ Raw<T> fresh_unit(const void *base, long long offset, int p, int D) {
    Raw<T> r;
    load_unit<T, MODE>(base, offset, p, D, r);
    return r;
}

template <typename T, int MODE>
__device__ __forceinline__ void store_unit(void *base, long long offset, int p, int D, const float2 (&v)[4]) {
    T *row = reinterpret_cast<T *>(base) + offset;
    constexpr int WORDS = 2 * sizeof(T);
    Raw<T> r;
    pack<T>(v, r);
    if constexpr (MODE == VECTOR) {
        const int i = index<MODE>(p, 0);
        if (i < D)
#pragma unroll
            for (int q = 0; q < WORDS / 4; q++)
                reinterpret_cast<uint4 *>(row + i)[q] =
                    make_uint4(r.w[4 * q], r.w[4 * q + 1], r.w[4 * q + 2], r.w[4 * q + 3]);
    } else {
#pragma unroll
        for (int j = 0; j < 8; j++) {
            const int i = index<MODE>(p, j);
            if (i >= D) continue;
            if constexpr (sizeof(T) == 4) reinterpret_cast<uint32_t *>(row)[i] = r.w[j];
            else reinterpret_cast<uint16_t *>(row)[i] = (uint16_t)(r.w[j / 2] >> (16 * (j % 2)));
        }
    }
}

// Sum over the CTA; every thread gets the same value.  part: 32 floats, zero past
// the CTA's warps, free of readers since the last barrier but one.
__device__ __forceinline__ float block_sum(float s, float *part) {
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    if (blockDim.x == 32) return s;
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = s;
    __syncthreads();
    float t = 0.0f;
    for (int w = 0; w < (int)(blockDim.x >> 5); w += 4) {
        const float4 f = *reinterpret_cast<const float4 *>(part + w);
        t += (f.x + f.y) + (f.z + f.w);
    }
    return t;
}

__device__ __forceinline__ float2 both(float a) { return make_float2(a, a); }

// act(gate).
//   sigmoid: 1 / (1 + 2^(-g log2 e)); the argument's rounding costs |g| 2^-24, the
//   exponential and the division 2^-22 each.  Below -87.3 the division gives 0 where
//   sigmoid is less than 2^-126.
//   tanh: from 0.3 on 1 - 2 / (1 + 2^(2 g log2 e)) (what the subtraction loses is at most
//   two bits there); below, its Taylor series to g^9 (the next term is 5e-8 of the sum).
// The library's tanhf inlined for every value of a row is code enough to make the
// kernel wait for instructions.
__device__ __forceinline__ float act_value(float g, int act) {
    if (act == GATE_SIGMOID) return __fdividef(1.0f, 1.0f + exp2f(-1.44269504f * g));
    const float s = g * g, x = fabsf(g);
    const float big = copysignf(1.0f - __fdividef(2.0f, 1.0f + exp2f(2.88539008f * x)), g);
    const float small = fmaf(g * s, fmaf(s, fmaf(s, fmaf(s, 62.0f / 2835.0f, -17.0f / 315.0f), 2.0f / 15.0f),
                                         -1.0f / 3.0f), g);
    return x < 0.3f ? small : big;
}
template <bool ACT>
__device__ __forceinline__ void apply_gate(float2 (&v)[4], const float2 (&g)[4], int act) {
#pragma unroll
    for (int j = 0; j < 4; j++)
        v[j] = __fmul2_rn(v[j], ACT ? make_float2(act_value(g[j].x, act), act_value(g[j].y, act)) : g[j]);
}

// A unit's factors in shared memory: written and read by its own thread alone (no
// barrier), the halves of a unit apart so that a warp's accesses meet no bank twice.
struct Kept {
    float4 *base;
    int units;
    __device__ __forceinline__ void put(int which, int u, const float2 (&v)[4]) const {
        base[(2 * which) * units + u] = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
        base[(2 * which + 1) * units + u] = make_float4(v[2].x, v[2].y, v[3].x, v[3].y);
    }
    __device__ __forceinline__ void multiply(int which, int u, float2 (&v)[4]) const {
        const float4 lo = base[(2 * which) * units + u], hi = base[(2 * which + 1) * units + u];
        v[0] = __fmul2_rn(v[0], make_float2(lo.x, lo.y));
        v[1] = __fmul2_rn(v[1], make_float2(lo.z, lo.w));
        v[2] = __fmul2_rn(v[2], make_float2(hi.x, hi.y));
        v[3] = __fmul2_rn(v[3], make_float2(hi.z, hi.w));
    }
};

template <typename T>
__device__ __forceinline__ void weight_values(const Raw<T> &r, float offset, float2 (&v)[4]) {
    unpack<T>(r, v);
#pragma unroll
    for (int j = 0; j < 4; j++) v[j] = __fadd2_rn(v[j], both(offset));
}

// QFMT 0: z in T; else z in that 4-bit format.  ACT: the gate goes through sigmoid or
// tanh.  KEEP: what every row is multiplied by (the weights, and a gate that serves
// every row) waits in shared memory, ready, and the next row is loaded ahead; without
// it (wide rows, which take the registers for themselves) everything is loaded where it
// is used.
//
// At 21 M values in 26 us (8192 x 2560 BF16 at the copy rate) an SM lane has 45 issue
// slots per value.  So the arithmetic is in pairs (f32x2), a thread takes two units
// where the row has them (the two reductions cost the same per thread), and the weights
// are unpacked once per CTA: in registers they cost either the unpacking for every row
// (one unit per thread: 46 slots, 36.4 us) or the warps that hide the loads.
template <typename T, int PV, int MAXT, int MINB, bool KEEP, int MODE, int QFMT, bool ACT>
__global__ void __launch_bounds__(MAXT, MINB) block_norm_kernel(const __grid_constant__ Args a) {
    __shared__ __align__(16) float part[4][32];
    extern __shared__ float4 kept_units[];
    // in this order: what the next kernel may read early is then complete
    const int zero = fp4::wait_prior_grid_zero();
    pdl_allow_dependents();
    const int D = a.D, t = (int)threadIdx.x, threads = (int)blockDim.x;
    const Kept kept = {kept_units, PV * threads};
    constexpr int KV = KEEP ? PV : 1;
    Raw<T> y[PV], h[KV], g[KV];
    int m = (int)blockIdx.x + zero;
    const bool one_gate = KEEP && a.gate_rows >= a.M;
    const float qg = QFMT == W4_FMT_NVFP4 ? fp4::load_scalar(a.q.global_scale) : 1.0f;
#pragma unroll
    for (int p = 0; p < PV; p++) load_unit<T, MODE>(a.y, m * a.ldy, p, D, y[p]);
    if constexpr (KEEP) {
#pragma unroll
        for (int p = 0; p < PV; p++) {
            if (a.h) load_unit<T, MODE>(a.h, m * a.ldh, p, D, h[p]);
            if (a.gate) load_unit<T, MODE>(a.gate, (m / a.gate_rows) * a.ldgate, p, D, g[p]);
        }
#pragma unroll
        for (int p = 0; p < PV; p++) {
            float2 v[4];
            if (a.w_post) {
                weight_values<T>(fresh_unit<T, MODE>(a.w_post, zero, p, D), a.offset, v);
                kept.put(0, p * threads + t, v);
            }
            if (a.w_pre) {
                weight_values<T>(fresh_unit<T, MODE>(a.w_pre, zero, p, D), a.offset, v);
                kept.put(1, p * threads + t, v);
            }
            if (a.gate && one_gate) {
                float2 one[4] = {both(1.0f), both(1.0f), both(1.0f), both(1.0f)};
                unpack<T>(g[p], v);
                apply_gate<ACT>(one, v, a.gate_act);
                kept.put(2, p * threads + t, one);
            }
        }
    }
    for (int i = t; i < 128; i += threads) part[i >> 5][i & 31] = 0.0f;
    __syncthreads();
    for (int row = 0;; row++) {
        float *sums = part[2 * (row & 1)];
        const int next = m + (int)gridDim.x;
        float2 b[PV][4];
        float2 ss = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int p = 0; p < PV; p++) {
            unpack<T>(y[p], b[p]);
            if (KEEP && next < a.M) load_unit<T, MODE>(a.y, next * a.ldy, p, D, y[p]);
        }
        float scale = a.block_scale;
        if (a.w_post) {
#pragma unroll
            for (int p = 0; p < PV; p++)
#pragma unroll
                for (int j = 0; j < 4; j++) ss = __ffma2_rn(b[p][j], b[p][j], ss);
            scale *= rsqrtf(block_sum(ss.x + ss.y, sums) * a.inv_D + a.eps);
            ss = make_float2(0.0f, 0.0f);
        }
        const float2 scale2 = both(scale), res2 = both(a.residual_scale);
#pragma unroll
        for (int p = 0; p < PV; p++) {
            const int u = p * threads + t;
#pragma unroll
            for (int j = 0; j < 4; j++) b[p][j] = __fmul2_rn(b[p][j], scale2);
            if (a.w_post) {
                if constexpr (KEEP) {
                    kept.multiply(0, u, b[p]);
                } else {
                    float2 v[4];
                    weight_values<T>(fresh_unit<T, MODE>(a.w_post, zero, p, D), a.offset, v);
#pragma unroll
                    for (int j = 0; j < 4; j++) b[p][j] = __fmul2_rn(b[p][j], v[j]);
                }
            }
            if (a.gate) {
                if (one_gate) {
                    kept.multiply(2, u, b[p]);
                } else {
                    float2 v[4];
                    unpack<T>(KEEP ? g[KEEP ? p : 0] : fresh_unit<T, MODE>(a.gate, (m / a.gate_rows) * a.ldgate, p, D),
                              v);
                    if (KEEP && next < a.M)
                        load_unit<T, MODE>(a.gate, (next / a.gate_rows) * a.ldgate, p, D, g[KEEP ? p : 0]);
                    apply_gate<ACT>(b[p], v, a.gate_act);
                }
            }
            if (a.h) {
                float2 v[4];
                unpack<T>(KEEP ? h[KEEP ? p : 0] : fresh_unit<T, MODE>(a.h, m * a.ldh, p, D), v);
                if (KEEP && next < a.M) load_unit<T, MODE>(a.h, next * a.ldh, p, D, h[KEEP ? p : 0]);
#pragma unroll
                for (int j = 0; j < 4; j++) b[p][j] = __ffma2_rn(res2, v[j], b[p][j]);
            }
            // values past D are zero in b and v, so they add nothing
#pragma unroll
            for (int j = 0; j < 4; j++) ss = __ffma2_rn(b[p][j], b[p][j], ss);
            if (a.h_out) store_unit<T, MODE>(a.h_out, m * a.ldh_out, p, D, b[p]);
        }
        const float2 r = both(rsqrtf(block_sum(ss.x + ss.y, sums + 32) * a.inv_D + a.eps));
#pragma unroll
        for (int p = 0; p < PV; p++) {
            const int u = p * threads + t;
#pragma unroll
            for (int j = 0; j < 4; j++) b[p][j] = __fmul2_rn(b[p][j], r);
            if (a.w_pre) {
                if constexpr (KEEP) {
                    kept.multiply(1, u, b[p]);
                } else {
                    float2 v[4];
                    weight_values<T>(fresh_unit<T, MODE>(a.w_pre, zero, p, D), a.offset, v);
#pragma unroll
                    for (int j = 0; j < 4; j++) b[p][j] = __fmul2_rn(b[p][j], v[j]);
                }
            }
            if constexpr (QFMT == 0) {
                store_unit<T, MODE>(a.z, m * a.ldz, p, D, b[p]);
            } else {
                const bool active = u < D / fp4::kUnit;
                const float v[8] = {b[p][0].x, b[p][0].y, b[p][1].x, b[p][1].y,
                                    b[p][2].x, b[p][2].y, b[p][3].x, b[p][3].y};
                // past D: 0 * r may be NaN (r of a row with Inf); the padding stays zero
                fp4::store_unit<QFMT>(a.q, m, u, active, v, active ? fp4::absmax_bits(v) : 0u, qg);
            }
        }
        if (next >= a.M) break;
        m = next;
        if (!KEEP)
#pragma unroll
            for (int p = 0; p < PV; p++) load_unit<T, MODE>(a.y, m * a.ldy, p, D, y[p]);
    }
}

}  // namespace norm

}  // namespace w4
