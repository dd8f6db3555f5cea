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
#pragma once

#include "fp4.cuh"

namespace w4 {

namespace norm {

enum { GATE_NONE = 0, GATE_SIGMOID = 1, GATE_TANH = 2 };

constexpr int kMaxD = 32768;   // 1024 threads, four units each

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
    int D, gate_rows, gate_act;
    float residual_scale, block_scale, eps, offset;
    fp4::Out q;   // 4-bit z
};

template <typename T> __device__ __forceinline__ float to_f32(T v);
template <> __device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <> __device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
template <> __device__ __forceinline__ float to_f32(float v) { return v; }
template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ __nv_bfloat16 from_f32(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half from_f32(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ float from_f32(float v) { return v; }

template <int MODE>
__device__ __forceinline__ int index(int p, int j) {
    return MODE == STRIDED ? (8 * p + j) * (int)blockDim.x + (int)threadIdx.x
                           : 8 * (p * (int)blockDim.x + (int)threadIdx.x) + j;
}

template <typename T, int MODE>
__device__ __forceinline__ void load_unit(const T *row, int p, int D, float (&v)[8]) {
    if constexpr (MODE == VECTOR) {
        const int i = index<MODE>(p, 0);
        uint32_t unused;
        if (i < D) {
            fp4::load8<T>(row + i, v, unused);
        } else {
#pragma unroll
            for (int j = 0; j < 8; j++) v[j] = 0.0f;
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; j++) {
            const int i = index<MODE>(p, j);
            v[j] = i < D ? to_f32<T>(row[i]) : 0.0f;
        }
    }
}

template <typename T, int MODE>
__device__ __forceinline__ void store_row_unit(T *row, int p, int D, const float (&v)[8]) {
    if constexpr (MODE == VECTOR) {
        const int i = index<MODE>(p, 0);
        if (i < D) fp4::store8(row + i, v);
    } else {
#pragma unroll
        for (int j = 0; j < 8; j++) {
            const int i = index<MODE>(p, j);
            if (i < D) row[i] = from_f32<T>(v[j]);
        }
    }
}

// Sum over the CTA; every thread gets the same value.
__device__ __forceinline__ float block_sum(float s, float *part) {
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    const int warps = blockDim.x >> 5;
    if (warps == 1) return s;
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = s;
    __syncthreads();
    float t = 0.0f;
    for (int w = 0; w < warps; w++) t += part[w];
    return t;
}

__device__ __forceinline__ float gate_value(float g, int act) {
    if (act == GATE_SIGMOID) return 1.0f / (1.0f + expf(-g));
    if (act == GATE_TANH) return tanhf(g);
    return g;
}

// QFMT 0: z in T; else z in that 4-bit format.
template <typename T, int PV, int MAXT, int MODE, int QFMT>
__global__ void __launch_bounds__(MAXT) block_norm_kernel(const Args a) {
    __shared__ float part[2][32];
    pdl_allow_dependents();
    const long long m = blockIdx.x;
    const int D = a.D;
    float b[PV][8];
    const T *yr = reinterpret_cast<const T *>(a.y) + m * a.ldy;
    float ss = 0.0f;
#pragma unroll
    for (int p = 0; p < PV; p++) load_unit<T, MODE>(yr, p, D, b[p]);
    float hv[PV][8];
    const T *hr = reinterpret_cast<const T *>(a.h) + m * a.ldh;
    if (a.h) {
#pragma unroll
        for (int p = 0; p < PV; p++) load_unit<T, MODE>(hr, p, D, hv[p]);
    }
    if (a.w_post) {
#pragma unroll
        for (int p = 0; p < PV; p++)
#pragma unroll
            for (int j = 0; j < 8; j++) ss = fmaf(b[p][j], b[p][j], ss);
        const float r = rsqrtf(block_sum(ss, part[0]) / (float)D + a.eps);
#pragma unroll
        for (int p = 0; p < PV; p++) {
            float w[8];
            load_unit<T, MODE>(reinterpret_cast<const T *>(a.w_post), p, D, w);
#pragma unroll
            for (int j = 0; j < 8; j++) b[p][j] = b[p][j] * r * (w[j] + a.offset);
        }
    }
    if (a.gate) {
        const T *gr = reinterpret_cast<const T *>(a.gate) + (m / a.gate_rows) * a.ldgate;
#pragma unroll
        for (int p = 0; p < PV; p++) {
            float g[8];
            load_unit<T, MODE>(gr, p, D, g);
#pragma unroll
            for (int j = 0; j < 8; j++) b[p][j] *= gate_value(g[j], a.gate_act);
        }
    }
    ss = 0.0f;
#pragma unroll
    for (int p = 0; p < PV; p++)
#pragma unroll
        for (int j = 0; j < 8; j++) {
            // values past D are zero in b and hv, so they add nothing
            b[p][j] = a.h ? fmaf(a.residual_scale, hv[p][j], a.block_scale * b[p][j]) : a.block_scale * b[p][j];
            ss = fmaf(b[p][j], b[p][j], ss);
        }
    if (a.h_out) {
        T *ho = reinterpret_cast<T *>(a.h_out) + m * a.ldh_out;
#pragma unroll
        for (int p = 0; p < PV; p++) store_row_unit<T, MODE>(ho, p, D, b[p]);
    }
    const float r = rsqrtf(block_sum(ss, part[1]) / (float)D + a.eps);
    const float g = QFMT == W4_FMT_NVFP4 ? __ldg(a.q.global_scale) : 1.0f;
#pragma unroll
    for (int p = 0; p < PV; p++) {
        float w[8];
        if (a.w_pre) load_unit<T, MODE>(reinterpret_cast<const T *>(a.w_pre), p, D, w);
#pragma unroll
        for (int j = 0; j < 8; j++) b[p][j] = a.w_pre ? b[p][j] * r * (w[j] + a.offset) : b[p][j] * r;
        if constexpr (QFMT == 0) {
            store_row_unit<T, MODE>(reinterpret_cast<T *>(a.z) + m * a.ldz, p, D, b[p]);
        } else {
            const int u = p * (int)blockDim.x + (int)threadIdx.x;
            const bool active = u < D / fp4::kUnit;
            // past D: 0 * r may be NaN (r of a row with Inf); the padding stays zero
            fp4::store_unit<QFMT>(a.q, (int)m, u, active, b[p], active ? fp4::absmax_bits(b[p]) : 0u, g);
        }
    }
}

}  // namespace norm

}  // namespace w4
