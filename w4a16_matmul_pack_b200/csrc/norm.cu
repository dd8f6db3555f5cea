// norm.cu -- w4_block_norm (declared in include/w4a16.h): host-side validation, the
// choice of kernel and its launch.
#include <cuda_runtime.h>

#include <algorithm>

#include "block_norm.cuh"
#include "fp4_host.cuh"

using namespace w4;

namespace w4 {

int norm_device_error(int *out, int clear) { return take_device_error(out, clear); }

}  // namespace w4

namespace {

template <typename T, int PV, int MAXT, int MINB, bool KEEP, int QFMT, bool ACT>
w4_status launch_block(const norm::Args &a, int mode, int grid, int threads, cudaStream_t st) {
    constexpr int ODD = QFMT != 0 ? norm::SCALAR : norm::STRIDED;
    return launch_behind(mode == norm::VECTOR
                             ? norm::block_norm_kernel<T, PV, MAXT, MINB, KEEP, norm::VECTOR, QFMT, ACT>
                             : norm::block_norm_kernel<T, PV, MAXT, MINB, KEEP, ODD, QFMT, ACT>,
                         (unsigned)grid, (unsigned)threads, KEEP ? (size_t)threads * PV * 96 : 0, st, a);
}

// Threads per SM that the register use leaves room for (64 registers each); CTAs beyond
// them would only start the loop over the rows late (8192 x 2560: 1536 threads 64 us,
// 1024 threads 55 us on the kernel's first version).
constexpr int kResident = 1024;

template <typename T, int QFMT, bool ACT>
w4_status launch_norm(const norm::Args &a, int mode, cudaStream_t st) {
    const int units = (a.D + fp4::kUnit - 1) / fp4::kUnit;
    int sms = 0;
    if (device_sms(sms) != W4_OK) return W4_ERR_CUDA;
    // a batch with no more rows than SMs has threads to spare for a shorter row (one row
    // of 2560: one unit per thread 2.7 us, two 3.1 us)
    const int pv = units <= 32 || (units <= 512 && a.M <= sms) ? 1 : units <= 1024 ? 2 : 4;
    const int threads = ((units + pv - 1) / pv + 31) / 32 * 32;
    const int grid = std::min(a.M, sms * std::max(1, kResident / threads));
    if (pv == 1) return launch_block<T, 1, 512, sizeof(T) == 2 ? 2 : 1, true, QFMT, ACT>(a, mode, grid, threads, st);
    if (pv == 2) return launch_block<T, 2, 512, sizeof(T) == 2 ? 2 : 1, true, QFMT, ACT>(a, mode, grid, threads, st);
    return launch_block<T, 4, 1024, 1, false, QFMT, ACT>(a, mode, grid, threads, st);
}

template <typename T, int QFMT>
w4_status launch_norm_act(const norm::Args &a, int mode, cudaStream_t st) {
    return a.gate && a.gate_act != norm::GATE_NONE ? launch_norm<T, QFMT, true>(a, mode, st)
                                                   : launch_norm<T, QFMT, false>(a, mode, st);
}

template <typename T>
w4_status launch_norm_fmt(const norm::Args &a, int mode, int fmt, cudaStream_t st) {
    if (fmt == 0) return launch_norm_act<T, 0>(a, mode, st);
    if (fmt == W4_FMT_MXFP4) return launch_norm_act<T, W4_FMT_MXFP4>(a, mode, st);
    return launch_norm_act<T, W4_FMT_NVFP4>(a, mode, st);
}

}  // namespace

extern "C" w4_status w4_block_norm(const w4_norm *n, void *stream) {
    if (!n || !n->y || n->M < 1 || n->D < 1 || !is_type(n->type) || !(n->eps >= 0.0f)) return W4_ERR_ARG;
    if (n->D > norm::kMaxD || n->M > norm::kMaxM) return W4_ERR_UNSUPPORTED;
    if (n->ldy < n->D || (n->h && n->ldh < n->D) || (n->h_out && n->ldh_out < n->D)) return W4_ERR_ARG;
    if (n->gate && (n->gate_rows < 1 || n->ldgate < n->D)) return W4_ERR_ARG;
    if (n->gate_act < W4_GATE_NONE || n->gate_act > W4_GATE_TANH) return W4_ERR_ARG;
    const int size = type_size(n->type);
    auto on = [&](const void *p, int bytes) { return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(bytes - 1)) == 0; };
    const void *ptrs[] = {n->y, n->h, n->w_post, n->w_pre, n->gate, n->h_out, n->z};
    bool vec = n->D % fp4::kUnit == 0 && rows16(n->ldy, n->type) && (!n->h || rows16(n->ldh, n->type)) &&
               (!n->h_out || rows16(n->ldh_out, n->type)) && (!n->gate || rows16(n->ldgate, n->type));
    for (const void *q : ptrs) {
        if (!on(q, size)) return W4_ERR_ALIGN;
        vec = vec && on(q, 16);
    }
    norm::Args a = {};
    if (n->quant_fmt) {
        const w4_status s = check_quantised(n->M, n->D, n->quant_fmt, n->scale_rule, n->global_scale, n->codes,
                                            n->scales, n->d_status);
        if (s != W4_OK) return s;
        if (n->z) return W4_ERR_ARG;
        a.q = quantised_out(n->D, n->quant_fmt, n->scale_rule, n->global_scale, n->codes, n->scales, n->d_status);
    } else {
        if (!n->z || n->ldz < n->D) return W4_ERR_ARG;
        vec = vec && rows16(n->ldz, n->type);
    }
    a.y = n->y, a.h = n->h, a.w_post = n->w_post, a.w_pre = n->w_pre, a.gate = n->gate;
    a.h_out = n->h_out, a.z = n->z;
    a.ldy = n->ldy, a.ldh = n->ldh, a.ldgate = n->ldgate, a.ldh_out = n->ldh_out, a.ldz = n->ldz;
    a.M = n->M, a.D = n->D, a.gate_rows = n->gate_rows, a.gate_act = n->gate_act;
    a.inv_D = 1.0f / (float)n->D, a.residual_scale = n->residual_scale, a.block_scale = n->block_scale, a.eps = n->eps, a.offset = n->weight_offset;
    cudaStream_t st = as_stream(stream);
    if (n->quant_fmt && clear_status(n->d_status, st) != W4_OK) return W4_ERR_CUDA;
    const int mode = vec ? norm::VECTOR : n->quant_fmt ? norm::SCALAR : norm::STRIDED;
    switch (n->type) {
    case W4_TYPE_BF16: return launch_norm_fmt<__nv_bfloat16>(a, mode, n->quant_fmt, st);
    case W4_TYPE_F16: return launch_norm_fmt<__half>(a, mode, n->quant_fmt, st);
    case W4_TYPE_F32: return launch_norm_fmt<float>(a, mode, n->quant_fmt, st);
    }
    return W4_ERR_ARG;
}
