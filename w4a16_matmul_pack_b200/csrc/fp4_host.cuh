// fp4_host.cuh -- host-side checks that the W4A4 entry points share (fp4.cu, norm.cu).
#pragma once

#include <atomic>

#include "fp4.cuh"

namespace w4 {

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
inline cudaStream_t as_stream(void *s) { return reinterpret_cast<cudaStream_t>(s); }
inline w4_status launch_status() { return cudaGetLastError() == cudaSuccess ? W4_OK : W4_ERR_CUDA; }

inline bool is_fp4(int fmt) { return fmt == W4_FMT_MXFP4 || fmt == W4_FMT_NVFP4; }
inline int type_size(int type) { return type == W4_TYPE_F32 ? 4 : 2; }
inline bool is_type(int type) { return type == W4_TYPE_BF16 || type == W4_TYPE_F16 || type == W4_TYPE_F32; }
// Rows of `ld` values of `type` that all start on 16 bytes.
inline bool rows16(long long ld, int type) { return ld * type_size(type) % 16 == 0; }

constexpr long long kMaxBlocks = 0x7FFFFFFFll;

// Rows and K of an operand: with a tile (256) added they still fit an int.
constexpr int kMaxExtent = 0x7FFFFFFF - 255;
inline bool too_large(int rows, int K) { return rows > kMaxExtent || K > kMaxExtent; }

// SMs of the current device (asked once per device; threads that ask at once read the same).
inline w4_status device_sms(int &sms) {
    constexpr int kMaxDevices = 64;
    static std::atomic<int> known[kMaxDevices];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return W4_ERR_CUDA;
    sms = known[dev].load(std::memory_order_relaxed);
    if (sms) return W4_OK;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return W4_ERR_CUDA;
    known[dev].store(sms, std::memory_order_relaxed);
    return W4_OK;
}

inline w4_status check_operand(const w4_fp4 *a) {
    if (!a || !is_fp4(a->fmt) || a->rows < 1 || a->K < 32 || a->K % 32 || !a->codes || !a->scales) return W4_ERR_ARG;
    if (too_large(a->rows, a->K)) return W4_ERR_UNSUPPORTED;
    if (a->fmt == W4_FMT_NVFP4 && !a->global_scale) return W4_ERR_ARG;
    if (!aligned16(a->codes) || !aligned16(a->scales) || !aligned4(a->global_scale)) return W4_ERR_ALIGN;
    return W4_OK;
}

// A quantiser's output side.
inline w4_status check_quantised(int rows, int K, int fmt, int scale_rule, const float *global_scale, const uint8_t *codes,
                          const uint8_t *scales, const int *d_status) {
    if (!is_fp4(fmt) || rows < 1 || K < 32 || K % 32 || !codes || !scales) return W4_ERR_ARG;
    if (too_large(rows, K)) return W4_ERR_UNSUPPORTED;
    if (scale_rule != W4_MX_SCALE_FLOOR && scale_rule != W4_MX_SCALE_CEIL) return W4_ERR_ARG;
    if (fmt == W4_FMT_NVFP4 && (!global_scale || scale_rule != W4_MX_SCALE_FLOOR)) return W4_ERR_ARG;
    if (!aligned16(codes) || !aligned16(scales) || !aligned4(global_scale) || !aligned4(d_status)) return W4_ERR_ALIGN;
    return W4_OK;
}

inline fp4::Out quantised_out(int K, int fmt, int scale_rule, const float *global_scale, uint8_t *codes, uint8_t *scales,
                       int *d_status) {
    fp4::Out o;
    o.codes = codes;
    o.scales = scales;
    o.global_scale = global_scale;
    o.d_status = d_status;
    o.K = K;
    o.tiles_k = fp4::scale_tiles_k(fmt, K);
    o.ceil_rule = scale_rule == W4_MX_SCALE_CEIL;
    return o;
}

inline w4_status clear_status(int *d_status, cudaStream_t st) {
    return !d_status || cudaMemsetAsync(d_status, 0, sizeof(int), st) == cudaSuccess ? W4_OK : W4_ERR_CUDA;
}

// Launch of a kernel whose first step is to wait for the previous one on the stream
// (pdl_wait_prior_grid): only its start overlaps that kernel's end.
template <typename... P, typename... A>
inline w4_status launch_behind(void (*kernel)(P...), unsigned grid, unsigned threads, size_t smem, cudaStream_t st,
                               A... args) {
    if (smem > 48 * 1024 - 1024 && !set_smem_limit(reinterpret_cast<const void *>(kernel), smem)) return W4_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid, 1, 1);
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...) == cudaSuccess ? launch_status() : W4_ERR_CUDA;
}

// This translation unit's sticky error word (each unit has its own, so the function is each
// unit's own too): added to *out if that is 0.
static inline w4_status take_device_error(int *out, int clear) {
    int v = 0;
    const int zero = 0;
    if (cudaMemcpyFromSymbol(&v, g_device_error, sizeof(int)) != cudaSuccess) return W4_ERR_CUDA;
    if (clear && cudaMemcpyToSymbol(g_device_error, &zero, sizeof(int)) != cudaSuccess) return W4_ERR_CUDA;
    if (*out == 0) *out = v;
    return W4_OK;
}

}  // namespace w4
