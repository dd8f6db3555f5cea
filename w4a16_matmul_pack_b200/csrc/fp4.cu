// fp4.cu -- the W4A4 part of the C ABI (declared in include/w4a16.h): host-side
// validation, launch configuration and launches of the sm_100a kernels that
// quantise activations to 4 bits and multiply two 4-bit operands.
#include <cuda_runtime.h>

#include <algorithm>

#include "fp4_host.cuh"
#include "fp4_pack.cuh"
#include "fp4_gemm.cuh"
#include "fp4_skinny.cuh"

using namespace w4;

namespace w4 {

int norm_device_error(int *out, int clear);   // norm.cu

// The sticky error word and the wait limit are one copy per translation unit;
// w4_device_error and w4_set_wait_limit act on those of the W4A4 kernels through
// these.
int fp4_device_error(int *out, int clear) {
    *out = 0;
    const w4_status s = take_device_error(out, clear);
    return s != W4_OK ? s : norm_device_error(out, clear);
}

int fp4_set_wait_limit(unsigned long long ns) {
    return cudaMemcpyToSymbol(g_wait_limit_ns, &ns, sizeof(ns)) == cudaSuccess ? W4_OK : W4_ERR_CUDA;
}

}  // namespace w4

namespace {

// Blocks of a pass over a matrix by lanes of 32 values, rows padded to whole scale words.
bool lane_blocks(int rows, int K, int &per_row, unsigned &blocks) {
    per_row = (K / 32 + 3) / 4 * 4;
    const long long n = ((long long)rows * per_row + 255) / 256;
    blocks = (unsigned)n;
    return n <= kMaxBlocks;
}

template <typename T, int FMT>
w4_status launch_quantize(const void *x, long long ldx, int rows, const fp4::Out &o, cudaStream_t st) {
    const T *p = reinterpret_cast<const T *>(x);
    const bool wide = (reinterpret_cast<uintptr_t>(x) | (uintptr_t)(ldx * sizeof(T))) % 32 == 0;
    int per_row;
    unsigned blocks;
    if (!lane_blocks(rows, o.K, per_row, blocks)) return W4_ERR_UNSUPPORTED;
    return launch_behind(wide ? fp4::quantize_kernel<T, FMT, true> : fp4::quantize_kernel<T, FMT, false>, blocks, 256,
                         0, st, p, ldx, rows, per_row, o);
}

template <typename T>
w4_status launch_quantize_fmt(const void *x, long long ldx, int rows, int fmt, const fp4::Out &o, cudaStream_t st) {
    return fmt == W4_FMT_MXFP4 ? launch_quantize<T, W4_FMT_MXFP4>(x, ldx, rows, o, st)
                               : launch_quantize<T, W4_FMT_NVFP4>(x, ldx, rows, o, st);
}

w4_status quantize(const void *x, int type, long long ldx, int rows, int fmt, const fp4::Out &o, cudaStream_t st) {
    switch (type) {
    case W4_TYPE_BF16: return launch_quantize_fmt<__nv_bfloat16>(x, ldx, rows, fmt, o, st);
    case W4_TYPE_F16: return launch_quantize_fmt<__half>(x, ldx, rows, fmt, o, st);
    case W4_TYPE_F32: return launch_quantize_fmt<float>(x, ldx, rows, fmt, o, st);
    }
    return W4_ERR_ARG;
}

template <typename T, int FMT>
w4_status launch_dequantize(const w4_fp4 *a, void *out, long long ldo, cudaStream_t st) {
    T *p = reinterpret_cast<T *>(out);
    const bool wide = (reinterpret_cast<uintptr_t>(out) | (uintptr_t)(ldo * sizeof(T))) % 32 == 0;
    int per_row;
    unsigned blocks;
    if (!lane_blocks(a->rows, a->K, per_row, blocks)) return W4_ERR_UNSUPPORTED;
    return launch_behind(wide ? fp4::dequantize_kernel<T, FMT, true> : fp4::dequantize_kernel<T, FMT, false>, blocks,
                         256, 0, st, a->codes, a->scales, a->global_scale, a->rows, a->K,
                         fp4::scale_tiles_k(FMT, a->K), per_row, p, ldo);
}

template <typename T>
w4_status launch_dequantize_fmt(const w4_fp4 *a, void *out, long long ldo, cudaStream_t st) {
    return a->fmt == W4_FMT_MXFP4 ? launch_dequantize<T, W4_FMT_MXFP4>(a, out, ldo, st)
                                  : launch_dequantize<T, W4_FMT_NVFP4>(a, out, ldo, st);
}

// ------------------------------------------------------------------ product --

// Codes [rows][K/2] bytes as boxes of 128 bytes x `box_rows`, 128-byte swizzle;
// bytes past a row's end and rows past the last arrive as zeros.
bool codes_map(CUtensorMap &map, const uint8_t *codes, int rows, int K, int box_rows) {
    PFN_encodeTiled enc = get_encode_tiled();
    const cuuint64_t dims[2] = {(cuuint64_t)K / 2, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)K / 2};
    const cuuint32_t box[2] = {fgemm::BK / 2, (cuuint32_t)box_rows};
    const cuuint32_t estr[2] = {1, 1};
    return enc && enc(&map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t *>(codes), dims, strides, box, estr,
                      CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// x of at most 16 tokens that the product quantises itself.
struct PlainX {
    const void *x;
    long long ldx;
    int rows, type, ceil_rule;
    const float *global_scale;
    int *d_status;
};

template <int FMT, int NT, typename T>
w4_status launch_skinny(const w4_fp4 *w, const w4_fp4 *x, const PlainX &plain, void *y, long long ldy, int out_type,
                        int splits, bool early_w, cudaStream_t st) {
    using namespace fgemm;
    constexpr bool fused = skinny::kFused<T>;
    const int M = fused ? plain.rows : x->rows;
    CUtensorMap wmap, xmap;
    if (!codes_map(wmap, w->codes, w->rows, w->K, BM)) return W4_ERR_CUDA;
    xmap = wmap;   // not read when x is quantised here
    if (!fused && !codes_map(xmap, x->codes, M, x->K, NT)) return W4_ERR_CUDA;
    constexpr size_t smem = sizeof(skinny::Shared<FMT, NT>) + 1024;
    static_assert(smem <= 227 * 1024, "shared memory of the product");
    auto kernel = skinny::gemm_kernel<FMT, NT, T>;
    if (!set_smem_limit(reinterpret_cast<const void *>(kernel), smem)) return W4_ERR_CUDA;
    skinny::Params p = {};
    p.sfw = w->scales;
    p.sfx = fused ? nullptr : x->scales;
    p.gw = FMT == W4_FMT_NVFP4 ? w->global_scale : nullptr;
    p.gx = FMT == W4_FMT_NVFP4 ? (fused ? plain.global_scale : x->global_scale) : nullptr;
    p.y = y;
    p.ldy = ldy;
    p.N = w->rows;
    p.M = M;
    p.K = w->K;
    p.tiles_n = (w->rows + BM - 1) / BM;
    p.tiles_k = fp4::scale_tiles_k(FMT, w->K);
    p.x = plain.x;
    p.ldx = plain.ldx;
    p.ceil_rule = plain.ceil_rule;
    p.d_status = plain.d_status;
    p.inv_m = M > 1 ? 0xFFFFFFFFu / (unsigned)M + 1u : 0u;
    p.splits = splits;
    p.out_type = out_type;
    p.early_w = early_w;
    const long long blocks = (long long)p.tiles_n * ((M + NT - 1) / NT) * splits;
    if (blocks > kMaxBlocks) return W4_ERR_UNSUPPORTED;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks, 1, 1);
    cfg.blockDim = dim3(skinny::kThreads<T>, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    // The kernel waits for the previous one on the stream before it reads x or writes
    // y (and, without early_w, before it reads w).
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = splits;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (cudaLaunchKernelEx(&cfg, kernel, wmap, xmap, p) != cudaSuccess) return W4_ERR_CUDA;
    return launch_status();
}

// Scale tiles as rows of 128 words, boxes of `tiles` rows; past the last row zeros.
bool scales_map(CUtensorMap &map, const uint8_t *scales, size_t bytes, int tiles) {
    PFN_encodeTiled enc = get_encode_tiled();
    const cuuint64_t dims[2] = {fgemm::SF_TILE / 4, (cuuint64_t)(bytes / fgemm::SF_TILE)};
    const cuuint64_t strides[1] = {fgemm::SF_TILE};
    const cuuint32_t box[2] = {fgemm::SF_TILE / 4, (cuuint32_t)tiles};
    const cuuint32_t estr[2] = {1, 1};
    return enc && enc(&map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<uint8_t *>(scales), dims, strides, box, estr,
                      CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// y as boxes of 32 rows x 128 bytes, 128-byte swizzle (rows on 16 bytes).
bool output_map(CUtensorMap &map, void *y, int rows, int cols, long long ldy, int type) {
    PFN_encodeTiled enc = get_encode_tiled();
    const int size = type_size(type);
    const CUtensorMapDataType t = type == W4_TYPE_BF16  ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                  : type == W4_TYPE_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                        : CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)ldy * size};
    const cuuint32_t box[2] = {(cuuint32_t)(128 / size), 32};
    const cuuint32_t estr[2] = {1, 1};
    return enc && enc(&map, t, 2, y, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                      CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int FMT, int NT>
w4_status launch_pair(const w4_fp4 *w, const w4_fp4 *x, void *y, long long ldy, int out_type, bool early_w, int sms,
                      cudaStream_t st) {
    using namespace fgemm;
    using namespace fgemm::pair;
    CUtensorMap xmap, wmap, sxmap, swmap;
    constexpr int ST = Scales<FMT>::TILES;
    if (!codes_map(xmap, x->codes, x->rows, x->K, BM) || !codes_map(wmap, w->codes, w->rows, w->K, NT / 2) ||
        !scales_map(sxmap, x->scales, fp4_scale_bytes(FMT, x->rows, x->K), ST) ||
        !scales_map(swmap, w->scales, fp4_scale_bytes(FMT, w->rows, w->K), ST))
        return W4_ERR_CUDA;
    constexpr size_t smem = sizeof(pair::Shared<FMT, NT>) + 1024;
    static_assert(smem <= 227 * 1024, "shared memory of the product");
    // y leaves as TMA boxes where its rows start on 16 bytes and, since a box is clipped
    // to the tensor in units of 16 bytes, end on them
    const bool tma = rows16(ldy, out_type) && rows16(w->rows, out_type);
    auto kernel = tma ? pair::gemm_kernel<FMT, NT, true> : pair::gemm_kernel<FMT, NT, false>;
    if (!set_smem_limit(reinterpret_cast<const void *>(kernel), smem)) return W4_ERR_CUDA;
    CUtensorMap ymap = xmap;   // not read without tma
    if (tma && !output_map(ymap, y, x->rows, w->rows, ldy, out_type)) return W4_ERR_CUDA;
    pair::Params p;
    p.gx = FMT == W4_FMT_NVFP4 ? x->global_scale : nullptr;
    p.gw = FMT == W4_FMT_NVFP4 ? w->global_scale : nullptr;
    p.out.y = y;
    p.out.ldy = ldy;
    p.out.rows = x->rows;
    p.out.cols = w->rows;
    p.out.type = out_type;
    p.K = x->K;
    p.early_w = early_w;
    p.tiles_m = (x->rows + 2 * BM - 1) / (2 * BM);
    p.tiles_n = (w->rows + NT - 1) / NT;
    p.tiles_k = fp4::scale_tiles_k(FMT, x->K);
    const long long ntiles = (long long)p.tiles_m * p.tiles_n;
    if (ntiles > kMaxBlocks) return W4_ERR_UNSUPPORTED;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * (unsigned)std::min<long long>(ntiles, std::max(1, sms / 2)), 1, 1);
    cfg.blockDim = dim3(pair::kThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (cudaLaunchKernelEx(&cfg, kernel, xmap, wmap, sxmap, swmap, ymap, p) != cudaSuccess) return W4_ERR_CUDA;
    return launch_status();
}

// Slices of K (CTAs of a cluster) for a product of `tiles` tiles of nt tokens: as few
// stages in a row as possible, an exchange of partial sums counted as the stages that
// take as long (0.3 us each; measured: 0.6 us at 16 tokens, 3.7 us at 128), and no more
// CTAs than run at once (at 16 tokens two fit an SM, and a few more than SMs still
// gain: 9728 x 2560, 9 tokens: 160 CTAs 6.3 us, 80 CTAs 6.7 us; at 64 tokens
// 152 CTAs 16 us, 76 CTAs 7.2 us).
int slices(long long tiles, int stages, int nt, int sms) {
    const long long room = nt <= 16 ? sms + sms / 8 : sms;
    const int exchange = nt <= 16 ? 2 : nt / 8;
    int best = 1, cost = stages;
    for (int s = 2; s <= fgemm::skinny::kMaxSplit && s <= stages && tiles * s <= room; s *= 2) {
        const int c = (stages + s - 1) / s + exchange;
        if (c < cost) best = s, cost = c;
    }
    return best;
}

template <int FMT, int NT, typename T = fgemm::skinny::Quantised>
w4_status few_tokens(const w4_fp4 *w, const w4_fp4 *x, void *y, long long ldy, int out_type, bool early_w, int sms,
                     cudaStream_t st, const PlainX &plain = {}) {
    const long long tiles = (w->rows + fgemm::BM - 1) / fgemm::BM;
    const int s = slices(tiles, (w->K + fgemm::BK - 1) / fgemm::BK, NT, sms);
    return launch_skinny<FMT, NT, T>(w, x, plain, y, ldy, out_type, s, early_w, st);
}

// The linear layer of at most kFusedTokens tokens in one kernel: for a call by itself the
// second launch costs the host 3.7 us, more than the GPU loses where it loses (nine NVFP4
// tokens, 9728 x 2560: 8.6 us, as two launches 7.4; one token, 2560 x 9728 MXFP4 6.0 and
// 6.6).
constexpr int kFusedTokens = 16;

template <int FMT>
w4_status fused_linear(const w4_fp4 *w, const PlainX &x, void *y, long long ldy, int out_type, cudaStream_t st) {
    int sms = 0;
    if (device_sms(sms) != W4_OK) return W4_ERR_CUDA;
    switch (x.type) {
    case W4_TYPE_BF16: return few_tokens<FMT, 16, __nv_bfloat16>(w, nullptr, y, ldy, out_type, false, sms, st, x);
    case W4_TYPE_F16: return few_tokens<FMT, 16, __half>(w, nullptr, y, ldy, out_type, false, sms, st, x);
    default: return few_tokens<FMT, 16, float>(w, nullptr, y, ldy, out_type, false, sms, st, x);
    }
}

// Width of a prompt's tiles: the least of launch + waves x max(stages x time per stage
// + time per tile, time to store a tile), in us: a least-squares fit to 22 shapes of
// 200 .. 8192 tokens, K 32 .. 30000, N 96 .. 9728 on 148 SMs (its choice is within 0.3%
// of the best on average, 14 shapes that were not fitted among them).  A stage is bound by its
// loads; tiles of 256 rows share tensor memory between two accumulators and wait for it
// (1.8 us a tile); short K is bound by the stores.  Measured at 128 / 192 / 256 rows
// (MXFP4): 2048 x 2560 x 9728 28.0 / 22.9 / 27.6 us; 8192 x 9728 x 2560 82.1 / 71.9 /
// 71.8; 512 x 2560 x 2560 7.2 / 8.0 / 9.0; 8192 x 256 x 1024 10.2 / 10.1 / 8.8.
int tile_width(int M, int N, int K, int sms) {
    const struct { int nt; double launch, stage, tile, store; } kinds[] = {
        {128, 4.33, 0.214, 0.59, 1.51}, {192, 4.49, 0.243, 0.86, 1.96}, {256, 3.95, 0.314, 1.80, 2.29}};
    const long long pairs = std::max(1, sms / 2), stages = (K + fgemm::BK - 1) / fgemm::BK;
    int best = 0;
    double least = 0;
    for (const auto &k : kinds) {
        const long long tiles = (long long)((M + 255) / 256) * ((N + k.nt - 1) / k.nt);
        const long long waves = (tiles + pairs - 1) / pairs;
        const double t = k.launch + (double)waves * std::max((double)stages * k.stage + k.tile, k.store);
        if (!best || t < least) best = k.nt, least = t;
    }
    return best;
}

template <int FMT>
w4_status gemm_fmt(const w4_fp4 *w, const w4_fp4 *x, void *y, long long ldy, int out_type, bool early_w,
                   cudaStream_t st) {
    const int M = x->rows;
    int sms = 0;
    if (device_sms(sms) != W4_OK) return W4_ERR_CUDA;
    // up to 128 tokens fit one tile of the kernel that streams weights (128 tokens,
    // 2560 x 2560: 7.9 us; a pair's tile of 256 tokens would be half empty)
    if (M <= 16) return few_tokens<FMT, 16>(w, x, y, ldy, out_type, early_w, sms, st);
    if (M <= 32) return few_tokens<FMT, 32>(w, x, y, ldy, out_type, early_w, sms, st);
    if (M <= 64) return few_tokens<FMT, 64>(w, x, y, ldy, out_type, early_w, sms, st);
    if (M <= 128) return few_tokens<FMT, 128>(w, x, y, ldy, out_type, early_w, sms, st);
    switch (tile_width(M, w->rows, w->K, sms)) {
    case 128: return launch_pair<FMT, 128>(w, x, y, ldy, out_type, early_w, sms, st);
    case 192: return launch_pair<FMT, 192>(w, x, y, ldy, out_type, early_w, sms, st);
    default: return launch_pair<FMT, 256>(w, x, y, ldy, out_type, early_w, sms, st);
    }
}

w4_status check_product(const w4_fp4 *w, const w4_fp4 *x, const void *y, long long ldy, int out_type) {
    w4_status s = check_operand(w);
    if (s != W4_OK) return s;
    if ((s = check_operand(x)) != W4_OK) return s;
    if (w->fmt != x->fmt || w->K != x->K || !y || !is_type(out_type) || ldy < w->rows) return W4_ERR_ARG;
    if (!aligned16(y)) return W4_ERR_ALIGN;
    return W4_OK;
}

w4_status product(const w4_fp4 *w, const w4_fp4 *x, void *y, long long ldy, int out_type, bool early_w,
                  cudaStream_t st) {
    return w->fmt == W4_FMT_MXFP4 ? gemm_fmt<W4_FMT_MXFP4>(w, x, y, ldy, out_type, early_w, st)
                                  : gemm_fmt<W4_FMT_NVFP4>(w, x, y, ldy, out_type, early_w, st);
}

// Codes first, then scales on the next 256 bytes.
size_t linear_scales_at(int rows, int K) { return ((size_t)rows * (K / 2) + 255) & ~(size_t)255; }

}  // namespace

// ======================================================================== ABI

extern "C" {

size_t fp4_scale_bytes(int fmt, int rows, int K) {
    if (!is_fp4(fmt) || rows < 1 || K < 32 || K % 32 || too_large(rows, K)) return 0;
    return ((size_t)rows + 127) / 128 * fp4::scale_tiles_k(fmt, K) * 512;
}

w4_status fp4_quantize(const void *x, int type, long long ldx, int rows, int K, int fmt, int scale_rule,
                       const float *global_scale, uint8_t *codes, uint8_t *scales, int *d_status, void *stream) {
    w4_status s = check_quantised(rows, K, fmt, scale_rule, global_scale, codes, scales, d_status);
    if (s != W4_OK) return s;
    if (!x || !is_type(type) || ldx < K) return W4_ERR_ARG;
    if (!aligned16(x) || !rows16(ldx, type)) return W4_ERR_ALIGN;
    cudaStream_t st = as_stream(stream);
    if (clear_status(d_status, st) != W4_OK) return W4_ERR_CUDA;
    return quantize(x, type, ldx, rows, fmt, quantised_out(K, fmt, scale_rule, global_scale, codes, scales, d_status),
                    st);
}

w4_status fp4_dequantize(const w4_fp4 *a, void *out, int type, long long ldo, void *stream) {
    const w4_status s = check_operand(a);
    if (s != W4_OK) return s;
    if (!out || !is_type(type) || ldo < a->K) return W4_ERR_ARG;
    if (!aligned16(out) || !rows16(ldo, type)) return W4_ERR_ALIGN;
    cudaStream_t st = as_stream(stream);
    if (type == W4_TYPE_BF16) return launch_dequantize_fmt<__nv_bfloat16>(a, out, ldo, st);
    if (type == W4_TYPE_F16) return launch_dequantize_fmt<__half>(a, out, ldo, st);
    return launch_dequantize_fmt<float>(a, out, ldo, st);
}

w4_status fp4_tile_scales(int fmt, int rows, int K, const uint8_t *row_scales, uint8_t *scales, void *stream) {
    if (!is_fp4(fmt) || rows < 1 || K < 32 || K % 32 || !row_scales || !scales) return W4_ERR_ARG;
    if (too_large(rows, K)) return W4_ERR_UNSUPPORTED;
    if (!aligned16(row_scales) || !aligned16(scales)) return W4_ERR_ALIGN;
    const int tiles_k = fp4::scale_tiles_k(fmt, K);
    const long long blocks = ((long long)rows * tiles_k + 255) / 256;
    if (blocks > kMaxBlocks) return W4_ERR_UNSUPPORTED;
    return launch_behind(fp4::tile_scales_kernel, (unsigned)blocks, 256, 0, as_stream(stream), row_scales, rows,
                         K / (fmt == W4_FMT_MXFP4 ? 32 : 16), tiles_k, scales);
}

w4_status w4a4_gemm(const w4_fp4 *w, const w4_fp4 *x, void *y, int out_type, long long ldy, unsigned flags,
                    void *stream) {
    const w4_status s = check_product(w, x, y, ldy, out_type);
    if (s != W4_OK) return s;
    if (flags & ~W4_LAUNCH_PDL) return W4_ERR_ARG;
    return product(w, x, y, ldy, out_type, (flags & W4_LAUNCH_PDL) != 0, as_stream(stream));
}

size_t w4a4_workspace_bytes(const w4_fp4 *w, int M) {
    if (check_operand(w) != W4_OK || M <= kFusedTokens) return 0;
    return linear_scales_at(M, w->K) + fp4_scale_bytes(w->fmt, M, w->K);
}

w4_status w4a4_linear(const w4_fp4 *w, const void *x, int type, long long ldx, int M, int scale_rule,
                      const float *global_scale, void *y, int out_type, long long ldy, void *workspace,
                      size_t workspace_bytes, int *d_status, void *stream) {
    w4_status s = check_operand(w);
    if (s != W4_OK) return s;
    if (M < 1 || !x || !is_type(type) || ldx < w->K) return W4_ERR_ARG;
    cudaStream_t st = as_stream(stream);
    if (M <= kFusedTokens) {
        // y's and x's arguments, checked as for an operand in w's own codes
        const w4_fp4 q = {w->fmt, M, w->K, w->codes, w->scales, global_scale};
        if ((s = check_quantised(M, w->K, w->fmt, scale_rule, global_scale, q.codes, q.scales, d_status)) != W4_OK)
            return s;
        if ((s = check_product(w, &q, y, ldy, out_type)) != W4_OK) return s;
        if (!aligned16(x) || !rows16(ldx, type)) return W4_ERR_ALIGN;
        if (clear_status(d_status, st) != W4_OK) return W4_ERR_CUDA;
        const PlainX p = {x, ldx, M, type, scale_rule == W4_MX_SCALE_CEIL, global_scale, d_status};
        return w->fmt == W4_FMT_MXFP4 ? fused_linear<W4_FMT_MXFP4>(w, p, y, ldy, out_type, st)
                                      : fused_linear<W4_FMT_NVFP4>(w, p, y, ldy, out_type, st);
    }
    if (!workspace || workspace_bytes < w4a4_workspace_bytes(w, M)) return W4_ERR_WORKSPACE;
    uint8_t *codes = reinterpret_cast<uint8_t *>(workspace), *scales = codes + linear_scales_at(M, w->K);
    const w4_fp4 q = {w->fmt, M, w->K, codes, scales, global_scale};
    if ((s = check_quantised(M, w->K, w->fmt, scale_rule, global_scale, codes, scales, d_status)) != W4_OK) return s;
    if ((s = check_product(w, &q, y, ldy, out_type)) != W4_OK) return s;
    if (!aligned16(x) || !rows16(ldx, type)) return W4_ERR_ALIGN;
    if (clear_status(d_status, st) != W4_OK) return W4_ERR_CUDA;
    s = quantize(x, type, ldx, M, w->fmt,
                 quantised_out(w->K, w->fmt, scale_rule, global_scale, codes, scales, d_status), st);
    if (s != W4_OK) return s;
    // the kernel just launched does not write the weights
    return product(w, &q, y, ldy, out_type, true, st);
}

}  // extern "C"
