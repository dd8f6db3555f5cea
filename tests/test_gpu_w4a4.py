"""The W4A4 product on the GPU against 64-bit products of the values its operands
stand for, and runs of the operators together.

Tolerance (fp4_ref.product_bound): two binary32 truncations of the running sum per
step of 64 k, plus half a step of the output type."""
import threading

import numpy as np
import pytest
import torch

import fp4_ref as R
import w4a16_inputs as I
import w4a16_matmul_pack_b200 as W4

pytestmark = pytest.mark.gpu

FMTS = ["mxfp4", "nvfp4"]
TYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.fixture(autouse=True)
def clean_error_word():
    W4.w4_device_error(clear=True)
    yield
    assert W4.w4_device_error(clear=True) == 0


def scale_of(x):
    return torch.tensor([max(float(x.float().abs().max()), 1e-30) / 2688.0 * 1.013], device="cuda")


def operand(x, fmt):
    """(Fp4Tensor, its values in 64 bits)."""
    q = W4.fp4_quantize(x.cuda(), fmt, global_scale=scale_of(x) if fmt == "nvfp4" else None)
    return q, values_of(q, fmt)


def values_of(q, fmt):
    s, _ = R.untile(q.scales.cpu().numpy(), q.rows, q.K, fmt)
    return R.values(R.nibbles(q.codes.cpu().numpy()), s, fmt, None if q.global_scale is None else q.global_scale.item())


def randn(*shape, seed, scale=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * scale).to(torch.bfloat16)


def check(y, xv, wv, dtype):
    yr, a = R.product(xv, wv)
    assert y.dtype == dtype and tuple(y.shape) == yr.shape
    got = R.f64(y)
    bound = R.product_bound(a, xv.shape[1])
    err = np.abs(got - yr)
    ok = err <= bound + R.half_step(np.abs(yr) + bound, dtype)
    assert ok.all(), (int((~ok).sum()), float(err.max()), np.argwhere(~ok)[:4].tolist())


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,N,K", [
    (1, 128, 256), (1, 1, 32), (1, 77, 64), (2, 8, 96), (7, 129, 128), (8, 256, 160), (9, 333, 288), (16, 128, 2592),
    (17, 40, 512), (33, 128, 1024), (64, 200, 544), (65, 129, 320), (128, 128, 256), (129, 127, 1056), (200, 300, 2048),
    (257, 1, 64), (300, 1000, 416), (513, 640, 2592)])
def test_shapes(fmt, M, N, K):
    x, xv = operand(randn(M, K, seed=M + K), fmt)
    w, wv = operand(randn(N, K, seed=N + K + 1, scale=0.02), fmt)
    check(W4.w4a4_gemm(w, x, out_dtype=torch.float32), xv, wv, torch.float32)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M", [1, 5, 16, 17, 40, 64, 65, 130, 300])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("N", [201, 200, 196, 192])
def test_output_types_and_row_distance(fmt, M, dtype, N):
    K = 384
    x, xv = operand(randn(M, K, seed=M), fmt)
    w, wv = operand(randn(N, K, seed=9, scale=0.02), fmt)
    check(W4.w4a4_gemm(w, x, out_dtype=dtype), xv, wv, dtype)
    for width in (N + 3, 256):
        wide = torch.full((M + 1, width), 5.0, dtype=dtype, device="cuda")
        y = W4.w4a4_gemm(w, x, out=wide[:M, :N])
        check(y, xv, wv, dtype)
        assert (wide[M] == 5).all() and (wide[:, N:] == 5).all()    # nothing beside or behind the rows


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,N,K", [
    (513, 1001, 2592), (300, 9728, 256), (1300, 3333, 800), (2304, 4104, 160), (700, 6100, 608), (1025, 9700, 288),
    (2100, 3999, 320)])
def test_wide_tiles(fmt, dtype, M, N, K):
    """Prompts whose tiles are 128, 192 (the next three) and 256 rows of w (the last
    three) on 148 SMs, one to several tiles per CTA pair; rows of y on and off 16 bytes."""
    x, xv = operand(randn(M, K, seed=M + K), fmt)
    w, wv = operand(randn(N, K, seed=N + K + 1, scale=0.02), fmt)
    check(W4.w4a4_gemm(w, x, out_dtype=dtype), xv, wv, dtype)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,K,N", [(1, 2560, 9728), (9, 9728, 2560), (16, 4096, 2560), (48, 2560, 1024), (2048, 2560, 1024)])
def test_layer_shapes(fmt, M, K, N):
    """The projections' shapes, weights with outliers; sampled rows of w, every token."""
    x, xv = operand(I.activations(M, K, 5, outlier_cols=16), fmt)
    W = I.matrix("student_t4", N, K, 6, 0.02, 1e-4)
    if fmt == "nvfp4":
        w = W4.fp4_from_packed(W4.pack_nvfp4(W.cuda()))
    else:
        w = W4.fp4_quantize(W.cuda(), fmt)
    wv = values_of(w, fmt)
    rows = np.unique(np.concatenate([np.arange(130), np.arange(N - 130, N), np.arange(0, N, 97)]))
    y = W4.w4a4_gemm(w, x, out_dtype=torch.float32)
    check(y[:, torch.from_numpy(rows).cuda()], xv, wv[rows], torch.float32)


@pytest.mark.parametrize("M", [3, 40, 100, 300])
def test_exact_sums(M):
    """Small integers under scale 1: every partial sum is exact, so is the result."""
    rng = np.random.default_rng(M)
    N, K = 150, 512
    xc, wc = rng.integers(0, 16, (M, K), dtype=np.uint8), rng.integers(0, 16, (N, K), dtype=np.uint8)
    for fmt, one in (("mxfp4", 127), ("nvfp4", 0x38)):
        g = torch.ones(1, device="cuda") if fmt == "nvfp4" else None
        ops = [W4.fp4_from_rows(fmt, torch.from_numpy(R.pack(c)).cuda(),
                                torch.full((c.shape[0], K // R.BLOCK[fmt]), one, dtype=torch.uint8, device="cuda"), g)
               for c in (wc, xc)]
        y = W4.w4a4_gemm(*ops, out_dtype=torch.float32)
        assert np.array_equal(R.f64(y), R.e2m1_values(xc) @ R.e2m1_values(wc).T)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M", [3, 40, 130])
def test_every_scale_lands_on_its_block(fmt, M):
    """One nonzero block per row of x at a time, every block scale different."""
    rng = np.random.default_rng(1)
    N, K = 140, 1088
    B = R.BLOCK[fmt]
    ops, vals = [], []
    for rows_, lo in ((N, 0), (M, 1)):
        codes = rng.integers(0, 16, (rows_, K), dtype=np.uint8)
        if lo:
            keep = rng.integers(0, K // B, rows_)
            keep[:min(rows_, K // B)] = np.arange(K // B)[:rows_]
            codes *= (np.arange(K)[None] // B == keep[:, None])
        sc = rng.integers(100, 150, (rows_, K // B), dtype=np.uint8) if fmt == "mxfp4" else \
            rng.integers(1, 0x7F, (rows_, K // B), dtype=np.uint8)
        g = torch.tensor([0.37 + lo], device="cuda") if fmt == "nvfp4" else None
        ops.append(W4.fp4_from_rows(fmt, torch.from_numpy(R.pack(codes)).cuda(), torch.from_numpy(sc).cuda(), g))
        vals.append(R.values(codes, sc, fmt, None if g is None else g.item()))
    check(W4.w4a4_gemm(ops[0], ops[1], out_dtype=torch.float32), vals[1], vals[0], torch.float32)


@pytest.mark.parametrize("M", [2, 150])
def test_extreme_scales(M):
    """MXFP4 scales whose product is in range though neither is; NVFP4 global scales
    whose product leaves binary32's range while the result does not."""
    N, K = 130, 256
    x, w = randn(M, K, seed=1).float(), randn(N, K, seed=2).float()
    xq, xv = operand(x * 2.0 ** 100, "mxfp4")
    wq, wv = operand(w * 2.0 ** -110, "mxfp4")
    check(W4.w4a4_gemm(wq, xq, out_dtype=torch.float32), xv, wv, torch.float32)
    for gx, gw in ((2.0 ** 90, 2.0 ** 45), (2.0 ** -80, 2.0 ** -60), (0.0, 1.0)):
        g = [torch.tensor([v], device="cuda") for v in (gx, gw)]
        sx = 2.0 ** -16 if gx > 1 else 1.0
        xq = W4.fp4_quantize((x * sx).cuda(), "nvfp4", global_scale=torch.ones(1, device="cuda"))
        wq = W4.fp4_quantize((w * sx).cuda(), "nvfp4", global_scale=torch.ones(1, device="cuda"))
        xq, wq = (W4.Fp4Tensor(q.fmt, q.rows, q.K, q.codes, q.scales, s) for q, s in ((xq, g[0]), (wq, g[1])))
        check(W4.w4a4_gemm(wq, xq, out_dtype=torch.float32), values_of(xq, "nvfp4"), values_of(wq, "nvfp4"),
              torch.float32)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M", [1, 20, 130])
def test_nan_rows_stay_in_their_rows(fmt, M):
    N, K = 140, 320
    x = randn(M, K, seed=3)
    x[M // 2, 77] = float("nan")
    w = randn(N, K, seed=4)
    w[5, 300] = float("inf")
    g = torch.tensor([0.002], device="cuda") if fmt == "nvfp4" else None
    xq, wq = (W4.fp4_quantize(t.cuda(), fmt, global_scale=g) for t in (x, w))
    assert W4.w4_device_error(clear=True) == 5
    y = R.f64(W4.w4a4_gemm(wq, xq, out_dtype=torch.float32))
    nan = np.zeros((M, N), bool)
    nan[M // 2], nan[:, 5] = True, True
    assert np.array_equal(np.isnan(y), nan) and np.isfinite(y[~nan]).all()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M", [1, 12, 50, 70, 260])
@pytest.mark.parametrize("dtype", TYPES)
def test_linear_is_quantise_then_product(fmt, M, dtype):
    N, K = 160, 672
    x = randn(M, K, seed=M).to(dtype).cuda()
    g = scale_of(x) if fmt == "nvfp4" else None
    w, _ = operand(randn(N, K, seed=2, scale=0.02), fmt)
    y = W4.w4a4_linear(w, x, global_scale=g, out_dtype=dtype)
    assert torch.equal(y, W4.w4a4_gemm(w, W4.fp4_quantize(x, fmt, global_scale=g), out_dtype=dtype))
    wide = torch.zeros(M, K + 16, dtype=dtype, device="cuda")
    wide[:, 16:] = x
    ws = torch.empty(W4.w4a4_workspace_bytes(w, M), dtype=torch.uint8, device="cuda")
    assert torch.equal(y, W4.w4a4_linear(w, wide[:, 16:], global_scale=g, out_dtype=dtype, workspace=ws))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M", [1, 9, 300])
def test_a_decoder_layers_path(fmt, M):
    """norms -> 4-bit z -> product -> norms -> product, as a layer runs them: each
    product is that of the operand the norm returned, each norm that of its inputs."""
    D, F = 512, 1376
    y, h = randn(M, D, seed=1).cuda(), randn(M, D, seed=2, scale=2.0).cuda()
    w1, w1v = operand(randn(F, D, seed=3, scale=0.05), fmt)
    w2, w2v = operand(randn(D, F, seed=4, scale=0.03), fmt)
    ones = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    g = torch.tensor([6.0 / 2688], device="cuda") if fmt == "nvfp4" else None
    h1, z = W4.block_norm(y, h, post_weight=ones, pre_weight=ones, quantize=fmt, global_scale=g)
    up = W4.w4a4_gemm(w1, z)
    check(up, values_of(z, fmt), w1v, torch.bfloat16)
    act = torch.relu(up)
    gs = scale_of(act) if fmt == "nvfp4" else None
    down = W4.w4a4_linear(w2, act, global_scale=gs)
    check(down, values_of(W4.fp4_quantize(act, fmt, global_scale=gs), fmt), w2v, torch.bfloat16)
    h2, z2 = W4.block_norm(down, h1, post_weight=ones, pre_weight=ones)
    hn, zn = R.block_norm(R.f64(down), R.f64(h1), np.ones(D), np.ones(D), None, None, 1, 1.0, 1.0,
                          float(np.float32(1e-6)), 0.0)
    size = np.abs(hn - R.f64(h1)) + np.abs(R.f64(h1))
    assert np.all(np.abs(R.f64(h2) - hn) <= 2.0 ** -18 * size + R.half_step(hn, torch.bfloat16) * 1.01)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M", [1, 16, 200])
def test_captured_replayed_and_on_other_streams(fmt, M):
    """The same bits from a graph (replayed on new x in place), a side stream, and
    two threads at once with workspaces of their own."""
    N, K = 300, 1280
    w, _ = operand(randn(N, K, seed=1, scale=0.02), fmt)
    xs = [randn(M, K, seed=10 + i).cuda() for i in range(3)]
    g = torch.tensor([0.002], device="cuda") if fmt == "nvfp4" else None
    want = [W4.w4a4_linear(w, x, global_scale=g) for x in xs]
    assert torch.equal(want[0], W4.w4a4_linear(w, xs[0], global_scale=g))
    x, y = xs[0].clone(), torch.empty_like(want[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        W4.w4a4_linear(w, x, global_scale=g, out=y)
    for i in (1, 2, 0):
        x.copy_(xs[i])
        graph.replay()
        assert torch.equal(y, want[i])
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        a = W4.w4a4_linear(w, xs[1], global_scale=g)
    b = W4.w4a4_linear(w, xs[2], global_scale=g, stream=st)
    torch.cuda.current_stream().wait_stream(st)
    assert torch.equal(a, want[1]) and torch.equal(b, want[2])
    got = {}

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(20):
                got[i] = W4.w4a4_linear(w, xs[i], global_scale=g)
            torch.cuda.current_stream().synchronize()
    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("M", [1, 16, 20, 300])
def test_x_made_by_a_kernel_that_is_still_running(M):
    """Every call waits for the kernel that makes its inputs (x, the global scale), however
    long that takes, and the caller may overwrite x right behind it."""
    N, K = 256, 1024
    w, _ = operand(randn(N, K, seed=1, scale=0.02), "nvfp4")
    xs = [randn(M, K, seed=5 + i).cuda() for i in range(2)]
    gs = [scale_of(x) for x in xs]
    want = [W4.w4a4_linear(w, x, global_scale=g) for x, g in zip(xs, gs)]
    x, g = torch.empty_like(xs[0]), torch.empty(1, device="cuda")
    big = torch.randn(4096, 4096, device="cuda")
    for i in range(12):
        (big @ big)                                # keeps the stream busy
        x.copy_(xs[i % 2])
        g.copy_(gs[i % 2])
        y = W4.w4a4_linear(w, x, global_scale=g)
        q = W4.fp4_quantize(x, "nvfp4", global_scale=g)
        x.zero_(), g.zero_()                       # behind the calls
        assert torch.equal(y, want[i % 2])
        q2 = W4.fp4_quantize(xs[i % 2], "nvfp4", global_scale=gs[i % 2])
        assert torch.equal(q.codes, q2.codes)


def test_weights_read_before_the_previous_kernel_ends():
    """W4_LAUNCH_PDL behind the kernel that makes x: the same bits."""
    w, _ = operand(randn(2560, 2560, seed=1, scale=0.02), "mxfp4")
    for M in (1, 200):
        y, h = randn(M, 2560, seed=2).cuda(), randn(M, 2560, seed=3).cuda()
        _, z = W4.block_norm(y, h, quantize="mxfp4")
        want = W4.w4a4_gemm(w, z)
        for i in range(20):
            y2 = y * (1 if i % 2 else -1)
            h2 = h * (1 if i % 2 else -1)
            W4.block_norm(y2, h2, quantize="mxfp4", out=z)
            got = W4.w4a4_gemm(w, z, flags=W4.LAUNCH_PDL)
            assert torch.equal(got, want if i % 2 else -want)


def test_rows_and_columns_past_many_tiles():
    """More tiles than SMs in both directions, ragged; the output's offsets pass 2^31."""
    fmt, K = "mxfp4", 64
    M, N = 20000, 110000
    x, xv = operand(randn(M, K, seed=1), fmt)
    w, wv = operand(randn(N, K, seed=2), fmt)
    y = W4.w4a4_gemm(w, x)
    assert M * N > 2 ** 31
    mr, nr = np.array([0, 1, 127, 128, 9999, 19998, 19999]), np.array([0, 5, 255, 256, 55555, 109998, 109999])
    got = y[torch.from_numpy(mr).cuda()][:, torch.from_numpy(nr).cuda()]
    check(got, xv[mr], wv[nr], torch.bfloat16)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M", [1, 9, 300])
def test_the_normalised_result_of_a_layer(fmt, M):
    """The second block norm of a layer: z too, within test_gpu_block_norm's bound."""
    D, F = 512, 1376
    y, h = randn(M, D, seed=1).cuda(), randn(M, D, seed=2, scale=2.0).cuda()
    w1, _ = operand(randn(F, D, seed=3, scale=0.05), fmt)
    w2, _ = operand(randn(D, F, seed=4, scale=0.03), fmt)
    post, pre = ((1 + randn(D, seed=s, scale=0.1).float()).to(torch.bfloat16).cuda() for s in (5, 6))
    g = torch.tensor([6.0 / 2688], device="cuda") if fmt == "nvfp4" else None
    h1, z = W4.block_norm(y, h, post_weight=post, pre_weight=pre, quantize=fmt, global_scale=g)
    act = torch.relu(W4.w4a4_gemm(w1, z))
    down = W4.w4a4_linear(w2, act, global_scale=scale_of(act) if fmt == "nvfp4" else None)
    h2, z2 = W4.block_norm(down, h1, post_weight=post, pre_weight=pre)
    hn, zn = R.block_norm(R.f64(down), R.f64(h1), R.f64(post), R.f64(pre), None, None, 1, 1.0, 1.0,
                          float(np.float32(1e-6)), 0.0)
    size = np.abs(hn - R.f64(h1)) + np.abs(R.f64(h1))
    assert np.all(np.abs(R.f64(h2) - hn) <= 2.0 ** -18 * size + R.half_step(hn, torch.bfloat16) * 1.01)
    zsize = size / np.sqrt((hn * hn).mean(1, keepdims=True) + 1e-6) * np.abs(R.f64(pre))
    assert np.all(np.abs(R.f64(z2) - zn) <= 2.0 ** -17 * zsize + R.half_step(zn, torch.bfloat16) * 1.01)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("K,N", [(2560, 9728), (9728, 2560), (2560, 20000), (4128, 19100)])
def test_fused_linear_goes_round_its_ring(fmt, K, N):
    """Up to 16 tokens with more stages of 256 k in a slice than the ring holds (5 in MXFP4,
    4 in NVFP4): up to four rounds and five, the last ragged; the same bits as quantising
    first, whose product goes by other loads."""
    w = W4.fp4_quantize(torch.randn(N, K, generator=torch.Generator("cuda").manual_seed(K), device="cuda").bfloat16(), fmt,
                        global_scale=torch.tensor([0.002], device="cuda") if fmt == "nvfp4" else None)
    for M, dtype in ((1, torch.bfloat16), (1, torch.float32), (9, torch.bfloat16), (9, torch.float16),
                     (16, torch.bfloat16), (16, torch.float32)):
        x = randn(M, K, seed=M).to(dtype).cuda()
        x[:, ::160] *= 30
        g = scale_of(x) if fmt == "nvfp4" else None
        y = W4.w4a4_linear(w, x, global_scale=g, out_dtype=torch.float32)
        assert torch.equal(y, W4.w4a4_gemm(w, W4.fp4_quantize(x, fmt, global_scale=g), out_dtype=torch.float32)), (M, dtype)
