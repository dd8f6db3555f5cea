"""The 4-bit operand quantiser on the GPU: codes and scales are bit-exact against
the numpy form (every step of the definition is exact or a named binary32
operation), the tiled scale layout, decoding, strided inputs, special values."""
import numpy as np
import pytest
import torch

import fp4_ref as R
import w4a16_inputs as I
import w4a16_matmul_pack_b200 as W4

pytestmark = pytest.mark.gpu

W4_ERR_NONFINITE = 5
DTYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.fixture(autouse=True)
def clean_error_word():
    W4.w4_device_error(clear=True)
    yield
    W4.w4_device_error(clear=True)


def rows(M, K, seed, dtype, spread=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, K, generator=g, dtype=torch.float64)
    if spread:   # blocks of very different size
        x *= torch.exp2(torch.randint(-9, 8, (M, K // 16), generator=g).repeat_interleave(16, 1).double())
    return x.to(dtype)


def g_of(x, g=None):
    g = float(x.float().abs().max()) / 2688.0 * 1.013 if g is None else g
    return torch.tensor([g], dtype=torch.float32, device="cuda")


def check(x, fmt, g=None, q=None, ceil=False):
    gt = g_of(x, g) if fmt == "nvfp4" else None
    if q is None:
        q = W4.fp4_quantize(x.cuda(), fmt, global_scale=gt, scale_rule=W4.MX_SCALE_CEIL if ceil else W4.MX_SCALE_FLOOR)
    gv = None if gt is None else gt.item()
    codes, scales = R.quantize(R.f32(x), fmt, gv, ceil)
    M, K = x.shape
    got, pad = R.untile(q.scales.cpu().numpy(), M, K, fmt)
    assert np.array_equal(got, scales)
    assert not pad.any()
    assert np.array_equal(R.nibbles(q.codes.cpu().numpy()), codes)
    # decoded: e2m1 * scale (* g) has at most 30 significant bits, so the 64-bit value
    # is exact and binary32 rounds it once; 4 * 2^126 (3e38 under the ceil rule) is
    # above binary32's range and rounds to Inf
    with np.errstate(all="ignore"):
        v = R.values(codes, scales, fmt, gv)
        d = W4.fp4_dequantize(q, torch.float32).cpu().numpy()
        assert np.array_equal(d, v.astype(np.float32), equal_nan=True)
    if fmt == "mxfp4":
        b = W4.fp4_dequantize(q, torch.bfloat16)
        assert np.array_equal(b.float().cpu().numpy(), d, equal_nan=True)
    return q


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,K", [(1, 32), (1, 2560), (3, 64), (7, 96), (31, 288), (129, 2592), (130, 544), (257, 128)])
def test_bit_exact(fmt, dtype, M, K):
    check(rows(M, K, M + K, dtype), fmt)


@pytest.mark.parametrize("dtype", DTYPES)
def test_ceil_rule_never_saturates(dtype):
    x = rows(33, 320, 5, dtype)
    q = check(x, "mxfp4", ceil=True)
    d = R.f64(W4.fp4_dequantize(q, torch.float32))
    top = np.abs(R.f64(x)).reshape(33, 10, 32).max(-1)
    # no value is further off than half the widest gap between levels (6 - 4 = 2 scales,
    # the scale being more than amax / 12 and at most amax / 3 ... / 6)
    assert np.all(np.abs(d - R.f64(x)).reshape(33, 10, 32).max(-1) <= top / 3)
    assert np.all(np.abs(d).reshape(33, 10, 32).max(-1) >= top * (1 - 1 / 3))


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_every_tie_and_boundary(fmt):
    """Values on and beside every rounding boundary, scale 1 (a 4 or 6 in each block)."""
    mids = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]
    vals = [s * v for m in mids for v in (np.nextafter(np.float32(m), np.float32(0)), m,
                                          np.nextafter(np.float32(m), np.float32(9))) for s in (1, -1)]
    vals += [0.0, -0.0, 0.5, 1.0, 6.0, -6.0]
    x = np.zeros((4, 64), np.float32)
    for i, v in enumerate(vals):
        x[i // 14, i % 14] = v
    x[:, 15::16] = 6.0 if fmt == "nvfp4" else 4.0
    check(torch.from_numpy(x), fmt, g=1.0)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_zero_blocks_and_extremes(fmt):
    x = torch.zeros(5, 128)
    x[1, 3] = 3.0e38
    x[1, 40] = -2.5e-38
    x[2, :32] = 1e-45                      # binary32's smallest value
    x[2, 32:64] = 2.0 ** -126
    x[2, 64:96] = 2.0 ** -125
    x[2, 96:] = 7.9 * 2.0 ** -127
    x[3, 5] = -0.0
    x[4] = 2.0 ** 127
    for g in ([None] if fmt == "mxfp4" else [0.0, 1.0, 1e-30, 1e-42, 3.0e38]):
        check(x, fmt, g=1.0 if g is None else g)
    if fmt == "mxfp4":
        check(x, fmt, ceil=True)


@pytest.mark.parametrize("g", [0.0, -1.0, float("inf")])
def test_global_scales_that_leave_nothing(g):
    """No value has a code under a global scale of zero, a negative or an infinite one:
    all zeros."""
    x = rows(3, 64, 2, torch.float32)
    q = W4.fp4_quantize(x.cuda(), "nvfp4", global_scale=torch.tensor([g], device="cuda"))
    scales, _ = R.untile(q.scales.cpu().numpy(), 3, 64, "nvfp4")
    assert not scales.any() and not (q.codes & 0x77).any()


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("dtype", DTYPES)
def test_nonfinite_blocks_are_nan(fmt, dtype):
    x = rows(4, 256, 9, dtype, spread=False)
    x[0, 17] = float("nan")
    x[1, 200] = float("inf")
    x[3, 31] = float("-inf")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    g = torch.tensor([0.002], device="cuda")
    q = W4.fp4_quantize(x.cuda(), fmt, global_scale=g if fmt == "nvfp4" else None, d_status=status)
    check(x, fmt, g=g.item(), q=q)
    assert status.item() == W4_ERR_NONFINITE
    assert W4.w4_device_error(clear=True) == W4_ERR_NONFINITE
    d = W4.fp4_dequantize(q).float().cpu()
    B = R.BLOCK[fmt]
    assert d[0, 17 // B * B:][:B].isnan().all() and d.isnan().sum() == 3 * B
    # a call on finite rows clears the status again
    W4.fp4_quantize(torch.zeros(1, 32, device="cuda"), "mxfp4", d_status=status)
    assert status.item() == 0


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("dtype", DTYPES)
def test_row_strides(fmt, dtype):
    big = rows(9, 512, 3, dtype).cuda()
    for view in (big[:, :256], big[:, 64:352], big[::2, 128:160], big[4:5, 8:40]):
        if view.data_ptr() % 16:
            continue
        check(view.cpu(), fmt, q=W4.fp4_quantize(view, fmt, global_scale=g_of(view.cpu()) if fmt == "nvfp4" else None))


def test_nvfp4_scales_are_the_packers():
    """With the packer's global scale the block scales are the packer's; so are the
    codes wherever one multiplication and one division round alike."""
    W = I.matrix("student_t4", 96, 512, 3, 0.02, 1e-3)
    pw = W4.pack_nvfp4(W.cuda())
    q = W4.fp4_quantize(W.cuda(), "nvfp4", global_scale=pw.global_scale)
    s, _ = R.untile(q.scales.cpu().numpy(), 96, 512, "nvfp4")
    assert np.array_equal(s, pw.scales.cpu().numpy())
    p = W4.fp4_from_packed(pw)
    # (the tile's rows behind the last are not written)
    assert np.array_equal(R.untile(p.scales.cpu().numpy(), 96, 512, "nvfp4")[0], s) and p.codes is pw.codes
    assert (q.codes != pw.codes).float().mean().item() < 0.02


@pytest.mark.parametrize("fmt,rows_,K", [("mxfp4", 1, 32), ("mxfp4", 130, 96), ("nvfp4", 257, 2592), ("nvfp4", 5, 64)])
def test_from_rows_layout(fmt, rows_, K):
    rng = np.random.default_rng(rows_ + K)
    codes = torch.from_numpy(rng.integers(0, 256, (rows_, K // 2), dtype=np.uint8)).cuda()
    scales = rng.integers(0, 0x7F, (rows_, K // R.BLOCK[fmt]), dtype=np.uint8)
    g = torch.tensor([0.5], device="cuda") if fmt == "nvfp4" else None
    q = W4.fp4_from_rows(fmt, codes, torch.from_numpy(scales).cuda(), g)
    got, pad = R.untile(q.scales.cpu().numpy(), rows_, K, fmt)
    assert np.array_equal(got, scales) and not pad.any()


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_nothing_written_past_the_result(fmt):
    """Canaries behind codes and around the scale words of the rows; rows of the last
    tile that do not exist are left as they were."""
    M, K = 70, 160
    x = rows(M, K, 4, torch.bfloat16)
    sb = W4.fp4_scale_bytes(W4._FP4_FMTS[fmt], M, K)
    codes = torch.full((M * K // 2 + 256,), 0xA5, dtype=torch.uint8, device="cuda")
    scales = torch.full((sb + 256,), 0xA5, dtype=torch.uint8, device="cuda")
    g = g_of(x) if fmt == "nvfp4" else None
    out = W4.Fp4Tensor(W4._FP4_FMTS[fmt], M, K, codes[:M * K // 2].view(M, K // 2), scales[:sb], g)
    assert W4.fp4_quantize(x.cuda(), fmt, global_scale=g, out=out) is out
    check(x, fmt, q=out)
    assert (codes[M * K // 2:] == 0xA5).all() and (scales[sb:] == 0xA5).all()
    per = K // R.BLOCK[fmt]
    assert (scales[:sb] != 0xA5).sum().item() <= M * (-(-per // 4)) * 4
    d = torch.full((M + 1, K + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    W4.fp4_dequantize(out, out=d[:M, :K])
    assert (d[M] == 7).all() and (d[:, K:] == 7).all()


def test_large_matrix_offsets_pass_32_bits():
    """Rows whose values lie more than 2^31 elements behind the first."""
    M, K = 2 ** 21 + 3, 1056
    x = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    tail = rows(3, K, 8, torch.bfloat16)
    x[-3:] = tail.cuda()
    q = W4.fp4_quantize(x, "mxfp4")
    del x
    codes, scales = R.quantize(R.f32(tail), "mxfp4")
    assert np.array_equal(R.nibbles(q.codes[-3:].cpu().numpy()), codes)
    d = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
    W4.fp4_dequantize(q, out=d)
    assert np.array_equal(R.f64(d[-3:]), R.values(codes, scales, "mxfp4"))
    assert not d[:-3].any()
