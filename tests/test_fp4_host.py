"""Host side of the 4-bit operators without a GPU: sizes of the scale tiles, and
every refusal before anything is launched (C ABI by dummy addresses, binding by
CPU tensors)."""
import ctypes

import pytest
import torch

import w4a16_matmul_pack_b200 as W4
from w4a16_matmul_pack_b200 import build as B

ARG, ALIGN, UNSUPPORTED, WORKSPACE = 1, 2, 3, 7
P, I, LL, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_float


class Fp4(ctypes.Structure):
    """w4_fp4 of include/w4a16.h."""
    _fields_ = [("fmt", I), ("rows", I), ("K", I), ("codes", P), ("scales", P), ("global_scale", P)]


class Norm(ctypes.Structure):
    """w4_norm of include/w4a16.h."""
    _fields_ = ([(n, I) for n in ("type", "M", "D")] + [(n, P) for n in ("y", "h", "w_post", "w_pre", "gate")]
                + [(n, LL) for n in ("ldy", "ldh", "ldgate")] + [(n, I) for n in ("gate_rows", "gate_act")]
                + [(n, F) for n in ("residual_scale", "block_scale", "eps", "weight_offset")]
                + [("h_out", P), ("ldh_out", LL), ("z", P), ("ldz", LL), ("quant_fmt", I), ("scale_rule", I)]
                + [(n, P) for n in ("global_scale", "codes", "scales", "d_status")])


@pytest.fixture(scope="module")
def lib():
    B.build()
    return W4.lib()


@pytest.mark.parametrize("rows,K,mx,nv", [(1, 32, 512, 512), (1, 128, 512, 1024), (128, 160, 1024, 1536),
                                          (129, 2560, 2 * 20 * 512, 2 * 40 * 512), (777, 2592, 7 * 21 * 512, 7 * 41 * 512)])
def test_scale_bytes(lib, rows, K, mx, nv):
    assert lib.fp4_scale_bytes(W4.FMT_MXFP4, rows, K) == mx
    assert lib.fp4_scale_bytes(W4.FMT_NVFP4, rows, K) == nv
    assert W4.fp4_scale_bytes(W4.FMT_MXFP4, rows, K) == mx and W4.fp4_scale_bytes(W4.FMT_NVFP4, rows, K) == nv


def test_packed_structs_are_the_headers():
    """The binding packs its structs as bytes: the same layout as the C structs."""
    v = (5, 7, 64, 1 << 40, 2 << 40, 3 << 40)
    assert W4._pack_fp4(*v) == bytes(Fp4(*v))
    v = (1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11, 12, 1, 1.5, 2.5, 3.5, 4.5, 13, 14, 15, 16, 5, 1, 17, 18, 19, 20)
    assert W4._pack_norm(*v) == bytes(Norm(*v))


def test_scale_bytes_of_bad_shapes(lib):
    assert lib.fp4_scale_bytes(2, 1, 32) == 0
    for rows, K in ((0, 32), (1, 0), (1, 16), (1, 48), (-1, 64)):
        assert lib.fp4_scale_bytes(W4.FMT_MXFP4, rows, K) == 0


def test_quantize_refusals(lib):
    def call(x=P(16), type=0, ldx=64, rows=2, K=64, fmt=5, rule=0, g=None, codes=P(16), scales=P(16), status=None):
        return lib.fp4_quantize(x, type, ldx, rows, K, fmt, rule, g, codes, scales, status, None)
    assert call(x=None) == ARG and call(codes=None) == ARG and call(scales=None) == ARG
    assert call(type=3) == ARG and call(type=-1) == ARG and call(fmt=2) == ARG and call(rule=2) == ARG
    assert call(rows=0) == ARG and call(K=48, ldx=48) == ARG and call(K=0) == ARG and call(ldx=63) == ARG
    assert call(fmt=1) == ARG                                   # NVFP4 without a global scale
    assert call(fmt=1, g=P(16), rule=1) == ARG                  # the rules are MXFP4's
    assert call(x=P(24)) == ALIGN and call(codes=P(24)) == ALIGN and call(scales=P(17)) == ALIGN
    assert call(ldx=68) == ALIGN and call(type=2, ldx=66) == ALIGN and call(status=P(18)) == ALIGN
    assert call(fmt=1, g=P(18)) == ALIGN


def operand(fmt=5, rows=8, K=64, codes=16, scales=16, g=None):
    return Fp4(fmt, rows, K, codes, scales, g)


def test_product_refusals(lib):
    def call(w=None, x=None, y=P(16), type=0, ldy=8, flags=0):
        return lib.w4a4_gemm(ctypes.byref(w or operand()), ctypes.byref(x or operand(rows=2)), y, type, ldy, flags, None)
    assert lib.w4a4_gemm(None, ctypes.byref(operand()), P(16), 0, 8, 0, None) == ARG
    assert call(y=None) == ARG and call(type=3) == ARG and call(ldy=7) == ARG and call(flags=2) == ARG
    assert call(w=operand(K=96)) == ARG and call(w=operand(fmt=1, g=16)) == ARG        # another K, another format
    assert call(w=operand(fmt=1), x=operand(fmt=1, rows=2, g=16)) == ARG               # a missing global scale
    assert call(w=operand(rows=0)) == ARG and call(x=operand(K=40)) == ARG and call(x=operand(scales=None)) == ARG
    assert call(w=operand(codes=20)) == ALIGN and call(x=operand(scales=24)) == ALIGN and call(y=P(20)) == ALIGN
    assert lib.fp4_dequantize(ctypes.byref(operand()), None, 0, 64, None) == ARG
    assert lib.fp4_dequantize(ctypes.byref(operand()), P(16), 0, 63, None) == ARG
    assert lib.fp4_dequantize(ctypes.byref(operand()), P(16), 0, 68, None) == ALIGN
    assert lib.fp4_tile_scales(5, 4, 48, P(16), P(16), None) == ARG
    assert lib.fp4_tile_scales(5, 4, 64, P(17), P(16), None) == ALIGN


def test_linear_refusals(lib):
    w = operand()
    need = lib.w4a4_workspace_bytes(ctypes.byref(w), 17)
    assert need >= 17 * 32 + 512
    assert lib.w4a4_workspace_bytes(ctypes.byref(w), 0) == lib.w4a4_workspace_bytes(ctypes.byref(w), 16) == 0
    for M in (1, 16, 17, 77, 129, 1000):       # the binding's own arithmetic
        for fmt, K in ((5, 64), (5, 2592), (1, 96)):
            c = operand(fmt, 8, K, g=16 if fmt == 1 else None)
            assert W4.w4a4_workspace_bytes(c, M) == lib.w4a4_workspace_bytes(ctypes.byref(c), M)

    def call(w=w, x=P(16), type=0, ldx=64, M=17, rule=0, g=None, y=P(16), out=0, ldy=8, ws=P(256), n=need):
        return lib.w4a4_linear(ctypes.byref(w), x, type, ldx, M, rule, g, y, out, ldy, ws, n, None, None)
    assert call(x=None) == ARG and call(M=0) == ARG and call(ldx=60) == ARG and call(type=5) == ARG
    assert call(ws=None) == WORKSPACE and call(n=need - 1) == WORKSPACE
    assert call(y=None) == ARG and call(out=3) == ARG and call(ldy=5) == ARG and call(rule=4) == ARG
    assert call(x=P(24)) == ALIGN and call(ldx=66) == ALIGN and call(ws=P(264)) == ALIGN and call(y=P(8)) == ALIGN
    assert call(w=operand(fmt=1, g=16), n=1 << 20) == ARG       # NVFP4 x without a global scale
    few = dict(M=16, ws=None, n=0)                              # no workspace, the same refusals
    assert call(**few, x=None) == ARG and call(**few, ldx=60) == ARG and call(**few, type=5) == ARG
    assert call(**few, y=None) == ARG and call(**few, out=3) == ARG and call(**few, ldy=5) == ARG and call(**few, rule=4) == ARG
    assert call(**few, x=P(24)) == ALIGN and call(**few, ldx=66) == ALIGN and call(**few, y=P(8)) == ALIGN
    assert call(**few, w=operand(fmt=1, g=16)) == ARG


def test_norm_refusals(lib):
    def call(**kw):
        d = dict(type=0, M=2, D=64, y=16, ldy=64, residual_scale=1.0, block_scale=1.0, eps=1e-6, z=16, ldz=64)
        d.update(kw)
        return lib.w4_block_norm(ctypes.byref(Norm(**d)), None)
    assert lib.w4_block_norm(None, None) == ARG
    assert call(y=None) == ARG and call(z=None) == ARG and call(M=0) == ARG and call(D=0) == ARG
    assert call(type=4) == ARG and call(ldy=63) == ARG and call(ldz=10) == ARG
    assert call(eps=-1.0) == ARG and call(eps=float("nan")) == ARG
    assert call(D=32769, ldy=40000, ldz=40000) == UNSUPPORTED and call(M=(1 << 30) + 1) == UNSUPPORTED
    assert call(h=16, ldh=3) == ARG and call(h_out=16, ldh_out=3) == ARG
    assert call(gate=16, ldgate=64, gate_rows=0) == ARG and call(gate=16, ldgate=10, gate_rows=1) == ARG
    assert call(gate_act=3) == ARG and call(gate_act=-1) == ARG
    assert call(y=17) == ALIGN and call(type=2, z=18) == ALIGN and call(w_pre=15) == ALIGN
    q = dict(z=None, quant_fmt=5, codes=16, scales=16)
    assert call(**dict(q, z=16)) == ARG and call(**dict(q, codes=None)) == ARG and call(**dict(q, quant_fmt=3)) == ARG
    assert call(**dict(q, D=40)) == ARG and call(**dict(q, quant_fmt=1)) == ARG and call(**dict(q, codes=20)) == ALIGN


def test_binding_refuses_cpu_tensors():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    for f in (lambda: W4.fp4_quantize(x), lambda: W4.block_norm(x), lambda: W4.block_norm(x, x),
              lambda: W4.fp4_from_rows("mxfp4", x.to(torch.uint8), x.to(torch.uint8)),
              lambda: W4.Fp4Tensor(W4.FMT_MXFP4, 4, 64, x.to(torch.uint8), x.to(torch.uint8))):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(ValueError):
        W4.fp4_quantize(x, "dual")


def test_largest_extents(lib):
    """Rows and K whose last tile would pass an int are refused, not wrapped."""
    top = 2 ** 31 - 256
    for fmt, per in ((W4.FMT_MXFP4, 128), (W4.FMT_NVFP4, 64)):
        for rows, K in ((top, 32), (1, top)):
            want = -(-rows // 128) * -(-K // per) * 512
            assert lib.fp4_scale_bytes(fmt, rows, K) == W4.fp4_scale_bytes(fmt, rows, K) == want
        for rows, K in ((top + 1, 32), (2 ** 31 - 1, 32), (1, 2 ** 31 - 32), (130, 2 ** 31 - 96)):
            assert lib.fp4_scale_bytes(fmt, rows, K) == W4.fp4_scale_bytes(fmt, rows, K) == 0
            g = 16 if fmt == W4.FMT_NVFP4 else None
            big, w = operand(fmt, rows, K, g=g), operand(fmt, 8, K, g=g)
            assert lib.fp4_quantize(P(16), 0, K, rows, K, fmt, 0, g, P(16), P(16), None, None) == UNSUPPORTED
            assert lib.fp4_dequantize(ctypes.byref(big), P(16), 0, K, None) == UNSUPPORTED
            assert lib.fp4_tile_scales(fmt, rows, K, P(16), P(16), None) == UNSUPPORTED
            assert lib.w4a4_gemm(ctypes.byref(big), ctypes.byref(w), P(16), 0, rows, 0, None) == UNSUPPORTED
            assert lib.w4a4_gemm(ctypes.byref(w), ctypes.byref(big), P(16), 0, 8, 0, None) == UNSUPPORTED
            assert lib.w4a4_linear(ctypes.byref(w), P(16), 0, K, rows, 0, g, P(16), 0, 8, P(256), 1 << 60, None,
                                   None) == UNSUPPORTED
