"""W4A4 kernels that start while the kernel before them still runs: however long that
takes, no limit of theirs runs meanwhile, and what they read is what it wrote."""
import ctypes
import os
import subprocess

import pytest
import torch

import w4a16_matmul_pack_b200 as W4

pytestmark = pytest.mark.gpu

NS = 20_000_000      # the previous kernel's time; a wait limit of 1 us allows about 0.13 ms


@pytest.fixture(scope="module")
def slow_copy(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("slow") / "slow.so")
    src = os.path.join(os.path.dirname(os.path.abspath(__file__)), "slow_kernel.cu")
    subprocess.check_call([os.environ.get("NVCC", "nvcc"), "-gencode", "arch=compute_100a,code=sm_100a", "-shared",
                           "-Xcompiler", "-fPIC", "-o", so, src])
    f = ctypes.CDLL(so).slow_copy
    f.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_longlong, ctypes.c_longlong, ctypes.c_void_p]

    def run(src, dst, ns=NS):
        n = src.numel() * src.element_size()
        assert dst.numel() * dst.element_size() == n
        assert f(src.data_ptr(), dst.data_ptr(), n, ns, torch.cuda.current_stream().cuda_stream) == 0
    return run


@pytest.fixture(autouse=True)
def short_limit():
    W4.w4_device_error(clear=True)
    yield
    W4.set_wait_limit(0)
    W4.w4_device_error(clear=True)


def clone(q):
    return W4.Fp4Tensor(q.fmt, q.rows, q.K, torch.zeros_like(q.codes), q.scales.clone(), q.global_scale)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("flags", [0, W4.LAUNCH_PDL])
@pytest.mark.parametrize("M,N,K", [(1, 300, 1024), (16, 2560, 2560), (100, 256, 512), (200, 300, 1024), (200, 300, 4096),
                                   (300, 2560, 64)])
def test_product_behind_a_slow_kernel(slow_copy, fmt, flags, M, N, K):
    """x comes from a kernel that runs on for 20 ms, with a wait limit of 1 us; K of fewer
    stages than the rings hold, and of more."""
    gen = torch.Generator().manual_seed(M + K)
    g = torch.tensor([0.002], device="cuda") if fmt == "nvfp4" else None
    x = W4.fp4_quantize(torch.randn(M, K, generator=gen).cuda(), fmt, global_scale=g)
    w = W4.fp4_quantize(torch.randn(N, K, generator=gen).cuda(), fmt, global_scale=g)
    want = W4.w4a4_gemm(w, x, out_dtype=torch.float32)
    late, out = clone(x), torch.empty_like(want)
    torch.cuda.synchronize()
    W4.set_wait_limit(1000)
    slow_copy(x.codes, late.codes)
    W4.w4a4_gemm(w, late, out=out, flags=flags)
    torch.cuda.synchronize()
    assert W4.w4_device_error(clear=True) == 0
    assert torch.equal(out, want)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("M", [3, 40, 200])
def test_linear_and_norms_behind_a_slow_kernel(slow_copy, fmt, M):
    K, N = 1024, 300
    gen = torch.Generator().manual_seed(M)
    x = torch.randn(M, K, generator=gen).cuda().bfloat16()
    g = torch.tensor([0.002], device="cuda") if fmt == "nvfp4" else None
    w = W4.fp4_quantize(torch.randn(N, K, generator=gen).cuda(), fmt, global_scale=g)
    want = W4.w4a4_linear(w, x, global_scale=g)
    _, z = W4.block_norm(x, x, quantize=fmt, global_scale=g)
    want_z = W4.w4a4_gemm(w, z)
    late, out, ws = torch.zeros_like(x), torch.empty_like(want), W4.w4a4_workspace_bytes(w, M)
    ws = torch.empty(ws, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    W4.set_wait_limit(1000)
    slow_copy(x, late)
    W4.w4a4_linear(w, late, global_scale=g, out=out, workspace=ws)
    torch.cuda.synchronize()
    assert W4.w4_device_error(clear=True) == 0 and torch.equal(out, want)
    late.zero_()
    h = torch.empty_like(x)
    slow_copy(x, late)
    W4.block_norm(late, late, quantize=fmt, global_scale=g, out=z, out_h=h)
    W4.w4a4_gemm(w, z, out=out, flags=W4.LAUNCH_PDL)
    torch.cuda.synchronize()
    assert W4.w4_device_error(clear=True) == 0 and torch.equal(out, want_z)
