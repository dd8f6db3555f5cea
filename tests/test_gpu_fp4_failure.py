"""Failure detection of the W4A4 products without a GPU fault: with a wait limit so
short that the first waits expire, a call records W4_ERR_TIMEOUT in the sticky word
and returns; with the default limit restored the next call is right and records
nothing."""
import time

import pytest
import torch

import w4a16_matmul_pack_b200 as W4

pytestmark = pytest.mark.gpu

W4_ERR_TIMEOUT = 6


@pytest.fixture(autouse=True)
def default_limit_after():
    W4.w4_device_error(clear=True)
    yield
    W4.set_wait_limit(0)
    W4.w4_device_error(clear=True)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("M,N,K", [(1, 2560, 2560), (9, 256, 9728), (100, 512, 2560), (300, 1000, 4096), (2048, 2560, 2560)])
def test_expired_waits_are_reported_and_pass(fmt, M, N, K):
    g = torch.tensor([0.002], device="cuda") if fmt == "nvfp4" else None
    gen = torch.Generator().manual_seed(M)
    x = W4.fp4_quantize(torch.randn(M, K, generator=gen).cuda(), fmt, global_scale=g)
    w = W4.fp4_quantize(torch.randn(N, K, generator=gen).cuda(), fmt, global_scale=g)
    want = W4.w4a4_gemm(w, x, out_dtype=torch.float32)
    torch.cuda.synchronize()
    W4.set_wait_limit(1)                      # 1 ns: the first wait that does not pass at once expires
    t = time.monotonic()
    W4.w4a4_gemm(w, x, out_dtype=torch.float32)
    torch.cuda.synchronize()
    assert time.monotonic() - t < 30          # every wait of the way out is bounded
    assert W4.w4_device_error(clear=True) == W4_ERR_TIMEOUT
    W4.set_wait_limit(0)
    got = W4.w4a4_gemm(w, x, out_dtype=torch.float32)
    torch.cuda.synchronize()
    assert W4.w4_device_error(clear=True) == 0
    assert torch.equal(got, want)


def test_nonfinite_inputs_reach_the_sticky_word_from_every_kernel():
    """The norms, the quantiser and the weight packers share one sticky word."""
    bad = torch.full((2, 64), float("inf"), device="cuda")
    for call in (lambda: W4.fp4_quantize(bad), lambda: W4.block_norm(bad, quantize="mxfp4"),
                 lambda: W4.pack_nvfp4(bad.to(torch.bfloat16))):
        assert W4.w4_device_error(clear=True) == 0
        call()
        assert W4.w4_device_error(clear=False) == 5
        assert W4.w4_device_error(clear=True) == 5
        assert W4.w4_device_error(clear=True) == 0


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("M,N,K", [(8192, 2560, 9728), (2048, 9728, 2560), (300, 9728, 30016)])
def test_a_pair_that_gives_up_frees_no_more_stages(fmt, M, N, K):
    """Up to 190 stages per pair of CTAs, waits expired from the first one on.  The pair's
    MMA issuer stops with its waiter: stages freed after the first CTA has stopped arming
    its barriers would have the second CTA's loads counted on them, past what they hold.
    Three times over, then right results on the same memory."""
    g = torch.tensor([0.002], device="cuda") if fmt == "nvfp4" else None
    gen = torch.Generator(device="cuda").manual_seed(K)
    x = W4.fp4_quantize(torch.randn(M, K, generator=gen, device="cuda").bfloat16(), fmt, global_scale=g)
    w = W4.fp4_quantize(torch.randn(N, K, generator=gen, device="cuda").bfloat16(), fmt, global_scale=g)
    want = W4.w4a4_gemm(w, x)
    out = torch.empty_like(want)
    torch.cuda.synchronize()
    for _ in range(3):
        W4.set_wait_limit(1)
        t = time.monotonic()
        W4.w4a4_gemm(w, x, out=out)
        torch.cuda.synchronize()
        assert time.monotonic() - t < 30
        assert W4.w4_device_error(clear=True) == W4_ERR_TIMEOUT
        W4.set_wait_limit(0)
        assert torch.equal(W4.w4a4_gemm(w, x, out=out), want)
        assert W4.w4_device_error(clear=True) == 0


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("M,N,K", [(1, 2560, 2560), (9, 2560, 9728), (16, 20000, 2560), (100, 512, 2560), (300, 1000, 4096)])
def test_expired_waits_of_the_linear_layer(fmt, M, N, K):
    """The same through w4a4_linear: up to 16 tokens the product's warps that quantise x
    leave their ring, in its first round and in later ones."""
    g = torch.tensor([0.002], device="cuda") if fmt == "nvfp4" else None
    gen = torch.Generator(device="cuda").manual_seed(M)
    x = torch.randn(M, K, generator=gen, device="cuda").bfloat16()
    w = W4.fp4_quantize(torch.randn(N, K, generator=gen, device="cuda").bfloat16(), fmt, global_scale=g)
    want = W4.w4a4_linear(w, x, global_scale=g)
    torch.cuda.synchronize()
    for _ in range(2):
        W4.set_wait_limit(1)
        t = time.monotonic()
        W4.w4a4_linear(w, x, global_scale=g)
        torch.cuda.synchronize()
        assert time.monotonic() - t < 30
        assert W4.w4_device_error(clear=True) == W4_ERR_TIMEOUT
        W4.set_wait_limit(0)
        assert torch.equal(W4.w4a4_linear(w, x, global_scale=g), want)
        assert W4.w4_device_error(clear=True) == 0
