"""What the binding of the 4-bit operators refuses, with CUDA tensors."""
import pytest
import torch

import w4a16_matmul_pack_b200 as W4

pytestmark = pytest.mark.gpu


def x(M=4, K=64, dtype=torch.bfloat16):
    return torch.ones(M, K, dtype=dtype, device="cuda")


def refused(f, error=ValueError):
    with pytest.raises(error):
        f()


def test_quantize():
    refused(lambda: W4.fp4_quantize(x()[0]))                                  # one dimension
    refused(lambda: W4.fp4_quantize(x(64, 64).t()))                           # columns, not rows
    refused(lambda: W4.fp4_quantize(x(dtype=torch.float64)))
    refused(lambda: W4.fp4_quantize(x(), "nvfp4"))                            # no global scale
    refused(lambda: W4.fp4_quantize(x(), "nvfp4", global_scale=torch.ones(2, device="cuda")))
    refused(lambda: W4.fp4_quantize(x(), "nvfp4", global_scale=torch.ones(1)))
    refused(lambda: W4.fp4_quantize(x(K=48)), W4.W4Error)
    refused(lambda: W4.fp4_quantize(x(M=0)), W4.W4Error)
    refused(lambda: W4.fp4_quantize(x(1, 64).expand(4, 64)), W4.W4Error)      # rows on top of each other
    refused(lambda: W4.fp4_quantize(x(4, 72)[:, 1:65]), W4.W4Error)           # rows off 16 bytes
    q = W4.fp4_quantize(x())
    refused(lambda: W4.fp4_quantize(x(5), out=q))
    refused(lambda: W4.fp4_quantize(x(), "nvfp4", global_scale=torch.ones(1, device="cuda"), out=q))
    refused(lambda: W4.Fp4Tensor(W4.FMT_MXFP4, 4, 64, q.codes, q.scales[:-1]))
    refused(lambda: W4.Fp4Tensor(W4.FMT_MXFP4, 5, 64, q.codes, q.scales))
    refused(lambda: W4.Fp4Tensor(W4.FMT_NVFP4, 4, 64, q.codes, q.scales))
    refused(lambda: W4.fp4_from_rows("mxfp4", q.codes, torch.zeros(4, 3, dtype=torch.uint8, device="cuda")))
    refused(lambda: W4.fp4_from_packed(W4.pack_rocmfp4(x())))


def test_product():
    w, q = W4.fp4_quantize(x(8)), W4.fp4_quantize(x())
    refused(lambda: W4.w4a4_gemm(w, x()))
    refused(lambda: W4.w4a4_gemm(x(), q))
    refused(lambda: W4.w4a4_gemm(w, q, out_dtype=torch.float64))
    refused(lambda: W4.w4a4_gemm(w, q, out=torch.zeros(4, 9, device="cuda")))
    refused(lambda: W4.w4a4_gemm(w, W4.fp4_quantize(x(K=96))), W4.W4Error)
    refused(lambda: W4.w4a4_gemm(w, q, flags=4), W4.W4Error)
    refused(lambda: W4.w4a4_linear(w, x(K=96)))
    refused(lambda: W4.w4a4_linear(w, x(M=0)), W4.W4Error)
    ws = torch.empty(W4.w4a4_workspace_bytes(w, 40) - 16, dtype=torch.uint8, device="cuda")
    refused(lambda: W4.w4a4_linear(w, x(40), workspace=ws), W4.W4Error)
    nv = W4.fp4_quantize(x(8), "nvfp4", global_scale=torch.ones(1, device="cuda"))
    refused(lambda: W4.w4a4_linear(nv, x()), W4.W4Error)                      # no global scale of x
    refused(lambda: W4.w4a4_gemm(nv, q), W4.W4Error)                          # two formats


def test_block_norm():
    y = x()
    refused(lambda: W4.block_norm(y, x(5)))
    refused(lambda: W4.block_norm(y, x(dtype=torch.float32)))
    refused(lambda: W4.block_norm(y, post_weight=torch.ones(63, dtype=torch.bfloat16, device="cuda")))
    refused(lambda: W4.block_norm(y, pre_weight=torch.ones(64, device="cuda")))
    refused(lambda: W4.block_norm(y, gate=x(3)))
    refused(lambda: W4.block_norm(y, gate=x(2), gate_rows=1))
    refused(lambda: W4.block_norm(y, gate=x(), gate_act="gelu"))
    refused(lambda: W4.block_norm(y, quantize="nvfp4"))
    refused(lambda: W4.block_norm(y, out=x(dtype=torch.float16)))
    refused(lambda: W4.block_norm(y, out_h=x(5)))
    refused(lambda: W4.block_norm(x(K=40), quantize="mxfp4"), W4.W4Error)
    refused(lambda: W4.block_norm(x(1, 64).expand(4, 64)), W4.W4Error)
    refused(lambda: W4.block_norm(x(1, 32800)), W4.W4Error)
    refused(lambda: W4.block_norm(y, eps=-1.0), W4.W4Error)


def test_memory_of_a_call_on_another_stream():
    """What a call allocates belongs to the stream it runs on: a workspace given back
    while that stream is busy is not handed to the current stream, and a result does not
    take memory that the current stream still reads."""
    torch.manual_seed(0)
    w = W4.fp4_quantize(torch.randn(256, 1024, device="cuda").bfloat16())
    a = torch.randn(300, 1024, device="cuda").bfloat16()
    want = W4.w4a4_linear(w, a)
    need = W4.w4a4_workspace_bytes(w, 300)
    big = torch.randn(4096, 4096, device="cuda")
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        with torch.cuda.stream(st):
            big @ big                                  # keeps the stream busy
        y = W4.w4a4_linear(w, a, stream=st)
        others = [torch.full((need,), 255, dtype=torch.uint8, device="cuda") for _ in range(4)]
        torch.cuda.synchronize()
        assert torch.equal(y, want)
        del others
    src = torch.full((300, 256), 7.0, dtype=torch.bfloat16, device="cuda")
    dst = torch.zeros_like(src)
    torch.cuda.synchronize()
    big @ big
    dst.copy_(src)                                     # behind the product, on the current stream
    del src
    ys = [W4.w4a4_linear(w, a, stream=st) for _ in range(4)]
    torch.cuda.synchronize()
    assert (dst == 7).all() and all(torch.equal(y, want) for y in ys)
    with torch.cuda.stream(st):
        z = W4.block_norm(a, quantize="mxfp4")[1]
    st.synchronize()
    for f in (lambda: W4.fp4_quantize(a, stream=st), lambda: W4.block_norm(a, quantize="mxfp4", stream=st)[1]):
        q = f()
        st.synchronize()
        assert q.codes.shape == z.codes.shape and q.scales.numel() == z.scales.numel()
        assert q._buf.data_ptr() % 512 == 0
