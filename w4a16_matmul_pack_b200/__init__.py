"""Python binding of libw4a16.so -- block-scaled 4-bit weight-only (W4A16) linear
layers on B200 (sm_100a).

Argument marshalling only: every step runs in the CUDA kernels behind the C ABI
declared in ``include/w4a16.h``.  PyTorch supplies device memory and streams.
The functions keep the C names:

    pack_nvfp4(W)            -> PackedWeights   (NVFP4: E2M1 + E4M3/16 + FP32 global)
    pack_rocmfp4(W, fmt)     -> PackedWeights   (ROCmFP4 Dual / FAST, Codebook10)
    w4a16_gemv(w, x)         -> y float32 [M][N]  (decode, M <= 16)
    w4a16_gemm(w, x)         -> (y float32, y bf16) (prefill)

and, with both operands in 4 bits (MXFP4 or NVFP4):

    fp4_quantize(x, fmt)     -> Fp4Tensor        (activations, or weights)
    fp4_from_packed(w)       -> Fp4Tensor        (NVFP4 PackedWeights, codes shared)
    w4a4_gemm(w, x)          -> y [M][N]         (any M, x an Fp4Tensor)
    w4a4_linear(w, x)        -> y [M][N]         (quantises x, then multiplies)
    block_norm(y, h, ...)    -> (h', z)          (post-norm, gate, residual, pre-norm; z may be an Fp4Tensor)

There is no CPU fallback: if the library is missing the import of a function
raises, and every call requires CUDA tensors.
"""
from __future__ import annotations

import ctypes
import os
import struct
from dataclasses import dataclass
from typing import Optional

import torch

__all__ = [
    "W4Error", "PackedWeights", "FMT_NVFP4", "FMT_ROCMFP4_DUAL", "FMT_ROCMFP4_FAST", "FMT_Q4_0",
    "pack_q4_0", "reconstruction_error", "plan_grouped",
    "LAUNCH_PDL", "set_wait_limit", "pack_nvfp4", "pack_rocmfp4", "w4a16_gemv", "w4a16_gemv_grouped", "w4a16_gemm",
    "w4a16_workspace_bytes", "pack_nvfp4_workspace_bytes", "w4_encode_scalars", "save_packed", "load_packed",
    "w4_device_error", "lib", "library_path",
    "Fp4Tensor", "FMT_MXFP4", "MX_SCALE_FLOOR", "MX_SCALE_CEIL", "fp4_quantize", "fp4_dequantize", "fp4_from_rows",
    "fp4_from_packed", "fp4_scale_bytes", "w4a4_gemm", "w4a4_linear", "w4a4_workspace_bytes", "block_norm",
]

FMT_NVFP4, FMT_ROCMFP4_DUAL, FMT_ROCMFP4_FAST, FMT_Q4_0, FMT_MXFP4 = 1, 2, 3, 4, 5
MX_SCALE_FLOOR, MX_SCALE_CEIL = 0, 1
SCALE_ABSMAX, SCALE_MSE = 0, 1
LAUNCH_PDL = 1
BLOCK_BYTES = {FMT_ROCMFP4_DUAL: 18, FMT_ROCMFP4_FAST: 17}
_FMT_NAMES = {"nvfp4": FMT_NVFP4, "dual": FMT_ROCMFP4_DUAL, "fast": FMT_ROCMFP4_FAST}

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libw4a16.so")


def library_path() -> str:
    return _LIB_PATH


class W4Error(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {lib().w4_status_string(status).decode()}")


class _Weights(ctypes.Structure):
    _fields_ = [("fmt", ctypes.c_int), ("K", ctypes.c_int), ("N", ctypes.c_int),
                ("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("global_scale", ctypes.c_void_p)]


_lib = None


def lib():
    """The loaded C library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(f"{_LIB_PATH} is missing: build it with "
                               "`python -m w4a16_matmul_pack_b200.build` (nvcc, sm_100a)")
        L = ctypes.CDLL(_LIB_PATH)
        P, I, U, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_uint, ctypes.c_size_t
        WP, LL = ctypes.POINTER(_Weights), ctypes.c_longlong
        sig = {
            "pack_nvfp4": ([P, I, I, I, I, P, P, P, P, S, P, P], I),
            "pack_nvfp4_ex": ([P, I, I, I, I, P, P, P, P, P, S, P, P], I),
            "pack_q4_0": ([P, I, I, I, P, P, P], I),
            "w4_plan_grouped": ([P, I, I, U, P], I),
            "w4_reconstruction_error": ([WP, P, P, P, S, P], I),
            "w4_reconstruction_workspace_bytes": ([], S),
            "pack_nvfp4_workspace_bytes": ([], S),
            "pack_rocmfp4": ([P, I, I, I, I, P, P, P, P], I),
            "w4a16_gemv": ([WP, P, I, P, P, S, P], I),
            "w4a16_gemv_ex": ([WP, P, I, P, P, S, U, P], I),
            "w4a16_gemv_grouped": ([WP, P, P, I, U, P], I),
            "w4a16_gemm": ([WP, P, I, P, P, P, S, P], I),
            "w4a16_workspace_bytes": ([WP, I], S),
            "w4_encode_scalars": ([P, S, P, P, P], I),
            "w4_device_error": ([ctypes.POINTER(ctypes.c_int), I], I),
            "w4_set_wait_limit": ([ctypes.c_ulonglong], I),
            "fp4_scale_bytes": ([I, I, I], S),
            "fp4_quantize": ([P, I, LL, I, I, I, I, P, P, P, P, P], I),
            "fp4_dequantize": ([P, P, I, LL, P], I),
            "fp4_tile_scales": ([I, I, I, P, P, P], I),
            "w4a4_gemm": ([P, P, P, I, LL, U, P], I),
            "w4a4_workspace_bytes": ([P, I], S),
            "w4a4_linear": ([P, P, I, LL, I, I, P, P, I, LL, P, S, P, P], I),
            "w4_block_norm": ([P, P], I),
            "w4_status_string": ([I], ctypes.c_char_p),
            "w4_version": ([], ctypes.c_char_p),
        }
        for name, (args, res) in sig.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = res
        _lib = L
    return _lib


def _check(status: int, what: str):
    if status != 0:
        raise W4Error(status, what)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _cuda(t: torch.Tensor, name: str, dtype=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (no CPU path)")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _stream(stream) -> ctypes.c_void_p:
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


@dataclass
class PackedWeights:
    """A packed K x N weight matrix (layout in include/w4a16.h)."""
    fmt: int
    K: int
    N: int
    codes: torch.Tensor                   # uint8: NVFP4 [N][K/2]; ROCmFP4 [N][K/32][18|17]
    scales: Optional[torch.Tensor] = None  # uint8 [N][K/16] (NVFP4)
    global_scale: Optional[torch.Tensor] = None  # float32 [1] (NVFP4)

    def struct(self) -> _Weights:
        return _Weights(self.fmt, self.K, self.N, self.codes.data_ptr(),
                        None if self.scales is None else self.scales.data_ptr(),
                        None if self.global_scale is None else self.global_scale.data_ptr())

    @property
    def nbytes(self) -> int:
        n = self.codes.numel()
        if self.scales is not None:
            n += self.scales.numel()
        return n


# Packed weights on disk: a 64-byte little-endian header, then the codes, the
# scales and the global scale as stored in memory.  Header: magic "W4A16PK",
# layout version (1), then int32 fmt, K, N, block, and int64 byte counts of
# codes, scales and global scale.
_MAGIC = b"W4A16PK"
_LAYOUT_VERSION = 1
_HEADER = struct.Struct("<7sB4i3q")


def _expected_bytes(fmt: int, K: int, N: int):
    if fmt == FMT_NVFP4:
        return N * K // 2, N * K // 16, 4
    if fmt in BLOCK_BYTES or fmt == FMT_Q4_0:
        return N * (K // 32) * (18 if fmt in (FMT_ROCMFP4_DUAL, FMT_Q4_0) else 17), 0, 0
    raise ValueError(f"unknown format {fmt}")


def save_packed(w: "PackedWeights", path) -> None:
    """Write packed weights with a versioned header (format, K, N, block, sizes)."""
    parts = [w.codes, w.scales, w.global_scale]
    raw = [b"" if t is None else t.detach().contiguous().cpu().view(torch.uint8).numpy().tobytes() for t in parts]
    if tuple(len(r) for r in raw) != _expected_bytes(w.fmt, w.K, w.N):
        raise ValueError("packed tensors do not match their format and shape")
    block = 16 if w.fmt == FMT_NVFP4 else 32
    with open(path, "wb") as f:
        f.write(_HEADER.pack(_MAGIC, _LAYOUT_VERSION, w.fmt, w.K, w.N, block, *(len(r) for r in raw)))
        f.write(b"\0" * (64 - _HEADER.size))
        for r in raw:
            f.write(r)


def load_packed(path, device="cuda") -> "PackedWeights":
    """Read packed weights written by save_packed; refuses unknown versions and
    headers whose sizes do not match the format and shape."""
    with open(path, "rb") as f:
        head = f.read(64)
        if len(head) != 64:
            raise ValueError("truncated header")
        magic, ver, fmt, K, N, block, nc, ns, ng = _HEADER.unpack(head[:_HEADER.size])
        if magic != _MAGIC or ver != _LAYOUT_VERSION:
            raise ValueError(f"not a packed-weights file of layout version {_LAYOUT_VERSION}")
        if K <= 0 or N <= 0 or block != (16 if fmt == FMT_NVFP4 else 32) or K % block:
            raise ValueError("bad shape in header")
        if (nc, ns, ng) != _expected_bytes(fmt, K, N):
            raise ValueError("byte counts do not match the format and shape")
        data = [f.read(n) for n in (nc, ns, ng)]
        if [len(d) for d in data] != [nc, ns, ng] or f.read(1):
            raise ValueError("truncated or oversized payload")
    def t(b, shape, dtype):
        return torch.frombuffer(bytearray(b), dtype=torch.uint8).view(dtype).reshape(shape).to(device)
    if fmt == FMT_NVFP4:
        return PackedWeights(fmt, K, N, t(data[0], (N, K // 2), torch.uint8), t(data[1], (N, K // 16), torch.uint8),
                             t(data[2], (1,), torch.float32))
    bb = nc // (N * (K // 32))
    return PackedWeights(fmt, K, N, t(data[0], (N, K // 32, bb), torch.uint8))


def pack_nvfp4_workspace_bytes() -> int:
    return lib().pack_nvfp4_workspace_bytes()


def pack_nvfp4(W: torch.Tensor, *, scale_search: int = SCALE_ABSMAX, importance: Optional[torch.Tensor] = None,
               out: Optional[PackedWeights] = None, workspace: Optional[torch.Tensor] = None,
               d_status: Optional[torch.Tensor] = None, stream=None) -> PackedWeights:
    """Quantise bf16 W[N][K] to NVFP4 (see pack_nvfp4 / pack_nvfp4_ex in include/w4a16.h);
    importance: float32 [K] channel weights for the W4_SCALE_MSE search."""
    _cuda(W, "W", torch.bfloat16)
    if importance is not None:
        _cuda(importance, "importance", torch.float32)
    N, K = W.shape
    dev = W.device
    if out is None:
        out = PackedWeights(FMT_NVFP4, K, N,
                            torch.empty(N, K // 2, dtype=torch.uint8, device=dev),
                            torch.empty(N, K // 16, dtype=torch.uint8, device=dev),
                            torch.empty(1, dtype=torch.float32, device=dev))
    if workspace is None:
        workspace = torch.empty(pack_nvfp4_workspace_bytes(), dtype=torch.uint8, device=dev)
    _check(lib().pack_nvfp4_ex(_ptr(W), K, N, 16, scale_search, _ptr(importance), _ptr(out.codes),
                               _ptr(out.scales), _ptr(out.global_scale), _ptr(workspace), workspace.numel(),
                               _ptr(d_status), _stream(stream)), "pack_nvfp4_ex")
    return out


def pack_rocmfp4(W: torch.Tensor, fmt="dual", *, importance: Optional[torch.Tensor] = None,
                 out: Optional[torch.Tensor] = None, d_status: Optional[torch.Tensor] = None,
                 stream=None) -> PackedWeights:
    """Quantise bf16 W[N][K] to ROCmFP4 Dual ("dual") or FAST ("fast"); importance:
    float32 [K] channel weights for the error search, or None."""
    fmt = _FMT_NAMES.get(fmt, fmt)
    _cuda(W, "W", torch.bfloat16)
    if importance is not None:
        _cuda(importance, "importance", torch.float32)
    N, K = W.shape
    if fmt not in BLOCK_BYTES:
        raise ValueError("fmt must be 'dual' or 'fast'")
    if out is None:
        out = torch.empty(N, K // 32, BLOCK_BYTES[fmt], dtype=torch.uint8, device=W.device)
    _check(lib().pack_rocmfp4(_ptr(W), K, N, 32, fmt, _ptr(importance), _ptr(out), _ptr(d_status),
                              _stream(stream)),
           "pack_rocmfp4")
    return PackedWeights(fmt, K, N, out)


def pack_q4_0(W: torch.Tensor, *, out: Optional[torch.Tensor] = None, d_status: Optional[torch.Tensor] = None,
              stream=None) -> PackedWeights:
    """Stock Q4_0, the comparison format (see pack_q4_0 in include/w4a16.h)."""
    _cuda(W, "W", torch.bfloat16)
    N, K = W.shape
    if out is None:
        out = torch.empty(N, K // 32, 18, dtype=torch.uint8, device=W.device)
    _check(lib().pack_q4_0(_ptr(W), K, N, 32, _ptr(out), _ptr(d_status), _stream(stream)), "pack_q4_0")
    return PackedWeights(FMT_Q4_0, K, N, out)


def reconstruction_error(w: PackedWeights, W: torch.Tensor, *, workspace: Optional[torch.Tensor] = None,
                         stream=None):
    """(sum (W - w_hat)^2, sum W^2) in binary64 for a packed matrix and its bf16
    source (see w4_reconstruction_error); reads the two numbers back to the host."""
    _cuda(W, "W", torch.bfloat16)
    out = torch.empty(2, dtype=torch.float64, device=W.device)
    if workspace is None:
        workspace = torch.empty(lib().w4_reconstruction_workspace_bytes(), dtype=torch.uint8, device=W.device)
    s = w.struct()
    _check(lib().w4_reconstruction_error(ctypes.byref(s), _ptr(W), _ptr(out), _ptr(workspace), workspace.numel(),
                                         _stream(stream)), "w4_reconstruction_error")
    e, q = out.tolist()
    return e, q


def w4a16_workspace_bytes(w: PackedWeights, M: int) -> int:
    s = w.struct()
    return lib().w4a16_workspace_bytes(ctypes.byref(s), M)


def w4a16_gemv(w: PackedWeights, x: torch.Tensor, *, out: Optional[torch.Tensor] = None,
               workspace: Optional[torch.Tensor] = None, flags: int = 0, stream=None) -> torch.Tensor:
    """y[M][N] = x[M][K] . w_hat for M <= 16 (float32 output)."""
    _cuda(x, "x", torch.bfloat16)
    M = x.shape[0]
    if out is None:
        out = torch.empty(M, w.N, dtype=torch.float32, device=x.device)
    need = w4a16_workspace_bytes(w, M)
    if workspace is None and need:
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    s = w.struct()
    _check(lib().w4a16_gemv_ex(ctypes.byref(s), _ptr(x), M, _ptr(out), _ptr(workspace),
                               0 if workspace is None else workspace.numel(), flags, _stream(stream)),
           "w4a16_gemv")
    return out


def plan_grouped(ws, sms: int, flags: int = 0):
    """Host only: the CTAs w4a16_gemv_grouped gives each problem on `sms` SMs."""
    G = len(ws)
    structs = (_Weights * G)(*[w.struct() for w in ws])
    out = (ctypes.c_int * G)()
    _check(lib().w4_plan_grouped(ctypes.cast(structs, ctypes.c_void_p), G, sms, flags,
                                 ctypes.cast(out, ctypes.c_void_p)), "w4_plan_grouped")
    return list(out)


def w4a16_gemv_grouped(ws, xs, *, outs=None, flags: int = 0, stream=None):
    """Several one-token NVFP4 GEMVs in one launch: returns [y_p[1][N_p] float32]."""
    G = len(ws)
    if len(xs) != G or (outs is not None and len(outs) != G):
        raise W4Error(-1, "w4a16_gemv_grouped: ws, xs and outs must have the same length")
    for x in xs:
        _cuda(x, "x", torch.bfloat16)
    if outs is None:
        outs = [torch.empty(1, w.N, dtype=torch.float32, device=xs[0].device) for w in ws]
    structs = (_Weights * G)(*[w.struct() for w in ws])
    xp = (ctypes.c_void_p * G)(*[_ptr(x) for x in xs])
    yp = (ctypes.c_void_p * G)(*[_ptr(y) for y in outs])
    _check(lib().w4a16_gemv_grouped(structs, ctypes.cast(xp, ctypes.c_void_p), ctypes.cast(yp, ctypes.c_void_p), G,
                                    flags, _stream(stream)), "w4a16_gemv_grouped")
    return outs


def w4a16_gemm(w: PackedWeights, x: torch.Tensor, *, want_f32: bool = True, want_bf16: bool = True,
               out_f32: Optional[torch.Tensor] = None, out_bf16: Optional[torch.Tensor] = None,
               workspace: Optional[torch.Tensor] = None, stream=None):
    """Prefill GEMM: returns (y float32 or None, y bf16 or None)."""
    _cuda(x, "x", torch.bfloat16)
    M = x.shape[0]
    if want_f32 and out_f32 is None:
        out_f32 = torch.empty(M, w.N, dtype=torch.float32, device=x.device)
    if want_bf16 and out_bf16 is None:
        out_bf16 = torch.empty(M, w.N, dtype=torch.bfloat16, device=x.device)
    need = w4a16_workspace_bytes(w, M)
    if workspace is None and need:
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    s = w.struct()
    _check(lib().w4a16_gemm(ctypes.byref(s), _ptr(x), M, _ptr(out_f32), _ptr(out_bf16), _ptr(workspace),
                            0 if workspace is None else workspace.numel(), _stream(stream)), "w4a16_gemm")
    return out_f32, out_bf16


# ------------------------------------------------------- 4-bit activations ----
#
# These calls take a few microseconds on the GPU for a single token, so the host
# side counts: tensors are checked by their cheapest accessors, structs are packed
# as bytes, and an operand's codes and scales share one allocation.

_TYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
_FP4_FMTS = {"mxfp4": FMT_MXFP4, "nvfp4": FMT_NVFP4, FMT_MXFP4: FMT_MXFP4, FMT_NVFP4: FMT_NVFP4}
_GATES = {"none": 0, "sigmoid": 1, "tanh": 2}
_MAX_EXTENT = 2 ** 31 - 256   # rows and K of an operand
_FUSED_TOKENS = 16   # tokens up to which w4a4_linear needs no workspace
_pack_fp4 = struct.Struct("@iiiPPP").pack                              # w4_fp4
_pack_norm = struct.Struct("@iiiPPPPPqqqiiffffPqPqiiPPPP").pack        # w4_norm
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _fp4_fmt(fmt) -> int:
    f = _FP4_FMTS.get(fmt)
    if f is None:
        raise ValueError("fmt must be 'mxfp4' or 'nvfp4'")
    return f


def _type(t: torch.Tensor, name: str) -> int:
    v = _TYPES.get(t.dtype)
    if v is None:
        raise ValueError(f"{name} must be bfloat16, float16 or float32, got {t.dtype}")
    return v


def _new(rows: int, width: int, dtype, device, stream=None) -> torch.Tensor:
    """torch.empty((rows, width)), by the call that costs the host least.  It belongs to the
    stream the call runs on, as if the caller had made that stream the current one: what the
    current stream still reads is not handed out, nor is what this stream still writes."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return _new(rows, width, dtype, device)
    return torch.empty_strided((rows, width), (width, 1), dtype=dtype, device=device)


def _rows(t: torch.Tensor, name: str, dev=None, rows=None, width=None):
    """(data pointer, row distance, rows, width) of a 2-D CUDA tensor with contiguous
    rows, on device `dev` and of the given shape where these are given."""
    try:
        d = t.get_device()
        (r, w), (s0, s1) = t.shape, t.stride()
    except (AttributeError, TypeError, ValueError):
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor (no CPU path)") from None
        raise ValueError(f"{name} must have two dimensions, got {tuple(t.shape)}") from None
    if d < 0:
        raise ValueError(f"{name} must be a CUDA tensor (no CPU path)")
    if (rows is not None and (r != rows or w != width)) or (dev is not None and d != dev):
        raise ValueError(f"{name} must have shape {(rows, width)} on cuda:{dev}, got {(r, w)} on {t.device}")
    if s1 != 1 and w > 1:
        raise ValueError(f"{name} must have contiguous rows")
    return t.data_ptr(), s0 if r > 1 else w, r, w


def _vector(t: Optional[torch.Tensor], name: str, dtype, dev: int, n: int) -> int:
    """Data pointer of an optional contiguous tensor of n values on device dev (0: none)."""
    if t is None:
        return 0
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.get_device() != dev or t.numel() != n \
            or not t.is_contiguous():
        _cuda(t, name, dtype)
        raise ValueError(f"{name} must hold {n} values on cuda:{dev}, got {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _call(dev: int, stream, what: str, fn, *args):
    """fn(*args, stream) with device `dev` current; on its current stream when none is given."""
    if dev != _current_device():
        with torch.cuda.device(dev):
            return _call(dev, stream, what, fn, *args)
    if stream is not None:
        s = stream.cuda_stream
    else:
        s = _raw_stream(dev) if _raw_stream else torch.cuda.current_stream(dev).cuda_stream
    status = fn(*args, s)
    if status:
        raise W4Error(status, what)


def fp4_scale_bytes(fmt: int, rows: int, K: int) -> int:
    """Bytes of an operand's scale tiles (as fp4_scale_bytes in include/w4a16.h)."""
    if fmt not in (FMT_MXFP4, FMT_NVFP4) or rows < 1 or K < 32 or K % 32 or max(rows, K) > _MAX_EXTENT:
        return 0
    return (rows + 127) // 128 * ((K + 127) // 128 if fmt == FMT_MXFP4 else (K + 63) // 64) * 512


class Fp4Tensor:
    """A block-scaled 4-bit operand of rows x K values (w4_fp4 in include/w4a16.h):

        codes         uint8 [rows][K/2]
        scales        uint8 [fp4_scale_bytes(fmt, rows, K)], tiles of 128 rows x 4 scales
        global_scale  float32 [1] (NVFP4), None (MXFP4)

    Holds its tensors; they do not change after construction."""
    __slots__ = ("fmt", "rows", "K", "global_scale", "_codes", "_scales", "_buf", "_scales_at", "_codes_ptr",
                 "_scales_ptr", "_gptr", "_c", "_dev", "device", "__weakref__")

    def __init__(self, fmt: int, rows: int, K: int, codes: torch.Tensor, scales: torch.Tensor,
                 global_scale: Optional[torch.Tensor] = None):
        fmt = _fp4_fmt(fmt)
        _cuda(codes, "codes", torch.uint8)
        dev = codes.get_device()
        n = fp4_scale_bytes(fmt, rows, K)
        if not n:
            raise W4Error(1, f"4-bit operand of {rows} x {K} (K % 32 == 0, one row at least)")
        if codes.numel() != rows * (K // 2):
            raise ValueError("codes must hold rows * K / 2 bytes")
        if (global_scale is None) != (fmt == FMT_MXFP4):
            raise ValueError("global_scale goes with NVFP4")
        self._scales_ptr = _vector(scales, "scales", torch.uint8, dev, n)
        self._gptr = _vector(global_scale, "global_scale", torch.float32, dev, 1)
        self.fmt, self.rows, self.K, self.global_scale = fmt, rows, K, global_scale
        self._codes, self._scales, self._buf, self._dev, self.device = codes, scales, None, dev, codes.device
        self._codes_ptr = codes.data_ptr()
        self._c = _pack_fp4(fmt, rows, K, self._codes_ptr, self._scales_ptr, self._gptr)

    @classmethod
    def _empty(cls, fmt: int, rows: int, K: int, device: torch.device, dev: int, global_scale, gptr: int, stream):
        """A new operand whose codes and scales are two parts of one allocation."""
        n = fp4_scale_bytes(fmt, rows, K)
        if not n:
            raise W4Error(1, f"4-bit operand of {rows} x {K} (K % 32 == 0, one row at least)")
        at = (rows * (K // 2) + 255) & ~255
        self = cls.__new__(cls)
        self._buf = _new(1, at + n, torch.uint8, device, stream)
        p = self._buf.data_ptr()
        self.fmt, self.rows, self.K, self.global_scale = fmt, rows, K, global_scale
        self._codes = self._scales = None
        self._scales_at, self._codes_ptr, self._scales_ptr, self._gptr, self._dev = at, p, p + at, gptr, dev
        self.device = device
        self._c = _pack_fp4(fmt, rows, K, p, p + at, gptr)
        return self

    @property
    def codes(self) -> torch.Tensor:
        if self._codes is None:
            self._codes = self._buf[0, :self.rows * (self.K // 2)].view(self.rows, self.K // 2)
        return self._codes

    @property
    def scales(self) -> torch.Tensor:
        if self._scales is None:
            self._scales = self._buf[0, self._scales_at:]
        return self._scales

    @property
    def nbytes(self) -> int:
        return self.rows * (self.K // 2) + fp4_scale_bytes(self.fmt, self.rows, self.K)

    def __repr__(self) -> str:
        name = "mxfp4" if self.fmt == FMT_MXFP4 else "nvfp4"
        return f"Fp4Tensor({name}, rows={self.rows}, K={self.K}, device={self.device})"


def _result(out: Optional[Fp4Tensor], fmt: int, rows: int, K: int, device, dev: int, global_scale,
            stream) -> Fp4Tensor:
    """The operand a quantiser writes: `out`, checked, or a new one."""
    g = _vector(global_scale, "global_scale", torch.float32, dev, 1) if fmt == FMT_NVFP4 else 0
    if out is None:
        if fmt == FMT_NVFP4 and not g:
            raise ValueError("nvfp4 needs a global_scale")
        return Fp4Tensor._empty(fmt, rows, K, device, dev, global_scale if g else None, g, stream)
    if not isinstance(out, Fp4Tensor) or (out.fmt, out.rows, out.K, out._dev) != (fmt, rows, K, dev):
        raise ValueError("out must be an Fp4Tensor of the result's format, shape and device")
    if g and g != out._gptr:
        raise ValueError("out.global_scale must be the given global_scale")
    return out


def fp4_quantize(x: torch.Tensor, fmt="mxfp4", *, global_scale: Optional[torch.Tensor] = None,
                 scale_rule: int = MX_SCALE_FLOOR, out: Optional[Fp4Tensor] = None,
                 d_status: Optional[torch.Tensor] = None, stream=None) -> Fp4Tensor:
    """Quantise x[rows][K] (bf16, f16 or f32, K % 32 == 0) to "mxfp4" or, under a given
    global_scale (float32 [1]), "nvfp4" (see fp4_quantize in include/w4a16.h)."""
    fmt = _fp4_fmt(fmt)
    ptr, ld, rows, K = _rows(x, "x")
    dev = x.get_device()
    out = _result(out, fmt, rows, K, x.device, dev, global_scale, stream)
    _call(dev, stream, "fp4_quantize", lib().fp4_quantize, ptr, _type(x, "x"), ld, rows, K, fmt, scale_rule, out._gptr,
          out._codes_ptr, out._scales_ptr, _vector(d_status, "d_status", torch.int32, dev, 1))
    return out


def fp4_dequantize(a: Fp4Tensor, dtype: torch.dtype = torch.bfloat16, *, out: Optional[torch.Tensor] = None,
                   stream=None) -> torch.Tensor:
    """The values [rows][K] an operand stands for (see fp4_dequantize in include/w4a16.h)."""
    if not isinstance(a, Fp4Tensor):
        raise ValueError("a must be an Fp4Tensor")
    if out is None:
        out = _new(a.rows, a.K, dtype, a.device, stream)
    ptr, ld, _, _ = _rows(out, "out", a._dev, a.rows, a.K)
    _call(a._dev, stream, "fp4_dequantize", lib().fp4_dequantize, a._c, ptr, _type(out, "out"), ld)
    return out


def fp4_from_rows(fmt, codes: torch.Tensor, row_scales: torch.Tensor, global_scale: Optional[torch.Tensor] = None, *,
                  stream=None) -> Fp4Tensor:
    """An operand from codes [rows][K/2] (used as they are) and row-major scales
    [rows][K/32] (MXFP4) or [rows][K/16] (NVFP4), which are laid out once."""
    fmt = _fp4_fmt(fmt)
    _cuda(codes, "codes", torch.uint8)
    if codes.dim() != 2:
        raise ValueError("codes must have shape [rows][K/2]")
    rows, K, dev = codes.shape[0], 2 * codes.shape[1], codes.get_device()
    src = _vector(row_scales, "row_scales", torch.uint8, dev, rows * (K // (32 if fmt == FMT_MXFP4 else 16)))
    scales = _new(1, fp4_scale_bytes(fmt, rows, K), torch.uint8, codes.device, stream)[0]
    out = Fp4Tensor(fmt, rows, K, codes, scales, global_scale)
    _call(dev, stream, "fp4_tile_scales", lib().fp4_tile_scales, fmt, rows, K, src, out._scales_ptr)
    return out


def fp4_from_packed(w: PackedWeights, *, stream=None) -> Fp4Tensor:
    """NVFP4 weights from pack_nvfp4 as an operand of w4a4_gemm: codes and global
    scale shared, scales laid out once."""
    if w.fmt != FMT_NVFP4:
        raise ValueError("only NVFP4 weights can be multiplied by 4-bit activations")
    return fp4_from_rows(FMT_NVFP4, w.codes, w.scales, w.global_scale, stream=stream)


def w4a4_gemm(w: Fp4Tensor, x: Fp4Tensor, *, out_dtype: torch.dtype = torch.bfloat16,
              out: Optional[torch.Tensor] = None, flags: int = 0, stream=None) -> torch.Tensor:
    """y[M][N] = x_hat[M][K] . w_hat[N][K], both operands in 4 bits and of the same
    format; any M (see w4a4_gemm in include/w4a16.h)."""
    if not isinstance(w, Fp4Tensor) or not isinstance(x, Fp4Tensor):
        raise ValueError("w and x must be Fp4Tensor (fp4_quantize, fp4_from_packed, block_norm)")
    dev = x._dev
    if w._dev != dev:
        raise ValueError(f"w must be on cuda:{dev}, got cuda:{w._dev}")
    if out is None:
        out = _new(x.rows, w.rows, out_dtype, x.device, stream)
    ptr, ld, _, _ = _rows(out, "out", dev, x.rows, w.rows)
    _call(dev, stream, "w4a4_gemm", lib().w4a4_gemm, w._c, x._c, ptr, _type(out, "out"), ld, flags)
    return out


def w4a4_workspace_bytes(w: Fp4Tensor, M: int) -> int:
    """Bytes of workspace w4a4_linear needs (as w4a4_workspace_bytes in include/w4a16.h)."""
    return ((M * (w.K // 2) + 255) & ~255) + fp4_scale_bytes(w.fmt, M, w.K) if M > _FUSED_TOKENS else 0


def w4a4_linear(w: Fp4Tensor, x: torch.Tensor, *, global_scale: Optional[torch.Tensor] = None,
                scale_rule: int = MX_SCALE_FLOOR, out_dtype: torch.dtype = torch.bfloat16,
                out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                d_status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """y[M][N] = quantised x[M][K] . w_hat: fp4_quantize to w's format (under
    global_scale for NVFP4), then w4a4_gemm, in one call."""
    if not isinstance(w, Fp4Tensor):
        raise ValueError("w must be an Fp4Tensor (fp4_quantize, fp4_from_packed)")
    dev = w._dev
    ptr, ld, M, K = _rows(x, "x", dev)
    if K != w.K:
        raise ValueError(f"x has {K} columns, w {w.K}")
    g = _vector(global_scale, "global_scale", torch.float32, dev, 1) if w.fmt == FMT_NVFP4 else 0
    device = x.device
    if out is None:
        out = _new(M, w.rows, out_dtype, device, stream)
    yptr, yld, _, _ = _rows(out, "out", dev, M, w.rows)
    wptr = need = 0
    if workspace is not None:
        _cuda(workspace, "workspace", torch.uint8)
        wptr, need = workspace.data_ptr(), workspace.numel()
        if workspace.get_device() != dev:
            raise ValueError(f"workspace must be on cuda:{dev}, got {workspace.device}")
    elif M > _FUSED_TOKENS:
        need = w4a4_workspace_bytes(w, M)
        workspace = _new(1, need, torch.uint8, device, stream)
        wptr = workspace.data_ptr()
    _call(dev, stream, "w4a4_linear", lib().w4a4_linear, w._c, ptr, _type(x, "x"), ld, M, scale_rule, g, yptr,
          _type(out, "out"), yld, wptr, need, _vector(d_status, "d_status", torch.int32, dev, 1))
    return out


def block_norm(y: torch.Tensor, h: Optional[torch.Tensor] = None, *, post_weight: Optional[torch.Tensor] = None,
               pre_weight: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None, gate_act: str = "none",
               gate_rows: Optional[int] = None, residual_scale: float = 1.0, block_scale: float = 1.0,
               eps: float = 1e-6, weight_offset: float = 0.0, quantize=None,
               global_scale: Optional[torch.Tensor] = None, scale_rule: int = MX_SCALE_FLOOR, want_h: bool = True,
               out_h: Optional[torch.Tensor] = None, out=None, d_status: Optional[torch.Tensor] = None, stream=None):
    """(h', z) between two blocks, for rows y[M][D], h[M][D] of one type (w4_block_norm
    in include/w4a16.h):

        b  = rmsnorm(y) * (post_weight + weight_offset)      (y itself without post_weight)
        h' = residual_scale * h + block_scale * act(gate) * b
        z  = rmsnorm(h') * (pre_weight + weight_offset)

    gate: [D], or [G][D] where each row serves gate_rows consecutive rows of y (M / G
    if not given); gate_act "none", "sigmoid" or "tanh".  quantize "mxfp4" or "nvfp4"
    (under global_scale) gives z as an Fp4Tensor.  out_h may be h or y; want_h=False
    leaves h' out (None)."""
    yp, ldy, M, D = _rows(y, "y")
    dt, t, dev, device = y.dtype, _type(y, "y"), y.get_device(), y.device

    def rows_of(v, name):
        if v.dtype != dt:
            raise ValueError(f"{name} must be {dt}, got {v.dtype}")
        return _rows(v, name, dev, M, D)

    hp = gp = ohp = zp = ldh = ldg = ldoh = ldz = 0
    if h is not None:
        hp, ldh, _, _ = rows_of(h, "h")
    act = _GATES.get(gate_act)
    if act is None:
        raise ValueError("gate_act must be 'none', 'sigmoid' or 'tanh'")
    if gate is None:
        gate_rows = 1
    else:
        if gate.dtype != dt:
            raise ValueError(f"gate must be {dt}, got {gate.dtype}")
        gp, ldg, G, gw = _rows(gate if gate.dim() == 2 else gate.unsqueeze(0), "gate", dev)
        if gw != D:
            raise ValueError(f"gate must have {D} columns, got {gw}")
        if gate_rows is None:
            if G < 1 or M % G:
                raise ValueError(f"{G} gate rows do not divide {M} rows: give gate_rows")
            gate_rows = M // G
        if gate_rows < 1 or G * gate_rows < M:
            raise ValueError(f"{G} gate rows of {gate_rows} rows each do not cover {M} rows")
        gate_rows = min(gate_rows, M)
    if out_h is not None:
        ohp, ldoh, _, _ = rows_of(out_h, "out_h")
    elif want_h:
        out_h = _new(M, D, dt, device, stream)
        ohp, ldoh = out_h.data_ptr(), D
    fmt = qg = qc = qs = qd = 0
    if quantize is None:
        if out is None:
            out = _new(M, D, dt, device, stream)
            zp, ldz = out.data_ptr(), D
        else:
            zp, ldz, _, _ = rows_of(out, "out")
    else:
        fmt = _fp4_fmt(quantize)
        out = _result(out, fmt, M, D, device, dev, global_scale, stream)
        qg, qc, qs = out._gptr, out._codes_ptr, out._scales_ptr
        qd = _vector(d_status, "d_status", torch.int32, dev, 1)
    n = _pack_norm(t, M, D, yp, hp, _vector(post_weight, "post_weight", dt, dev, D),
                   _vector(pre_weight, "pre_weight", dt, dev, D), gp, ldy, ldh, ldg, gate_rows, act, residual_scale,
                   block_scale, eps, weight_offset, ohp, ldoh, zp, ldz, fmt, scale_rule, qg, qc, qs, qd)
    _call(dev, stream, "w4_block_norm", lib().w4_block_norm, n)
    return out_h, out


def w4_encode_scalars(v: torch.Tensor, stream=None):
    """Elementwise float32 -> (E4M3 byte, E2M1 nibble) with the packers' rounding."""
    _cuda(v, "v", torch.float32)
    e4 = torch.empty(v.shape, dtype=torch.uint8, device=v.device)
    e2 = torch.empty(v.shape, dtype=torch.uint8, device=v.device)
    _check(lib().w4_encode_scalars(_ptr(v), v.numel(), _ptr(e4), _ptr(e2), _stream(stream)),
           "w4_encode_scalars")
    return e4, e2


def set_wait_limit(ns: int = 0):
    """Limit (ns) of the device-side waits that gate progress, on the current
    device; 0 restores the default (2 s).  For exercising failure detection."""
    _check(lib().w4_set_wait_limit(ns), "w4_set_wait_limit")


def w4_device_error(clear: bool = True) -> int:
    """Sticky device error word of the current device (0 = none)."""
    out = ctypes.c_int(0)
    _check(lib().w4_device_error(ctypes.byref(out), 1 if clear else 0), "w4_device_error")
    return out.value
