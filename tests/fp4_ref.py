"""Plain numpy forms of the 4-bit operands, their product and the block norms, in
64 bits (the NVFP4 encoder's few binary32 steps in binary32, as it is defined)."""
import numpy as np
import torch

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
BLOCK = {"mxfp4": 32, "nvfp4": 16}


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().to(torch.float64).numpy()


def f32(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().to(torch.float32).numpy()


def e2m1_codes(v):
    """Nearest E2M1 code (ties to the even code, saturating, sign kept); v in 64 bits."""
    a = np.abs(v)
    mid = (E2M1[1:] + E2M1[:-1]) / 2
    lo, hi = np.searchsorted(mid, a, side="left"), np.searchsorted(mid, a, side="right")
    idx = np.where(lo % 2 == 0, lo, hi)
    return (idx + 8 * np.signbit(v)).astype(np.uint8)


def e2m1_values(codes):
    return np.where(codes >= 8, -1.0, 1.0) * E2M1[codes & 7]


def e4m3_value(b):
    b = b.astype(np.int64)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * 2.0 ** (e - 7.0))
    return np.where(b == 0x7F, np.nan, v)


def e4m3_byte(v):
    """Nearest E4M3 byte of v >= 0 (ties to even, saturating at 448)."""
    table = e4m3_value(np.arange(0x7F))
    mid = (table[1:] + table[:-1]) / 2
    lo, hi = np.searchsorted(mid, v, side="left"), np.searchsorted(mid, v, side="right")
    return np.where(lo % 2 == 0, lo, hi).astype(np.uint8)


def quantize(x32, fmt, g=None, ceil=False):
    """(codes [rows][K] one per value, scale bytes [rows][K / block]) of binary32 rows."""
    rows, K = x32.shape
    B = BLOCK[fmt]
    b = x32.reshape(rows, K // B, B)
    bad = ~np.isfinite(b).all(-1)
    fin = np.where(np.isfinite(b), b, np.float32(0))
    top = np.where(bad, np.float32(0), np.abs(fin).max(-1))
    if fmt == "mxfp4":
        m, e = np.frexp(top.astype(np.float64))          # top = m 2^e, m in [1/2, 1)
        e = e - 1 - 2
        if ceil:
            e = e + (m > 0.75)
        byte = np.where(top > 0, np.clip(e + 127, 0, 254), 0).astype(np.int64)
        q = fin.astype(np.float64) * (2.0 ** (127.0 - byte))[..., None]
        byte = np.where(bad, 0xFF, byte)
    else:
        g = np.float32(g)
        with np.errstate(all="ignore"):
            byte = e4m3_byte(((top / np.float32(6)) / g).astype(np.float64)) if g > 0 else np.zeros(top.shape, np.uint8)
            d = (e4m3_value(byte).astype(np.float32) * g).astype(np.float32)
            r = np.float32(1) / d
        ok = np.isfinite(r)
        byte = np.where(ok, byte, 0)
        q = (fin * np.where(ok, r, np.float32(0))[..., None]).astype(np.float32).astype(np.float64)
        byte = np.where(bad, 0x7F, byte)
    codes = np.where(bad[..., None], 0, e2m1_codes(q))
    return codes.reshape(rows, K).astype(np.uint8), byte.astype(np.uint8)


def values(codes, scales, fmt, g=None):
    """The values in 64 bits."""
    rows, K = codes.shape
    if fmt == "mxfp4":
        s = np.where(scales == 0xFF, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    else:
        s = e4m3_value(scales) * np.float64(np.float32(g))
    return (e2m1_values(codes).reshape(rows, -1, BLOCK[fmt]) * s[..., None]).reshape(rows, K)


def nibbles(packed):
    out = np.empty((packed.shape[0], 2 * packed.shape[1]), np.uint8)
    out[:, 0::2], out[:, 1::2] = packed & 15, packed >> 4
    return out


def pack(codes):
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)


def untile(tiles, rows, K, fmt):
    """(row-major scales, the padding scales) of the tiled layout."""
    per = K // BLOCK[fmt]
    T = -(-per // 4)
    r, j = np.meshgrid(np.arange(rows), np.arange(4 * T), indexing="ij")
    at = ((r // 128) * T + j // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + j % 4
    all_scales = tiles[at]
    return all_scales[:, :per], all_scales[:, per:]


def product(xv, wv):
    """(y, sum |x w|) in 64 bits."""
    return xv @ wv.T, np.abs(xv) @ np.abs(wv).T


def product_bound(a, K):
    """How far a binary32 accumulation may be from y: the tensor cores add 64 products
    to the accumulator per step; allow each step the error of two truncations of the
    running sum (2 * 2^-23 of at most sum |x w|), and two more for the scaling."""
    return (-(-K // 64) + 2) * 2.0 ** -22 * a


def half_step(v, dtype):
    """Half a unit in the last place of |v| in dtype (its subnormal step included)."""
    if dtype == torch.float32:
        eps, tiny = 2.0 ** -24, 2.0 ** -150
    elif dtype == torch.bfloat16:
        eps, tiny = 2.0 ** -8, 2.0 ** -134
    else:
        eps, tiny = 2.0 ** -11, 2.0 ** -25
    return np.abs(v) * eps + tiny


def block_norm(y, h, w_post, w_pre, gate, act, gate_rows, rs, bs, eps, off):
    """(h', z) in 64 bits; arrays or None."""
    b = y
    if w_post is not None:
        b = b / np.sqrt((b * b).mean(1, keepdims=True) + eps) * (w_post + off)
    if gate is not None:
        a = gate
        if act == "sigmoid":
            a = 1 / (1 + np.exp(-a))
        elif act == "tanh":
            a = np.tanh(a)
        b = b * a[np.arange(y.shape[0]) // gate_rows]
    hn = bs * b if h is None else rs * h + bs * b
    z = hn / np.sqrt((hn * hn).mean(1, keepdims=True) + eps)
    return hn, z if w_pre is None else z * (w_pre + off)
