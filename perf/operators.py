"""The W4A4 operators: what each computes, in elementary torch operations, and the
cases they are measured on.

  quantise     activations -> block-scaled 4-bit values (MXFP4: E2M1 with one power
               of two per 32 values; NVFP4: E2M1 with one E4M3 scale per 16 values
               under a calibrated global scale), returned as the values they stand for
  linear       y = q(x) . w_hat with both operands in 4 bits: x is quantised, then
               multiplied by weights that are already packed
  norm         h' = rs * h + bs * act(gate) * rmsnorm(y) * w_post,
               z = rmsnorm(h') * w_pre: what stands between two blocks of a decoder
  norm_linear  the same with z quantised to 4 bits and multiplied by the next
               block's packed weights

`run` computes the plain form unless `own` is true; then it calls this library.
"""
import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
EPS = 1e-6


# ------------------------------------------------------------------ cases ----

def listed():
    return [
        # one token's hidden state on its way into the q, k and v projections
        dict(name="quantise-mx-1", op="quantise", fmt="mxfp4", dtype="bf16", M=1, K=2560),
        # a prompt's MLP activations before the down projection
        dict(name="quantise-mx-2048", op="quantise", fmt="mxfp4", dtype="bf16", M=2048, K=9728),
        # an odd batch, binary32 activations, a width that is no whole number of tiles
        dict(name="quantise-nv-333", op="quantise", fmt="nvfp4", dtype="f32", M=333, K=2592),
        # decoding one token: the up projection
        dict(name="linear-mx-1", op="linear", fmt="mxfp4", dtype="bf16", out="bf16", M=1, K=2560, N=9728),
        # verifying nine drafted tokens: the down projection
        dict(name="linear-nv-9", op="linear", fmt="nvfp4", dtype="bf16", out="bf16", M=9, K=9728, N=2560),
        # a prompt of 2048 tokens: the up projection
        dict(name="linear-mx-2048", op="linear", fmt="mxfp4", dtype="bf16", out="bf16", M=2048, K=2560, N=9728),
        # a large prefill batch: the down projection
        dict(name="linear-nv-8192", op="linear", fmt="nvfp4", dtype="bf16", out="bf16", M=8192, K=9728, N=2560),
        # ragged in every dimension, binary32 results
        dict(name="linear-mx-777", op="linear", fmt="mxfp4", dtype="f16", out="f32", M=777, K=2592, N=1000),
        # one token between attention and MLP: post-norm, gate, residual, pre-norm
        dict(name="norm-1", op="norm", dtype="bf16", M=1, D=2560, post=True, gate="sigmoid", gate_rows=1,
             residual_scale=1.0, block_scale=1.0),
        # the same for a large prefill batch, one gate for all tokens
        dict(name="norm-8192", op="norm", dtype="bf16", M=8192, D=2560, post=True, gate="none", gate_rows=8192,
             residual_scale=1.0, block_scale=0.5),
        # sixteen tokens through the norms into the q projection
        dict(name="norm-linear-mx-16", op="norm_linear", fmt="mxfp4", dtype="bf16", out="bf16", M=16, D=2560, N=4096,
             post=True, gate="sigmoid", gate_rows=1, residual_scale=1.0, block_scale=1.0),
        # a prompt through the norms into the up projection
        dict(name="norm-linear-nv-2048", op="norm_linear", fmt="nvfp4", dtype="bf16", out="bf16", M=2048, D=2560,
             N=9728, post=False, gate="tanh", gate_rows=2048, residual_scale=1.0, block_scale=1.0),
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["quantise", "linear", "linear", "norm", "norm_linear"])
    M = _log_uniform(rng, 1, 8192)
    K = 32 * _log_uniform(rng, 2, 304)
    case = dict(op=op, dtype=rng.choice(["bf16", "bf16", "f16", "f32"]), M=M)
    if op != "norm":
        case["fmt"] = rng.choice(["mxfp4", "nvfp4"])
    if op in ("quantise", "linear"):
        case["K"] = K
    else:
        # the norms alone take any width; a 4-bit result needs whole blocks
        case["D"] = rng.choice([K, _log_uniform(rng, 9, 9728)]) if op == "norm" else K
        gate = rng.choice(["none", "sigmoid", "tanh", "off"])
        rows = rng.choice([1, M] if M % 2 else [1, M, M // 2])
        case.update(post=rng.random() < 0.5, gate=gate, gate_rows=rows, residual_scale=rng.choice([1.0, 1.25]),
                    block_scale=rng.choice([1.0, 0.5]))
    if op in ("linear", "norm_linear"):
        case["N"] = _log_uniform(rng, 8, 9728)
        # 4-bit rounding of a norm's result is not the same to the last bit on both
        # sides, so its products come in 16 bits
        case["out"] = rng.choice(["bf16", "bf16", "f16" if op == "norm_linear" else "f32"])
        while 2 * case["M"] * K * case["N"] > 4.0e11:
            case["M"] = max(1, case["M"] // 2)
            if "gate_rows" in case:
                case["gate_rows"] = case["M"]
    return case


# ----------------------------------------------------------------- inputs ----

def _activations(gen, M, K, dtype):
    x = torch.randn(M, K, generator=gen, device="cuda")
    cols = torch.randint(0, K, (max(1, K // 160),), generator=gen, device="cuda")
    x[:, cols] *= 30.0          # outlier channels
    return x.to(_TYPES[dtype])


def _pack_rows(W, fmt):
    """Codes [N][K/2] (even element in the low nibble), scales [N][K/32 | K/16] and
    the global scale of a binary32 matrix, by torch."""
    N, K = W.shape
    if fmt == "mxfp4":
        g = None
        byte, inv = _mx_scales(W)
        v = W.view(N, K // 32, 32) * inv[..., None]
        scales = byte.to(torch.uint8)
    else:
        g = (W.abs().amax() / 2688.0).reshape(1)
        s = _e4m3((W.view(N, K // 16, 16).abs().amax(-1) / 6.0) / g)
        d = s * g
        v = torch.where(d[..., None] > 0, W.view(N, K // 16, 16) / d[..., None], torch.zeros((), device=W.device))
        scales = s.to(torch.float8_e4m3fn).view(torch.uint8)
    r = _round_e2m1(v).reshape(N, K)
    mag = torch.bucketize(r.abs(), torch.tensor(_E2M1, device=W.device))
    code = (mag + 8 * torch.signbit(r)).to(torch.uint8).view(N, K // 2, 2)
    return code[..., 0] | (code[..., 1] << 4), scales.contiguous(), g


def _weights(gen, N, K, fmt):
    W = torch.randn(N, K, generator=gen, device="cuda") * 0.02
    hit = torch.rand(N, K, generator=gen, device="cuda") < 1e-4
    W = torch.where(hit, W * 20.0, W)
    return _pack_rows(W.to(torch.bfloat16).float(), fmt)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, M = case["op"], case["M"]
    K = case.get("K", case.get("D"))
    t = _TYPES[case["dtype"]]
    st = dict(case=case, op=op)
    if op in ("quantise", "linear"):
        st["x"] = _activations(gen, M, K, case["dtype"])
        # calibrated: a running mean of other batches' largest values
        amax = st["x"].float().abs().amax() * (0.9 + 0.2 * torch.rand((), generator=gen, device="cuda"))
    else:
        st["y"] = (torch.randn(M, K, generator=gen, device="cuda") * 0.7).to(t)
        st["h"] = (torch.randn(M, K, generator=gen, device="cuda") * 2.0).to(t)
        st["w_post"] = (1.0 + 0.1 * torch.randn(K, generator=gen, device="cuda")).to(t) if case["post"] else None
        st["w_pre"] = (1.0 + 0.1 * torch.randn(K, generator=gen, device="cuda")).to(t)
        st["gate"] = None
        if case["gate"] != "off":
            G = -(-M // case["gate_rows"])
            st["gate"] = torch.randn(G, K, generator=gen, device="cuda").to(t)
        # calibrated: a normalised row's usual largest value
        amax = 6.0 * (0.9 + 0.2 * torch.rand((), generator=gen, device="cuda"))
    st["g"] = (amax / 2688.0).reshape(1) if case.get("fmt") == "nvfp4" else None
    if op in ("linear", "norm_linear"):
        codes, scales, gw = _weights(gen, case["N"], K, case["fmt"])
        st.update(w_codes=codes, w_scales=scales, w_g=gw)
        if own:   # the handle a program keeps beside its packed weights
            import w4a16_matmul_pack_b200 as W4
            st["weights"] = W4.fp4_from_rows(case["fmt"], codes, scales, gw)
    return st


# ------------------------------------------------------------- plain forms ----

def _mx_scales(x):
    """Scale bytes (E8M0) and reciprocals of the scales of each 32 values."""
    M, K = x.shape
    amax = x.view(M, K // 32, 32).abs().amax(-1)
    _, e = torch.frexp(amax)                       # amax = m 2^e, 0.5 <= m < 1
    byte = (e.to(torch.int32) - 3 + 127).clamp(0, 254)
    byte = torch.where(amax > 0, byte, torch.zeros_like(byte))
    return byte, ((254 - byte) << 23).view(torch.float32)


def _pow2(byte):
    """2^(byte - 127) in binary32 (byte 0: the subnormal 2^-127)."""
    return torch.where(byte > 0, byte << 23, torch.full_like(byte, 1 << 22)).view(torch.float32)


def _e4m3(v):
    """Nearest E4M3 value, ties to even, saturating."""
    return v.clamp(max=448.0).to(torch.float8_e4m3fn).float()


def _round_e2m1(v):
    """Nearest E2M1 value, ties to the even code, saturating at 6."""
    a = v.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return torch.copysign((torch.round(a / step) * step).clamp(max=6.0), v)


def _quantised(x, fmt, g):
    """The binary32 values that the 4-bit form of binary32 x stands for."""
    M, K = x.shape
    if fmt == "mxfp4":
        byte, inv = _mx_scales(x)
        r = _round_e2m1(x.view(M, K // 32, 32) * inv[..., None])
        return (r * _pow2(byte)[..., None]).reshape(M, K)
    b = x.view(M, K // 16, 16)
    s = _e4m3((b.abs().amax(-1) / 6.0) / g)
    d = s * g
    r = _round_e2m1(b * torch.where(d > 0, 1.0 / d, torch.zeros_like(d))[..., None])
    return ((r * s[..., None]) * g).reshape(M, K)


def _decoded(codes, scales, fmt, g):
    N, half = codes.shape
    t = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), device=codes.device)
    v = torch.stack((t[(codes & 15).int()], t[(codes >> 4).int()]), -1).reshape(N, 2 * half)
    if fmt == "mxfp4":
        return (v.view(N, half // 16, 32) * _pow2(scales.int())[..., None]).reshape(N, 2 * half)
    s = scales.view(torch.float8_e4m3fn).float()
    return ((v.view(N, half // 8, 16) * s[..., None]) * g).reshape(N, 2 * half)


def _rms(v):
    return v * torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS)


def _norm_values(st):
    """(h', z) in binary32."""
    c = st["case"]
    b = st["y"].float()
    if st["w_post"] is not None:
        b = _rms(b) * st["w_post"].float()
    if st["gate"] is not None:
        g = st["gate"].float()
        g = torch.sigmoid(g) if c["gate"] == "sigmoid" else torch.tanh(g) if c["gate"] == "tanh" else g
        b = b * g.repeat_interleave(c["gate_rows"], 0)[:c["M"]]
    h = c["residual_scale"] * st["h"].float() + c["block_scale"] * b
    return h, _rms(h) * st["w_pre"].float()


def run(st):
    c, op = st["case"], st["op"]
    if own:
        import w4a16_matmul_pack_b200 as W4
        if op == "quantise":
            return W4.fp4_dequantize(W4.fp4_quantize(st["x"], c["fmt"], global_scale=st["g"]))
        if op == "linear":
            return W4.w4a4_linear(st["weights"], st["x"], global_scale=st["g"], out_dtype=_TYPES[c["out"]])
        h, z = W4.block_norm(st["y"], st["h"], post_weight=st["w_post"], pre_weight=st["w_pre"], gate=st["gate"],
                             gate_act="none" if c["gate"] == "off" else c["gate"], gate_rows=c["gate_rows"],
                             residual_scale=c["residual_scale"], block_scale=c["block_scale"], eps=EPS,
                             quantize=c.get("fmt"), global_scale=st["g"])
        if op == "norm":
            return h, z
        return h, W4.w4a4_gemm(st["weights"], z, out_dtype=_TYPES[c["out"]])
    if op == "quantise":
        return _quantised(st["x"].float(), c["fmt"], st["g"]).to(torch.bfloat16)
    if op == "linear":
        w = _decoded(st["w_codes"], st["w_scales"], c["fmt"], st["w_g"])
        return (_quantised(st["x"].float(), c["fmt"], st["g"]) @ w.t()).to(_TYPES[c["out"]])
    h, z = _norm_values(st)
    t = _TYPES[c["dtype"]]
    if op == "norm":
        return h.to(t), z.to(t)
    w = _decoded(st["w_codes"], st["w_scales"], c["fmt"], st["w_g"])
    return h.to(t), (_quantised(z, c["fmt"], st["g"]) @ w.t()).to(_TYPES[c["out"]])


# ------------------------------------------------------------------- work ----

def work(case):
    M, op = case["M"], case["op"]
    K = case.get("K", case.get("D"))
    size = 4 if case["dtype"] == "f32" else 2
    scale = {"mxfp4": 1 / 32, "nvfp4": 1 / 16}.get(case.get("fmt"), 0)
    if op == "quantise":
        return {"bytes": M * K * (size + 2), "flops": 4 * M * K}
    b = f = 0
    if op in ("linear", "norm_linear"):
        N = case["N"]
        b += int(N * K * (0.5 + scale)) + M * N * (4 if case["out"] == "f32" else 2)
        f += 2 * M * N * K
    if op == "linear":
        return {"bytes": b + M * K * size, "flops": f}
    gate = 0 if case["gate"] == "off" else -(-M // case["gate_rows"]) * K
    b += (3 * M * K + gate + K * (2 if case["post"] else 1) + (M * K if op == "norm" else 0)) * size
    return {"bytes": b, "flops": f + 12 * M * K}


# --------------------------------------------- the definitions in 64 bits ----

def _nearest_e2m1(v):
    """Nearest of the eight magnitudes by their midpoints, a tie to the even index."""
    levels = torch.tensor(_E2M1, dtype=torch.float64, device=v.device)
    mid = (levels[1:] + levels[:-1]) / 2
    a = v.abs()
    lo, hi = torch.bucketize(a, mid), torch.bucketize(a, mid, right=True)
    idx = torch.where(lo % 2 == 0, lo, hi)         # lo == hi but at a midpoint
    return levels[idx] * torch.sign(v)


def _exact_blocks(x, fmt, g):
    if fmt == "mxfp4":
        b = x.unflatten(1, (-1, 32))
        top = b.abs().amax(-1, keepdim=True)
        e = torch.floor(torch.log2(torch.where(top > 0, top, torch.ones_like(top))))
        e = torch.where(torch.exp2(e) > top, e - 1, torch.where(torch.exp2(e + 1) <= top, e + 1, e))
        s = torch.exp2((e - 2).clamp(min=-127.0))
    else:
        b = x.unflatten(1, (-1, 16))
        t = (b.abs().amax(-1, keepdim=True) / (6.0 * g)).clamp(max=448.0)
        step = torch.exp2(torch.floor(torch.log2(t.clamp(min=2.0 ** -6))) - 3)
        s = torch.round(t / step) * step * g
    v = _nearest_e2m1(torch.where(s > 0, b / torch.where(s > 0, s, torch.ones_like(s)), torch.zeros_like(b)))
    return (v * s).flatten(1)


def _exact_weights(st, fmt):
    codes = st["w_codes"].long()
    nib = torch.stack((codes % 16, codes // 16), 2).flatten(1)
    e, m = (nib % 8) // 2, nib % 2                 # exponent (bias 1) and mantissa of the magnitude
    mag = torch.where(e == 0, 0.5 * m, (1.0 + 0.5 * m) * torch.exp2(e.double() - 1))
    v = torch.where(nib >= 8, -mag, mag)
    if fmt == "mxfp4":
        return (v.unflatten(1, (-1, 32)) * torch.exp2(st["w_scales"].double() - 127)[..., None]).flatten(1)
    u = st["w_scales"].long()
    e, m = u // 8, u % 8                           # E4M3, no sign
    s = torch.where(e == 0, m * 2.0 ** -9, (1.0 + m / 8.0) * torch.exp2(e.double() - 7))
    return (v.unflatten(1, (-1, 16)) * s[..., None]).flatten(1) * st["w_g"].double()


def exact(case, seed):
    st = prepare(case, seed)
    op, fmt = case["op"], case.get("fmt")
    g = None if st["g"] is None else st["g"].double()
    if op in ("quantise", "linear"):
        q = _exact_blocks(st["x"].double(), fmt, g)
        return q if op == "quantise" else q @ _exact_weights(st, fmt).t()
    b = st["y"].double()
    if case["post"]:
        b = b / torch.sqrt(b.pow(2).mean(1, keepdim=True) + EPS) * st["w_post"].double()
    if st["gate"] is not None:
        a = st["gate"].double()
        if case["gate"] == "sigmoid":
            a = 1 / (1 + torch.exp(-a))
        elif case["gate"] == "tanh":
            a = torch.tanh(a)
        b = b * a[torch.arange(case["M"], device="cuda") // case["gate_rows"]]
    h = case["residual_scale"] * st["h"].double() + case["block_scale"] * b
    z = h / torch.sqrt(h.pow(2).mean(1, keepdim=True) + EPS) * st["w_pre"].double()
    if op == "norm":
        return h, z
    return h, _exact_blocks(z, fmt, g) @ _exact_weights(st, fmt).t()
