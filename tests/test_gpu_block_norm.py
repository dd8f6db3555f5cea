"""w4_block_norm on the GPU against the 64-bit formula.

Tolerances: h' is at most five binary32 operations behind the statistic, whose sum
of D squares in lanes and warps is at most D / threads + 15 <= 64 additions deep;
the relative error of a norm's factor is at most half of (64 + 4) * 2^-24, and act()
is within 2^-21.  So b is within (34 + 5) 2^-24 + 2^-21 < 2^-18 of itself, h' within
2^-18 (|rs h| + |bs b|), and z, another such factor on top, within 2^-17 of
(|rs h| + |bs b|) r |w|; each output is rounded once more to its type."""
import numpy as np
import pytest
import torch

import fp4_ref as R
import w4a16_matmul_pack_b200 as W4

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.fixture(autouse=True)
def clean_error_word():
    W4.w4_device_error(clear=True)
    yield
    W4.w4_device_error(clear=True)


def make(M, D, dtype, seed, gate_rows=None, post=True, pre=True, residual=True):
    g = torch.Generator().manual_seed(seed)

    def t(*shape, scale=1.0, mean=0.0):
        return (torch.randn(*shape, generator=g) * scale + mean).to(dtype).cuda()
    G = None if gate_rows is None else -(-M // gate_rows)
    return dict(y=t(M, D, scale=0.7), h=t(M, D, scale=2.0) if residual else None,
                post=t(D, scale=0.1, mean=1.0) if post else None, pre=t(D, scale=0.1, mean=1.0) if pre else None,
                gate=None if G is None else t(G, D))


def reference(s, act="none", gate_rows=1, rs=1.0, bs=1.0, eps=1e-6, off=0.0):
    d = {k: None if v is None else R.f64(v) for k, v in s.items()}
    hn, z = R.block_norm(d["y"], d["h"], d["post"], d["pre"], d["gate"], act, gate_rows, np.float64(np.float32(rs)),
                         np.float64(np.float32(bs)), np.float64(np.float32(eps)), off)
    b = hn if d["h"] is None else hn - rs * d["h"]
    size = np.abs(b) + (0 if d["h"] is None else np.abs(rs * d["h"]))
    r = 1 / np.sqrt((hn * hn).mean(1, keepdims=True) + eps)
    zsize = size * r * (1 if d["pre"] is None else np.abs(d["pre"] + off))
    return hn, z, size, zsize


def check(s, got_h, got_z, dtype, **kw):
    hn, z, size, zsize = reference(s, **kw)
    if got_h is not None:
        err = np.abs(R.f64(got_h) - hn)
        assert np.all(err <= 2.0 ** -18 * size + R.half_step(hn, dtype) * 1.01), err.max()
    err = np.abs(R.f64(got_z) - z)
    assert np.all(err <= 2.0 ** -17 * zsize + R.half_step(z, dtype) * 1.01), err.max()


def call(s, **kw):
    return W4.block_norm(s["y"], s["h"], post_weight=s["post"], pre_weight=s["pre"], gate=s["gate"], **kw)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,D", [(1, 1), (1, 2560), (2, 7), (3, 8), (5, 40), (4, 257), (17, 1321), (2, 4096), (3, 4104),
                                 (2, 8947), (2, 9728), (1, 16392), (1, 32768), (2, 32761)])
def test_all_parts(dtype, M, D):
    s = make(M, D, dtype, M + D, gate_rows=1)
    h, z = call(s, gate_act="sigmoid", residual_scale=1.25, block_scale=0.5)
    check(s, h, z, dtype, act="sigmoid", rs=1.25, bs=0.5)


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("pre", [False, True])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("act", [None, "none", "sigmoid", "tanh"])
def test_parts_left_out(post, pre, residual, act):
    s = make(5, 136, torch.bfloat16, 3, gate_rows=None if act is None else 5, post=post, pre=pre, residual=residual)
    h, z = call(s, gate_act=act or "none", block_scale=0.75, weight_offset=1.0, eps=1e-5)
    check(s, h, z, torch.bfloat16, act=act, gate_rows=5, bs=0.75, off=1.0, eps=1e-5)


@pytest.mark.parametrize("M,gate_rows", [(6, 1), (6, 2), (6, 3), (6, 6), (7, 3), (7, 100)])
def test_gate_rows(M, gate_rows):
    s = make(M, 64, torch.float32, M, gate_rows=gate_rows)
    h, z = call(s, gate_act="tanh", gate_rows=gate_rows)
    check(s, h, z, torch.float32, act="tanh", gate_rows=gate_rows)
    if M % gate_rows == 0:      # the same without saying so
        h2, z2 = call(s, gate_act="tanh")
        assert torch.equal(h, h2) and torch.equal(z, z2)
    one = dict(s, gate=s["gate"][0])
    h, z = call(one, gate_act="tanh")
    check(dict(s, gate=s["gate"][:1]), h, z, torch.float32, act="tanh", gate_rows=M)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D,off", [(64, 0), (64, 1), (72, 8), (63, 3)])
def test_strides_and_alignment(dtype, D, off):
    """Rows of wider buffers, on and off 16 bytes."""
    M = 6
    s = make(M, D, dtype, D + off, gate_rows=1)
    wide = {k: torch.full((M, D + 24), 9.0, dtype=dtype, device="cuda") for k in ("y", "h", "gate", "out_h", "out")}
    v = {k: t[:, off:off + D] for k, t in wide.items()}
    for k in ("y", "h", "gate"):
        v[k].copy_(s[k])
    W4.block_norm(v["y"], v["h"], post_weight=s["post"], pre_weight=s["pre"], gate=v["gate"], gate_act="sigmoid",
                  out_h=v["out_h"], out=v["out"])
    check(s, v["out_h"], v["out"], dtype, act="sigmoid")
    for k in ("out_h", "out"):
        wide[k][:, off:off + D] = 9.0
        assert (wide[k] == 9).all()       # nothing beside the rows


@pytest.mark.parametrize("D", [256, 131])
def test_in_place(D):
    s = make(9, D, torch.bfloat16, 4, gate_rows=1)
    h0, z0 = call(s)
    y, h = s["y"].clone(), s["h"].clone()
    h1, z1 = W4.block_norm(y, h, post_weight=s["post"], pre_weight=s["pre"], gate=s["gate"], out_h=h, out=y)
    assert h1 is h and z1 is y and torch.equal(h0, h) and torch.equal(z0, y)
    _, z2 = call(s, want_h=False)
    assert torch.equal(z2, z0)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,D,shift", [(1, 32, 0), (3, 96, 0), (130, 2560, 0), (2, 9728, 0), (2, 17408, 0), (3, 64, 1),
                                       (2, 2592, 1)])
def test_four_bit_z(fmt, dtype, M, D, shift):
    """4-bit z stands for z within the quantiser's own error: the code is the nearest
    to z / s for the scale that was written, up to z's tolerance; and the scale is the
    one of amax up to that tolerance.  shift: rows that do not start on 16 bytes."""
    s = make(M, D, dtype, D + M)
    if shift:
        wide = torch.zeros(M, D + 8, dtype=dtype, device="cuda")
        wide[:, 1:D + 1] = s["y"]
        s["y"] = wide[:, 1:D + 1]
    g = torch.tensor([5.3 / 2688], device="cuda") if fmt == "nvfp4" else None
    h, q = call(s, quantize=fmt, global_scale=g)
    h2, z2 = call(s)
    assert torch.equal(h, h2)                 # h' does not depend on z's form
    hn, z, size, zsize = reference(s)
    B = R.BLOCK[fmt]
    scales, pad = R.untile(q.scales.cpu().numpy(), M, D, fmt)
    assert not pad.any()
    tol = (2.0 ** -17 * zsize).reshape(M, D // B, B)
    top = np.abs(z).reshape(M, D // B, B).max(-1)
    ttol = tol.max(-1)
    sv = 2.0 ** (scales.astype(np.float64) - 127) if fmt == "mxfp4" else R.e4m3_value(scales)
    if fmt == "mxfp4":        # 4 s <= amax < 8 s
        assert np.all(top + ttol >= 4 * sv) and np.all(top - ttol < 8 * sv)
    else:                     # s = E4M3(amax / 6 / g): its ends round to s or beyond
        lo, hi = ((top + d) / 6 / g.item() for d in (-ttol, ttol))
        assert np.all(R.e4m3_byte(lo * (1 - 2.0 ** -22)) <= scales) and np.all(R.e4m3_byte(hi * (1 + 2.0 ** -22)) >= scales)
        sv = sv * g.item()
    d = R.f64(W4.fp4_dequantize(q, torch.float32)).reshape(M, D // B, B)
    zb = z.reshape(M, D // B, B)
    level = np.round(2 * np.abs(d / sv[..., None])) / 2     # d is e2m1 * s * g rounded to binary32
    gap = np.where(level < 2, 0.25, np.where(level < 4, 0.5, 1.0)) * sv[..., None]     # half the gap above
    sat = np.abs(zb) > 6 * sv[..., None]
    err = np.where(sat, np.maximum(np.abs(zb) - 8 * sv[..., None], 0) if fmt == "mxfp4" else 0, np.abs(d - zb))
    assert np.all(err <= gap * (1 + 2.0 ** -20) + tol)
    # the same bits as quantising z itself in binary32, wherever z is binary32
    if dtype == torch.float32:
        q2 = W4.fp4_quantize(z2, fmt, global_scale=g)
        assert torch.equal(q.codes, q2.codes)
        assert np.array_equal(scales, R.untile(q2.scales.cpu().numpy(), M, D, fmt)[0])


def test_zero_rows_and_nonfinite():
    s = make(3, 64, torch.float32, 1)
    s["y"][0] = 0
    s["h"][0] = 0
    s["h"][1, 7] = float("nan")
    h, z = call(s)
    assert not h[0].any() and not z[0].any() and torch.isfinite(z[0]).all()
    assert z[1].isnan().all() and h[1].isnan().sum() == 1
    assert torch.isfinite(z[2]).all()
    h, q = call(s, quantize="mxfp4")
    d = W4.fp4_dequantize(q)
    assert not d[0].any() and d[1].isnan().all() and torch.isfinite(d[2]).all()
    assert W4.w4_device_error(clear=True) == 5


def test_deterministic_and_captured():
    s = make(64, 2560, torch.bfloat16, 2, gate_rows=1)
    h0, z0 = call(s, gate_act="sigmoid")
    out_h, out = torch.empty_like(h0), torch.empty_like(z0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(s, gate_act="sigmoid", out_h=out_h, out=out)
    for _ in range(3):
        out_h.zero_(), out.zero_()
        graph.replay()
        assert torch.equal(out_h, h0) and torch.equal(out, z0)


def act_tolerance(g, act):
    """Relative error of act(g).  sigmoid: the argument of 2^x is off by |g| log2(e)
    (2^-24 + 2^-26) (its rounding and the constant's), which ln 2 turns into |g| 1.25 * 2^-24
    of the power; the power and the division cost 2^-22 each, the sum 2^-24.  tanh from 0.3
    on, 1 - q with q = 2 / (1 + 2^x): q is off by as much with 2 |g| for |g|, and q <= 2.44
    tanh there; 2.44 (0.6 * 1.25 * 2^-24 + 2^-21 + 2^-24) < 2^-19 at 0.3 and less further
    out.  Below: the series' next term 2^-24 and five roundings."""
    return np.minimum(np.abs(g), 1e3) * 1.25 * 2.0 ** -24 + 2.0 ** -20 if act == "sigmoid" else np.full_like(g, 2.0 ** -19)


@pytest.mark.parametrize("act", ["sigmoid", "tanh"])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("own_rows", [False, True])
def test_gates_far_from_zero(act, dtype, own_rows):
    """Gates of both signs from 2^-20 to 200, beside tanh's border at 0.3, zeros of both
    signs, and infinities.  sigmoid below 2^-126 is 0."""
    D, M = 96, 4
    border = np.float32(0.3)
    mags = [0.0, 2.0 ** -20, 1e-3, 0.05, 0.29, np.nextafter(border, np.float32(0)), border,
            np.nextafter(border, np.float32(1)), 0.2988, 0.3008, 0.31, 0.5, 1, 2, 4, 8, 9.5, 10, 12, 16, 17, 20, 30, 44, 60,
            80, 86, 87, 87.5, 88, 88.75, 89, 95, 100, 103, 104, 120, 150, 200, np.inf]
    g = np.zeros(D)
    g[:2 * len(mags)] = np.concatenate([mags, np.negative(mags)])
    gate = torch.from_numpy(np.stack([g, g[::-1], np.roll(g, 7), np.roll(g, 40)]) if own_rows else g[None]).to(dtype).cuda()
    s = make(M, D, dtype, 5, post=False)
    s["gate"], rows = gate, 1 if own_rows else M
    h, z = call(s, gate_act=act, gate_rows=rows, block_scale=0.5)
    h1, _ = W4.block_norm(s["y"], gate=gate, gate_act=act, gate_rows=rows, block_scale=0.5)    # the gated term alone
    gv, yv = R.f64(gate)[np.arange(M) // rows], R.f64(s["y"])
    with np.errstate(over="ignore"):
        a = 1 / (1 + np.exp(-gv)) if act == "sigmoid" else np.tanh(gv)
    b = 0.5 * a * yv
    tol = (act_tolerance(gv, act) + 2.0 ** -23) * np.abs(b) + 2.0 ** -126 * np.abs(yv)
    assert np.all(np.abs(R.f64(h1) - b) <= tol + R.half_step(b, dtype) * 1.01)
    hv = R.f64(s["h"])
    hn = hv + b
    htol = tol + 2.0 ** -23 * (np.abs(hv) + np.abs(b))
    assert np.all(np.abs(R.f64(h) - hn) <= htol + R.half_step(hn, dtype) * 1.01)
    ms = (hn * hn).mean(1, keepdims=True) + 1e-6
    r = 1 / np.sqrt(ms)
    # the factor's relative error: that of half the mean square, whose sum is at most 64 additions deep
    rtol = (htol * np.abs(hn)).mean(1, keepdims=True) / ms + 36 * 2.0 ** -24
    zn = hn * r * R.f64(s["pre"])
    ztol = htol * r * np.abs(R.f64(s["pre"])) + (rtol + 2.0 ** -22) * np.abs(zn)
    assert np.all(np.abs(R.f64(z) - zn) <= ztol + R.half_step(zn, dtype) * 1.01)


@pytest.mark.parametrize("act", ["none", "sigmoid", "tanh"])
@pytest.mark.parametrize("own_rows", [False, True])
def test_a_nan_gate_stays_in_its_rows(act, own_rows):
    M, D = 3, 64
    s = make(M, D, torch.float32, 6, gate_rows=1 if own_rows else M)
    s["gate"][-1, 9] = float("nan")
    h, z = call(s, gate_act=act, gate_rows=1 if own_rows else M)
    bad = np.zeros((M, D), bool)
    bad[M - 1 if own_rows else slice(None), 9] = True
    assert np.array_equal(np.isnan(R.f64(h)), bad)
    assert np.array_equal(np.isnan(R.f64(z)), np.broadcast_to(bad.any(1, keepdims=True), (M, D)))
