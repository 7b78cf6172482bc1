"""What is measured of the norm in front of a quantised Linear and of the Linear in 4 bits.

Kinds of cases (every matrix is row-major BF16 unless said otherwise):

  norm     h = bf16(x + residual); y = h / sqrt(mean(h^2) + eps) * gamma, written as FP8 codes with a per-tensor scale
           ("fp8": codes, amax, inverse scale), as MXFP8 codes with one E8M0 scale per 32 values ("mxfp8") or as BF16
           ("bf16"), and 1 / sqrt(mean(h^2) + eps) per row for the backward pass
  grad     the backward pass: the gradient of h (with the gradient that reaches the residual stream directly added, where
           there is one) and of gamma
  linear   D = X . W^T with X quantised to 4 bits here and W's 4-bit codes given (serving and prefill)
  serve    the norm written as 4-bit codes and the Linear that reads them
  step     the three products of a training step: X, W [in, out] and dY quantised along both of their axes,
           Y = X.W, dX = dY.W^T, dW = X^T.dY

The 4-bit formats hold E2M1 values (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives), two to a byte, the first in the low half:
  "mxfp4"  one E8M0 scale 2^X per 32 values, X = floor(log2(amax)) - 2, clamped to [-127, 127]
  "nvfp4"  one E4M3 scale s per 16 values under a per-tensor scale g: s = e4m3(amax * g / 6), values e2m1(x * (g / s)), all
           in f32; the product is multiplied by 1/g of both operands
Their scales are stored in 512-byte atoms, one for 128 rows and 4 consecutive scales of each: byte (i % 32) * 16 + (i / 32) * 4 + j
for row i and scale j; atoms in the order [row block][along K], K padded with zero bytes to a multiple of 256. MXFP8's
atoms are the same with K as it is.
"""
import math

import torch

own = False

EPS = 1e-5
OUTLIERS = 6            # columns of the residual stream that are 100 times larger, as in the block7b workload


def listed():
    return [
        # one token of a 4096-wide model: latency
        dict(name="norm decode", kind="norm", rows=1, cols=4096, out="mxfp8", residual=True),
        # the X of the 4096 Linear's training step under delayed scaling
        dict(name="norm fp8 train", kind="norm", rows=8192, cols=4096, out="fp8", residual=True),
        # a ragged prompt, the width of the stress workload, first layer (no residual yet)
        dict(name="norm ragged", kind="norm", rows=1237, cols=1024, out="mxfp8", residual=False),
        # the small Linear's batch
        dict(name="grad small", kind="grad", rows=512, cols=256, residual=True),
        # the 4096 Linear's batch
        dict(name="grad train", kind="grad", rows=8192, cols=4096, residual=True),
        # odd number of rows, no gradient from the residual stream
        dict(name="grad ragged", kind="grad", rows=1999, cols=1024, residual=False),
        # one token through a 4096 projection
        dict(name="serve one token", kind="serve", rows=1, cols=4096, out_features=4096, fmt="mxfp4"),
        # a small batch of tokens through the 7B block's up projection
        dict(name="serve 16 tokens", kind="serve", rows=16, cols=4096, out_features=11008, fmt="nvfp4"),
        # a prompt of 1000 tokens
        dict(name="prefill 1000", kind="linear", rows=1000, cols=4096, out_features=4096, fmt="nvfp4"),
        # the small workload's training step
        dict(name="step 256", kind="step", rows=512, cols=256, out_features=256, fmt="mxfp4"),
        # the benchmark's training step
        dict(name="step 4096", kind="step", rows=8192, cols=4096, out_features=4096, fmt="mxfp4"),
        # the largest: the 7B block's up projection on its 16384 tokens
        dict(name="linear 7b", kind="linear", rows=16384, cols=4096, out_features=11008, fmt="nvfp4"),
    ]


def _log(rng, lo, hi, multiple=1):
    """A size between lo and hi, spread over its logarithm, in whole multiples."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(multiple, int(v / multiple) * multiple)


def draw(rng):
    kind = rng.choice(["norm", "grad", "linear", "serve", "step"])
    if kind in ("norm", "grad"):
        c = dict(kind=kind, rows=_log(rng, 1, 9000), cols=_log(rng, 64, 12000, 32), residual=rng.random() < 0.7)
        if kind == "norm":
            c["out"] = rng.choice(["fp8", "mxfp8", "bf16"])
        return c
    fmt = rng.choice(["mxfp4", "nvfp4"])
    if kind == "step":
        return dict(kind=kind, rows=_log(rng, 64, 8192, 32), cols=_log(rng, 64, 4096, 32),
                    out_features=_log(rng, 64, 4096, 32), fmt=fmt)
    return dict(kind=kind, rows=_log(rng, 1, 128 if kind == "serve" else 8192), cols=_log(rng, 64, 4096, 32),
                out_features=_log(rng, 64, 11008, 8), fmt=fmt)


# ------------------------------------------------------------------ quantisation, in elementary operations
def _e2m1(v):
    """Nearest E2M1 value (ties to the even code) of |v| <= any, saturating at 6; the sign is v's."""
    a = v.abs()
    r = torch.where(a < 2, torch.round(a * 2) / 2, torch.where(a < 4, torch.round(a), torch.round(a / 2) * 2))
    return torch.copysign(r.clamp(max=6.0), v)


def _pow2(e):
    return torch.ldexp(torch.ones((), dtype=torch.float32, device=e.device), e)


def _mx_exponent(amax, emax):
    """floor(log2(amax)) - emax within [-127, 127]; -127 for an amax of zero."""
    e = torch.frexp(amax)[1] - 1 - emax
    return torch.where(amax == 0, torch.full_like(e, -127), e).clamp(-127, 127)


def _fp4(x, fmt, g):
    """E2M1 values and scales (as numbers) of x [rows, K] along its rows."""
    block = 32 if fmt == "mxfp4" else 16
    b = x.float().reshape(x.shape[0], -1, block)
    amax = b.abs().amax(-1)
    if fmt == "mxfp4":
        e = _mx_exponent(amax, 2)
        return _e2m1(b * _pow2(-e)[..., None]).reshape(x.shape), _pow2(e)
    s = ((amax * g) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn).float()
    r = torch.where(s > 0, g / s, torch.zeros_like(s))
    return _e2m1(b * r[..., None]).reshape(x.shape), s


def _times_scales(v, s):
    return (v.reshape(*s.shape, -1) * s[..., None]).reshape(v.shape)


def _pad(t, rows, cols):
    out = torch.zeros(rows, cols, dtype=t.dtype, device=t.device)
    out[:t.shape[0], :t.shape[1]] = t
    return out


def _atoms(codes, per):
    """Scale codes [rows, n] in 512-byte atoms; the atoms of a row block are a multiple of `per`."""
    rows, n = codes.shape
    R, N = -(-rows // 128) * 128, -(-n // (4 * per)) * 4 * per
    a = _pad(codes, R, N).reshape(R // 128, 4, 32, N // 4, 4)
    return a.permute(0, 3, 2, 1, 4).contiguous().reshape(-1)


def _from_atoms(atoms, rows, n, per):
    R, N = -(-rows // 128) * 128, -(-n // (4 * per)) * 4 * per
    a = atoms.reshape(R // 128, N // 4, 32, 4, 4).permute(0, 3, 2, 1, 4)
    return a.reshape(R, N)[:rows, :n]


def _pack(v):
    """E2M1 values to 4-bit codes, two to a byte."""
    c = torch.zeros(v.shape, dtype=torch.uint8, device=v.device)
    a = v.abs()
    c += (a >= 0.5).to(torch.uint8) + (a >= 1).to(torch.uint8) + (a >= 1.5).to(torch.uint8) + (a >= 2).to(torch.uint8)
    c += (a >= 3).to(torch.uint8) + (a >= 4).to(torch.uint8) + (a >= 6).to(torch.uint8) + 8 * torch.signbit(v).to(torch.uint8)
    return (c[:, 0::2] | (c[:, 1::2] << 4)).contiguous()


def _unpack(q, dtype):
    """4-bit codes, two to a byte, to their values."""
    table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], dtype=dtype, device=q.device)
    c = torch.stack((q & 15, q >> 4), -1).reshape(q.shape[0], -1)
    return table[c.int()]


def _scale_codes(s, fmt):
    """The bytes of scales given as numbers."""
    if fmt == "nvfp4":
        return s.to(torch.float8_e4m3fn).view(torch.uint8)
    return (torch.frexp(s)[1] - 1 + 127).clamp(0, 254).to(torch.uint8)


def _scale_values(codes, fmt, dtype):
    if fmt == "nvfp4":
        return codes.view(torch.float8_e4m3fn).to(dtype)
    return torch.ldexp(torch.ones((), dtype=dtype, device=codes.device), codes.int() - 127)


def _weights(q, sf, shape, fmt, dtype):
    """The values that a weight's codes [out, in / 2] and scale atoms stand for."""
    per = 2 if fmt == "mxfp4" else 4
    block = 32 if fmt == "mxfp4" else 16
    s = _scale_values(_from_atoms(sf, shape[0], shape[1] // block, per).contiguous(), fmt, dtype)
    return _times_scales(_unpack(q, dtype), s)


# ------------------------------------------------------------------ inputs
def _normal(gen, rows, cols, sigma):
    return (torch.randn(rows, cols, generator=gen, device="cuda") * sigma).to(torch.bfloat16)


def _stream(gen, rows, cols):
    """A residual stream: N(0, 1) with a few large columns."""
    v = torch.randn(rows, cols, generator=gen, device="cuda")
    at = torch.randperm(cols, generator=gen, device="cuda")[:OUTLIERS]
    v[:, at] *= 100
    return v.to(torch.bfloat16)


def _gamma(gen, cols):
    return (1 + 0.1 * torch.randn(cols, generator=gen, device="cuda")).to(torch.bfloat16)


def _tensor_scale(gen, x, top):
    """The per-tensor scale that the last steps' amax would give: near the present one, but not it."""
    return torch.empty(1, device="cuda").uniform_(0.7, 0.9, generator=gen) * top / x.float().abs().amax().clamp(min=1e-30)


def _inputs(case, seed):
    """The inputs proper, made from the seed alone."""
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    rows, cols, kind = case["rows"], case["cols"], case["kind"]
    s = {}
    if kind in ("norm", "serve"):
        s["x"] = _stream(gen, rows, cols)
        s["residual"] = _stream(gen, rows, cols) if case.get("residual", True) else None
        s["gamma"] = _gamma(gen, cols)
    if kind == "norm":
        s["scale"] = torch.full((1,), 20.0, device="cuda") * torch.empty(1, device="cuda").uniform_(0.8, 1.2, generator=gen)
    if kind == "grad":
        s["dy"] = _normal(gen, rows, cols, 1e-3)
        s["h"] = _stream(gen, rows, cols)
        s["gamma"] = _gamma(gen, cols)
        s["dres"] = _normal(gen, rows, cols, 1e-3) if case["residual"] else None
        s["rstd"] = torch.rsqrt(s["h"].double().square().mean(1) + EPS).float()
    if kind in ("linear", "serve"):
        fmt, n = case["fmt"], case["out_features"]
        w = _normal(gen, n, cols, 0.02)
        s["w_scale"] = _tensor_scale(gen, w, 2688.0)
        v, sc = _fp4(w, fmt, s["w_scale"])
        s["wq"], s["wsf"] = _pack(v), _atoms(_scale_codes(sc, fmt), 2 if fmt == "mxfp4" else 4)
        s["w_scale_inv"] = 1.0 / s["w_scale"]
    if kind == "linear":
        s["x"] = _normal(gen, rows, cols, 1.0)
        s["x_scale"] = _tensor_scale(gen, s["x"], 2688.0)
    if kind == "serve":
        s["x_scale"] = torch.empty(1, device="cuda").uniform_(120.0, 150.0, generator=gen)
    if kind == "step":
        n = case["out_features"]
        s["x"], s["w"], s["dy"] = _normal(gen, rows, cols, 1.0), _normal(gen, cols, n, 0.02), _normal(gen, rows, n, 1e-3)
        for k in ("x", "w", "dy"):
            s[k + "_scale"] = _tensor_scale(gen, s[k], 2688.0)
    return s


def prepare(case, seed):
    s = dict(case, **_inputs(case, seed))
    rows, cols, kind = case["rows"], case["cols"], case["kind"]
    u8 = dict(dtype=torch.uint8, device="cuda")
    bf = dict(dtype=torch.bfloat16, device="cuda")
    f32 = dict(dtype=torch.float32, device="cuda")
    pad = lambda v, m: -(-v // m) * m  # noqa: E731
    if kind == "norm":
        s["h_out"] = torch.empty(rows, cols, **bf) if case["residual"] else None
        s["rstd_out"] = torch.empty(rows, **f32)
        if case["out"] == "bf16":
            s["y_out"] = torch.empty(rows, cols, **bf)
        else:
            s["q_out"] = torch.empty(rows, cols, **u8)
        if case["out"] == "fp8":
            s["amax"], s["scale_inv"] = torch.zeros(1, **f32), torch.empty(1, **f32)
        if case["out"] == "mxfp8":
            s["sf_out"] = torch.zeros(pad(rows, 128) * pad(cols, 128) // 32, **u8)
    if kind == "grad":
        s["dh"], s["dgamma"] = torch.empty(rows, cols, **bf), torch.empty(cols, **f32)
    if kind in ("linear", "serve", "step"):
        n, block = case["out_features"], 32 if case["fmt"] == "mxfp4" else 16
        sf = lambda mn, k: torch.zeros(pad(mn, 128) * pad(k, 256) // block, **u8)  # noqa: E731
        s["xq"], s["xsf"] = torch.empty(rows, cols // 2, **u8), sf(rows, cols)
        s["y"] = torch.empty(rows, n, **bf)
        s["x_scale_inv"] = torch.empty(1, **f32)
        if kind == "serve":
            s["h_out"] = torch.empty(rows, cols, **bf)
        if kind == "step":
            s["xqT"], s["xsfT"] = torch.empty(cols, rows // 2, **u8), sf(cols, rows)
            s["wq"], s["wsf"] = torch.empty(cols, n // 2, **u8), sf(cols, n)
            s["wqT"], s["wsfT"] = torch.empty(n, cols // 2, **u8), sf(n, cols)
            s["dyq"], s["dysf"] = torch.empty(rows, n // 2, **u8), sf(rows, n)
            s["dyqT"], s["dysfT"] = torch.empty(n, rows // 2, **u8), sf(n, rows)
            s["w_scale_inv"], s["dy_scale_inv"] = torch.empty(1, **f32), torch.empty(1, **f32)
            s["dx"], s["dw"] = torch.empty(rows, cols, **bf), torch.empty(cols, n, **bf)
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    return _own(state) if own else _plain(state)


def _own(s):
    import optimizer_fp8_cast_b200 as fp8
    kind = s["kind"]
    if kind == "norm":
        out = s["out"]
        if out == "bf16":
            fp8.fp8_rmsnorm_cast(s["x"], s["gamma"], EPS, residual=s["residual"], h=s["h_out"], rstd=s["rstd_out"],
                                 y=s["y_out"])
            return dict(h=s["h_out"], rstd=s["rstd_out"], y=s["y_out"])
        if out == "fp8":
            fp8.fp8_rmsnorm_cast(s["x"], s["gamma"], EPS, residual=s["residual"], h=s["h_out"], rstd=s["rstd_out"],
                                 quant=fp8.Q_FP8, q=s["q_out"], scale=s["scale"], amax=s["amax"],
                                 scale_inv=s["scale_inv"])
            return dict(h=s["h_out"], rstd=s["rstd_out"], q=s["q_out"].view(torch.float8_e4m3fn), amax=s["amax"],
                        scale_inv=s["scale_inv"])
        fp8.fp8_rmsnorm_cast(s["x"], s["gamma"], EPS, residual=s["residual"], h=s["h_out"], rstd=s["rstd_out"],
                             quant=fp8.Q_MXFP8, q=s["q_out"], sf=s["sf_out"])
        return dict(h=s["h_out"], rstd=s["rstd_out"], q=s["q_out"].view(torch.float8_e4m3fn),
                    sf=s["sf_out"].view(torch.float8_e8m0fnu))
    if kind == "grad":
        fp8.fp8_rmsnorm_backward(s["dy"], s["h"], s["gamma"], s["rstd"], s["dh"], dres=s["dres"], dgamma=s["dgamma"])
        return dict(dh=s["dh"], dgamma=s["dgamma"])
    nv = s["fmt"] == "nvfp4"
    quant = fp8.Q_NVFP4 if nv else fp8.Q_MXFP4
    extra = lambda k: dict(scale=s[k + "_scale"], scale_inv=s[k + "_scale_inv"]) if nv else {}  # noqa: E731
    inv = lambda a, b: dict(a_scale_inv=s[a + "_scale_inv"], b_scale_inv=s[b + "_scale_inv"]) if nv else {}  # noqa: E731
    if kind == "serve":
        fp8.fp8_rmsnorm_cast(s["x"], s["gamma"], EPS, residual=s["residual"], h=s["h_out"], quant=quant, q=s["xq"],
                             sf=s["xsf"], **extra("x"))
        fp8.fp4_gemm_multi([dict(A=s["xq"], a_sf=s["xsf"], B=s["wq"], b_sf=s["wsf"], quant=quant, D=s["y"],
                                 **inv("x", "w"))])
        return dict(h=s["h_out"], y=s["y"])
    if kind == "linear":
        fp8.fp4_cast_multi([dict(x=s["x"], quant=quant, q_row=s["xq"], sf_row=s["xsf"], **extra("x"))])
        fp8.fp4_gemm_multi([dict(A=s["xq"], a_sf=s["xsf"], B=s["wq"], b_sf=s["wsf"], quant=quant, D=s["y"],
                                 **inv("x", "w"))])
        return s["y"]
    fp8.fp4_cast_multi([dict(x=s[k], quant=quant, q_row=s[k + "q"], sf_row=s[k + "sf"], q_col=s[k + "qT"],
                             sf_col=s[k + "sfT"], **extra(k)) for k in ("x", "w", "dy")])
    fp8.fp4_gemm_multi([dict(A=s["xq"], a_sf=s["xsf"], B=s["wqT"], b_sf=s["wsfT"], quant=quant, D=s["y"], **inv("x", "w")),
                        dict(A=s["dyq"], a_sf=s["dysf"], B=s["wq"], b_sf=s["wsf"], quant=quant, D=s["dx"], **inv("dy", "w")),
                        dict(A=s["xqT"], a_sf=s["xsfT"], B=s["dyqT"], b_sf=s["dysfT"], quant=quant, D=s["dw"],
                             **inv("x", "dy"))])
    return dict(y=s["y"], dx=s["dx"], dw=s["dw"])


def _norm(s):
    h = s["x"] if s["residual"] is None else (s["x"].float() + s["residual"].float()).to(torch.bfloat16)
    hf = h.float()
    rstd = torch.rsqrt(hf.square().mean(1) + EPS)
    return h, rstd, hf * rstd[:, None] * s["gamma"].float()


def _plain(s):
    kind = s["kind"]
    if kind == "norm":
        h, rstd, y = _norm(s)
        h = None if s["residual"] is None else h
        if s["out"] == "bf16":
            return dict(h=h, rstd=rstd, y=y.to(torch.bfloat16))
        if s["out"] == "fp8":
            return dict(h=h, rstd=rstd, q=(y * s["scale"]).clamp(-448, 448).to(torch.float8_e4m3fn),
                        amax=y.abs().amax().reshape(1), scale_inv=1.0 / s["scale"])
        b = y.reshape(y.shape[0], -1, 32)
        e = _mx_exponent(b.abs().amax(-1), 8)
        q = (b * _pow2(-e)[..., None]).clamp(-448, 448).reshape(y.shape).to(torch.float8_e4m3fn)
        return dict(h=h, rstd=rstd, q=q, sf=_atoms((e + 127).to(torch.uint8), 1).view(torch.float8_e8m0fnu))
    if kind == "grad":
        dy, xh = s["dy"].float(), s["h"].float() * s["rstd"][:, None]
        g = dy * s["gamma"].float()
        dh = s["rstd"][:, None] * (g - xh * (g * xh).mean(1, keepdim=True))
        if s["dres"] is not None:
            dh = dh + s["dres"].float()
        return dict(dh=dh.to(torch.bfloat16), dgamma=(dy * xh).sum(0))
    fmt = s["fmt"]
    if kind in ("linear", "serve"):
        h, x = None, s["x"]
        if kind == "serve":
            h, _, x = _norm(s)
        a = _times_scales(*_fp4(x, fmt, s["x_scale"]))
        w = _weights(s["wq"], s["wsf"], (s["out_features"], s["cols"]), fmt, torch.float32)
        y = a @ w.T
        if fmt == "nvfp4":
            y = y * ((1.0 / s["x_scale"]) * s["w_scale_inv"])
        y = y.to(torch.bfloat16)
        return y if kind == "linear" else dict(h=h, y=y)
    back = {k: (1.0 / s[k + "_scale"] if fmt == "nvfp4" else 1.0) for k in ("x", "w", "dy")}
    row = {k: _times_scales(*_fp4(s[k], fmt, s[k + "_scale"])) for k in ("x", "w", "dy")}
    col = {k: _times_scales(*_fp4(s[k].T, fmt, s[k + "_scale"])) for k in ("x", "w", "dy")}
    return dict(y=((row["x"] @ col["w"].T) * (back["x"] * back["w"])).to(torch.bfloat16),
                dx=((row["dy"] @ row["w"].T) * (back["dy"] * back["w"])).to(torch.bfloat16),
                dw=((col["x"] @ col["dy"].T) * (back["x"] * back["dy"])).to(torch.bfloat16))


def work(case):
    rows, cols, kind = case["rows"], case["cols"], case["kind"]
    e = rows * cols
    if kind == "norm":
        codes = {"fp8": 1.0, "mxfp8": 1.0 + 1 / 32, "bf16": 2.0}[case["out"]]
        return dict(bytes=e * (2 + codes + (4 if case["residual"] else 0)) + 2 * cols + 4 * rows, flops=5 * e)
    if kind == "grad":
        return dict(bytes=e * (8 if case["residual"] else 6) + 6 * cols + 4 * rows, flops=10 * e)
    n = case["out_features"]
    if kind == "step":
        return dict(bytes=4 * (e + cols * n + rows * n), flops=6 * e * n)
    held = 0.5 + (1 / 32 if case["fmt"] == "mxfp4" else 1 / 16)
    return dict(bytes=e * (6 if kind == "serve" else 2) + cols * n * held + 2 * rows * n, flops=2 * e * n)


# ------------------------------------------------------------------ in 64 bits
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _nearest(v, values, half):
    """The nearest of the sorted non-negative `values` (ties to the even index) to |v|, with v's sign; `half`: the middles."""
    a = v.abs()
    up, down = torch.bucketize(a, half, right=True), torch.bucketize(a, half)      # differ at a tie
    at = torch.where(up == down, up, torch.where(up % 2 == 0, up, down))
    return torch.where(torch.signbit(v), -values[at], values[at])


def _grid(values, like):
    v = torch.tensor(values, dtype=torch.float64, device=like.device)
    return v, (v[1:] + v[:-1]) / 2


def _e4m3_values():
    return [m / 8 * 2.0 ** -6 for m in range(8)] + [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)][:-1]


def _exact_exponent(amax, emax):
    e = torch.floor(torch.log2(amax.clamp(min=2.0 ** -200)))
    e = torch.where(torch.exp2(e) > amax, e - 1, e)
    e = torch.where(torch.exp2(e + 1) <= amax, e + 1, e)
    return torch.where(amax > 0, (e - emax).clamp(-127, 127), torch.full_like(e, -127))


def _exact_fp4(x, fmt, g):
    """The numbers that the 4-bit form of x [rows, K] stands for, without the per-tensor factor."""
    values, half = _grid(_E2M1, x)
    rows, k = x.shape
    block = 32 if fmt == "mxfp4" else 16
    b = x.double().reshape(rows, k // block, block)
    amax = b.abs().amax(-1, keepdim=True)
    if fmt == "mxfp4":
        unit = torch.exp2(_exact_exponent(amax, 2))
        return (_nearest(b / unit, values, half) * unit).reshape(rows, k)
    s = _nearest(amax * g.double() / 6, *_grid(_e4m3_values(), x))
    scaled = torch.where(s > 0, b * g.double() / s, torch.zeros_like(b))
    return (_nearest(scaled, values, half) * s).reshape(rows, k)


def exact(case, seed):
    s = _inputs(case, seed)
    kind, fmt = case["kind"], case.get("fmt")
    if kind in ("norm", "serve"):
        h = s["x"].double()
        if s["residual"] is not None:
            h = (s["x"].double() + s["residual"].double()).to(torch.bfloat16)
        hd = h.double()
        rstd = 1 / torch.sqrt((hd * hd).sum(1) / case["cols"] + EPS)
        y = hd * rstd[:, None] * s["gamma"].double()
        h = None if s["residual"] is None else h
    if kind == "norm":
        if case["out"] == "bf16":
            return dict(h=h, rstd=rstd, y=y)
        values, half = _grid(_e4m3_values(), y)
        if case["out"] == "fp8":
            g = s["scale"].double()
            return dict(h=h, rstd=rstd, q=_nearest(y * g, values, half), amax=y.abs().amax().reshape(1), scale_inv=1 / g)
        b = y.reshape(case["rows"], -1, 32)
        e = _exact_exponent(b.abs().amax(-1), 8)
        q = _nearest(b / torch.exp2(e)[..., None], values, half).reshape(y.shape)
        n = -(-case["rows"] // 128) * 128
        k = -(-e.shape[1] // 4) * 4
        sf = torch.full((n, k), -127.0, dtype=torch.float64, device="cuda")
        sf[:case["rows"], :e.shape[1]] = e
        sf = torch.exp2(sf.reshape(n // 128, 4, 32, k // 4, 4).permute(0, 3, 2, 1, 4)).reshape(-1)
        return dict(h=h, rstd=rstd, q=q, sf=sf)
    if kind == "grad":
        dy, h, gamma, r = s["dy"].double(), s["h"].double(), s["gamma"].double(), s["rstd"].double()[:, None]
        dot = (dy * gamma * h).sum(1, keepdim=True) / case["cols"]
        dh = r * dy * gamma - r ** 3 * h * dot
        if s["dres"] is not None:
            dh += s["dres"].double()
        return dict(dh=dh, dgamma=torch.einsum("rc,rc->c", dy, h * r))
    nv = fmt == "nvfp4"
    if kind in ("linear", "serve"):
        a = _exact_fp4(y if kind == "serve" else s["x"], fmt, s["x_scale"])
        w = _weights(s["wq"], s["wsf"], (case["out_features"], case["cols"]), fmt, torch.float64)
        d = a @ w.T
        if nv:
            d /= s["x_scale"].double() / s["w_scale_inv"].double()
        return d if kind == "linear" else dict(h=h, y=d)
    f = {k: (1 / s[k + "_scale"].double() if nv else 1.0) for k in ("x", "w", "dy")}
    row = {k: _exact_fp4(s[k], fmt, s[k + "_scale"]) for k in ("x", "w", "dy")}
    col = {k: _exact_fp4(s[k].T, fmt, s[k + "_scale"]) for k in ("x", "w", "dy")}
    return dict(y=row["x"] @ col["w"].T * (f["x"] * f["w"]), dx=row["dy"] @ row["w"].T * (f["dy"] * f["w"]),
                dw=col["x"] @ col["dy"].T * (f["x"] * f["dy"]))
