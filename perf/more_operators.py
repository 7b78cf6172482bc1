"""What is measured of a gated feed-forward block: its FP8 training products, the Muon step of its matrices and its
4-bit weights serving a few tokens (every matrix is row-major).

Kinds of cases:

  gated    [G | U] = (A . W) * sa * sb with A [rows, k] and W the gate's and the up projection's weights side by side, all FP8 codes
           under one scale each; h = act(G) * U in f32, written as FP8 codes under a scale (with their amax and the scale's
           inverse) or as BF16, and [G | U] as BF16 where the gradient will need it
  back     its gradient: dH = (dY . Wd^T) * sa * sb of the down projection's FP8 codes, dG = dH * U * act'(G), dU = dH * act(G),
           [dG | dU] as E5M2 codes under one scale (with amax and inverse scale) or as BF16
  orth     the nearest-orthogonal factor of a matrix by five Newton-Schulz steps: X = X0 / |X0|; A = X X^T; X <- aX + (bA + cA^2) X
  muon     the Muon step of a list of matrices: m <- beta m + g / S; U = g / S + beta m; p <- p (1 - lr wd) - lr r sqrt(max(rows, cols)) O
           with O the orthogonal factor of U; the BF16 weight is p rounded
  matvec   y = x . W^T for one to eight BF16 rows x and 4-bit weights W with block scales; gated: y = act(g) * u of both halves of the outputs

act is SiLU, g * sigmoid(g), or GELU in its tanh form, which is g * sigmoid(2 sqrt(2 / pi) (g + 0.044715 g^3)).
The 4-bit formats hold E2M1 values, two to a byte, the first in the low half, under E8M0 scales per 32 values ("mxfp4") or E4M3
scales per 16 values and one f32 factor ("nvfp4"); the scales lie in 512-byte atoms of 128 rows x 4 scales: byte
(i % 32) * 16 + (i / 32) * 4 + j, K padded to a multiple of 256.
"""
import math

import torch

own = False

NS = (3.4445, -4.7750, 2.0315)
STEPS = 5
# the optimiser's settings: lr, weight decay and loss scale of the small Linear's workload
LR, BETA, WD, RMS, LOSS_SCALE = 1e-4, 0.95, 0.01, 0.2, 1024.0


def listed():
    return [
        # one token through a 4096 -> 11008 block's gate and up projections in FP8: latency and the weights' bytes
        dict(name="gated one token", kind="gated", rows=1, k=4096, n=11008, act="silu", out="fp8", keep=False, in_out=True),
        # a ragged batch of the 1024-wide workload, weights stored [out, in], GELU, BF16 output and what the gradient needs
        dict(name="gated ragged", kind="gated", rows=1237, k=1024, n=2752, act="gelu", out="bf16", keep=True, in_out=False),
        # the 7B block's gate and up projections on its 16384 tokens, training
        dict(name="gated 7b", kind="gated", rows=16384, k=4096, n=11008, act="silu", out="fp8", keep=True, in_out=True),
        # the small workload's 512 tokens
        dict(name="back small", kind="back", rows=512, k=256, n=688, act="gelu", out="bf16"),
        # the 7B block's gradient
        dict(name="back 7b", kind="back", rows=16384, k=4096, n=11008, act="silu", out="fp8"),
        # the small Linear's gradient: launches and latency
        dict(name="orth 256", kind="orth", rows=256, cols=256, dtype="bf16"),
        # a tall matrix of odd sizes
        dict(name="orth ragged", kind="orth", rows=1237, cols=611, dtype="f32"),
        # the benchmark's Linear
        dict(name="muon 4096", kind="muon", shapes="4096x4096"),
        # all matrices of the 7B block: q, k, v, o, gate, up, down
        dict(name="muon 7b", kind="muon", shapes="4096x4096,4096x4096,4096x4096,4096x4096,4096x11008,4096x11008,11008x4096"),
        # one token through a 4096 projection
        dict(name="matvec one token", kind="matvec", rows=1, k=4096, n=4096, fmt="mxfp4", act="none"),
        # four tokens through the 7B block's gate and up projections
        dict(name="matvec gated", kind="matvec", rows=4, k=4096, n=11008, fmt="nvfp4", act="silu"),
        # eight tokens through its down projection
        dict(name="matvec 8 tokens", kind="matvec", rows=8, k=11008, n=4096, fmt="mxfp4", act="none"),
    ]


def _log(rng, lo, hi, multiple=1):
    """A size between lo and hi, spread over its logarithm, in whole multiples."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(multiple, int(v / multiple) * multiple)


def draw(rng):
    kind = rng.choice(["gated", "back", "orth", "muon", "matvec"])
    if kind in ("gated", "back"):
        c = dict(kind=kind, rows=_log(rng, 1, 16384), k=_log(rng, 64, 4096, 16), n=_log(rng, 64, 11008, 16),
                 act=rng.choice(["silu", "gelu"]), out=rng.choice(["fp8", "bf16"]))
        if kind == "gated":
            c.update(keep=rng.random() < 0.6, in_out=rng.random() < 0.5)
        return c
    if kind == "orth":
        return dict(kind=kind, rows=_log(rng, 1, 6000), cols=_log(rng, 1, 6000), dtype=rng.choice(["bf16", "f32"]))
    if kind == "muon":
        return dict(kind=kind, shapes=",".join("%dx%d" % (_log(rng, 8, 4096), _log(rng, 8, 4096)) for _ in range(rng.randint(1, 4))))
    return dict(kind=kind, rows=rng.randint(1, 8), k=_log(rng, 64, 11008, 32), n=_log(rng, 64, 11008, 8),
                fmt=rng.choice(["mxfp4", "nvfp4"]), act=rng.choice(["none", "silu", "gelu"]))


def _shapes(case):
    return [tuple(int(v) for v in s.split("x")) for s in case["shapes"].split(",")]


# ------------------------------------------------------------------ inputs
def _normal(gen, rows, cols, sigma):
    return torch.randn(rows, cols, generator=gen, device="cuda") * sigma


def _codes(x, top, kind, gen):
    """FP8 codes of x under the scale that the last steps' amax would give (near the present one), and the inverse scale."""
    scale = torch.empty(1, device="cuda").uniform_(0.7, 0.9, generator=gen) * top / x.abs().amax().clamp(min=1e-30)
    return (x * scale).clamp(-top, top).to(kind).view(torch.uint8), 1.0 / scale


def _gradient(gen, rows, cols):
    """A weight's gradient: noise and a few strong directions, as large together."""
    r = 4
    noise = _normal(gen, rows, cols, 1e-3)
    strong = _normal(gen, rows, r, 1.0) @ _normal(gen, r, cols, 1.0) * (1e-3 / math.sqrt(r))
    return noise + strong


def _pack(c):
    return (c[:, 0::2] | (c[:, 1::2] << 4)).contiguous()


def _atoms(codes, per):
    """Scale codes [rows, n] in 512-byte atoms, K padded with zero bytes to 256 values (`per` atoms)."""
    rows, n = codes.shape
    R, N = -(-rows // 128) * 128, -(-n // (4 * per)) * 4 * per
    out = torch.zeros(R, N, dtype=torch.uint8, device=codes.device)
    out[:rows, :n] = codes
    return out.reshape(R // 128, 4, 32, N // 4, 4).permute(0, 3, 2, 1, 4).contiguous().reshape(-1)


def _from_atoms(atoms, rows, n, per):
    R, N = -(-rows // 128) * 128, -(-n // (4 * per)) * 4 * per
    return atoms.reshape(R // 128, N // 4, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(R, N)[:rows, :n]


def _fp4_weights(gen, rows, k, fmt):
    """4-bit weights whose values are near N(0, 0.02): codes, scale atoms and the inverse of the tensor scale."""
    block = 32 if fmt == "mxfp4" else 16
    w = _normal(gen, rows, k, 0.02)
    amax = w.reshape(rows, -1, block).abs().amax(-1)
    if fmt == "mxfp4":
        e = torch.floor(torch.log2(amax)) - 2
        s, code, inv = torch.exp2(e), (e + 127).to(torch.uint8), torch.ones(1, device="cuda")
    else:
        g = 2688.0 * 0.8 / amax.max()
        s8 = (amax * g / 6).clamp(min=2.0 ** -9, max=448).to(torch.float8_e4m3fn)
        s, code, inv = s8.float() / g, s8.view(torch.uint8), (1.0 / g).reshape(1)
    a = (w.reshape(rows, -1, block) / s[..., None]).reshape(rows, k)
    c = torch.zeros(rows, k, dtype=torch.uint8, device="cuda")
    for border in (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0):
        c += (a.abs() > border).to(torch.uint8)
    c += 8 * (a < 0).to(torch.uint8)
    return _pack(c), _atoms(code, 2 if fmt == "mxfp4" else 4), inv


def _inputs(case, seed):
    """The inputs proper, made from the seed alone."""
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    kind, s = case["kind"], {}
    e4, e5 = torch.float8_e4m3fn, torch.float8_e5m2
    scale = lambda v: torch.full((1,), v, device="cuda") * torch.empty(1, device="cuda").uniform_(0.7, 0.9, generator=gen)  # noqa: E731
    if kind == "gated":
        M, K, N = case["rows"], case["k"], case["n"]
        s["a"], s["a_inv"] = _codes(_normal(gen, M, K, 1.0), 448.0, e4, gen)
        w, s["w_inv"] = _codes(_normal(gen, K, 2 * N, 2.0 / math.sqrt(K)), 448.0, e4, gen)
        s["w"] = w if case["in_out"] else w.T.contiguous()
        s["scale"] = scale(8.0)            # h reaches about 50
    if kind == "back":
        M, K, N = case["rows"], case["k"], case["n"]
        s["a"], s["a_inv"] = _codes(_normal(gen, M, K, 1e-3), 57344.0, e5, gen)
        s["w"], s["w_inv"] = _codes(_normal(gen, N, K, 1.0 / math.sqrt(K)), 448.0, e4, gen)
        s["gu"] = _normal(gen, M, 2 * N, 2.0).to(torch.bfloat16)
        s["scale"] = scale(57344.0 / 0.05)
    if kind == "orth":
        x = _gradient(gen, case["rows"], case["cols"])
        s["x"] = x.to(torch.bfloat16) if case["dtype"] == "bf16" else x
    if kind == "muon":
        s["p"], s["m"], s["g"] = [], [], []
        for r, c in _shapes(case):
            s["p"].append(_normal(gen, r, c, 0.02))
            s["m"].append(_gradient(gen, r, c) * 4)
            s["g"].append((_gradient(gen, r, c) * LOSS_SCALE).to(torch.bfloat16))
    if kind == "matvec":
        M, K, N = case["rows"], case["k"], case["n"]
        s["x"] = _normal(gen, M, K, 1.0).to(torch.bfloat16)
        s["q"], s["sf"], s["w_inv"] = _fp4_weights(gen, N if case["act"] == "none" else 2 * N, K, case["fmt"])
    return s


def prepare(case, seed):
    s = dict(case, **_inputs(case, seed))
    kind = case["kind"]
    dev = dict(device="cuda")
    if kind in ("gated", "back"):
        wide = case["n"] * (1 if kind == "gated" else 2)
        if case["out"] == "fp8":
            s["q_out"] = torch.empty(case["rows"], wide, dtype=torch.uint8, **dev)
            s["amax"], s["scale_inv"] = torch.zeros(1, **dev), torch.empty(1, **dev)
        else:
            s["h_out"] = torch.empty(case["rows"], wide, dtype=torch.bfloat16, **dev)
        if kind == "gated" and case["keep"]:
            s["gu_out"] = torch.empty(case["rows"], 2 * case["n"], dtype=torch.bfloat16, **dev)
    if kind == "orth":
        s["out"] = torch.empty(case["rows"], case["cols"], dtype=torch.bfloat16, **dev)
    if kind == "muon":
        s["w"] = [p.to(torch.bfloat16) for p in s["p"]]
    if kind == "matvec":
        s["y"] = torch.empty(case["rows"], case["n"], dtype=torch.bfloat16, **dev)
    if kind in ("orth", "muon"):
        # scratch as a program keeps it over the steps, grown by the first call
        s["workspace"] = {}
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    return _own(state) if own else _plain(state)


def _workspace(fp8, s, shapes):
    if "bytes" not in s["workspace"]:
        s["workspace"]["bytes"] = torch.empty(fp8.muon_workspace_bytes(shapes), dtype=torch.uint8, device="cuda")
    return s["workspace"]["bytes"]


def _own(s):
    import optimizer_fp8_cast_b200 as fp8
    kind = s["kind"]
    act = {"silu": fp8.ACT_SILU, "gelu": fp8.ACT_GELU, "none": fp8.ACT_NONE}[s.get("act", "none")]
    if kind == "gated":
        if s["out"] == "fp8":
            fp8.fp8_gated_gemm(s["a"], fp8.E4M3, s["w"], fp8.E4M3, s["a_inv"], s["w_inv"], act=act, b_mn=s["in_out"],
                               gu=s.get("gu_out"), q=s["q_out"], q_fmt=fp8.E4M3, scale=s["scale"], amax=s["amax"],
                               scale_inv=s["scale_inv"])
            return dict(gu=s.get("gu_out"), q=s["q_out"].view(torch.float8_e4m3fn), amax=s["amax"], scale_inv=s["scale_inv"])
        fp8.fp8_gated_gemm(s["a"], fp8.E4M3, s["w"], fp8.E4M3, s["a_inv"], s["w_inv"], act=act, b_mn=s["in_out"],
                           gu=s.get("gu_out"), h=s["h_out"])
        return dict(gu=s.get("gu_out"), h=s["h_out"])
    if kind == "back":
        if s["out"] == "fp8":
            fp8.fp8_gated_gemm_backward(s["a"], fp8.E5M2, s["w"], fp8.E4M3, s["a_inv"], s["w_inv"], s["gu"], act=act,
                                        q=s["q_out"], q_fmt=fp8.E5M2, scale=s["scale"], amax=s["amax"],
                                        scale_inv=s["scale_inv"])
            return dict(q=s["q_out"].view(torch.float8_e5m2), amax=s["amax"], scale_inv=s["scale_inv"])
        fp8.fp8_gated_gemm_backward(s["a"], fp8.E5M2, s["w"], fp8.E4M3, s["a_inv"], s["w_inv"], s["gu"], act=act,
                                    dgu=s["h_out"])
        return s["h_out"]
    if kind == "orth":
        fp8.muon_orthogonalize([s["x"]], [s["out"]], steps=STEPS, workspace=_workspace(fp8, s, [s["x"].shape]))
        return s["out"]
    if kind == "muon":
        fp8.fused_muon_multi_tensor(s["p"], s["m"], s["g"], s["w"], lr=LR, beta=BETA, weight_decay=WD, update_rms=RMS,
                                    loss_scale=LOSS_SCALE, nesterov=True, steps=STEPS,
                                    workspace=_workspace(fp8, s, [p.shape for p in s["p"]]))
        return dict(p=s["p"], m=s["m"], w=s["w"])
    quant = fp8.Q_MXFP4 if s["fmt"] == "mxfp4" else fp8.Q_NVFP4
    fp8.fp4_matvec(s["x"], s["q"], s["sf"], quant, s["y"], w_scale_inv=s["w_inv"] if s["fmt"] == "nvfp4" else None, act=act)
    return s["y"]


def _gate(g, act):
    """The argument of the sigmoid in act(g) = g * sigmoid(w), and its derivative."""
    if act == "silu":
        return g, torch.ones_like(g)
    c = 2 * math.sqrt(2 / math.pi)
    return c * (g + 0.044715 * g ** 3), c * (1 + 3 * 0.044715 * g * g)


def _e2m1(q, dtype):
    table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], dtype=dtype, device=q.device)
    return table[torch.stack((q & 15, q >> 4), -1).reshape(q.shape[0], -1).int()]


def _fp4_values(s, dtype):
    block, per = (32, 2) if s["fmt"] == "mxfp4" else (16, 4)
    rows, k = s["q"].shape[0], s["k"]
    codes = _from_atoms(s["sf"], rows, k // block, per).contiguous()
    if s["fmt"] == "mxfp4":
        sc = torch.ldexp(torch.ones((), dtype=dtype, device="cuda"), codes.int() - 127)
    else:
        sc = codes.view(torch.float8_e4m3fn).to(dtype)
    return (_e2m1(s["q"], dtype).reshape(rows, -1, block) * sc[..., None]).reshape(rows, k)


def _newton_schulz(x):
    a, b, c = NS
    tall = x.shape[0] > x.shape[1]
    x = x.T if tall else x
    norm = torch.linalg.vector_norm(x)
    x = x / torch.where(norm > 0, norm, torch.ones_like(norm))
    for _ in range(STEPS):
        g = x @ x.T
        x = a * x + (b * g + c * (g @ g)) @ x
    return x.T if tall else x


def _plain(s):
    kind = s["kind"]
    e4, e5 = torch.float8_e4m3fn, torch.float8_e5m2
    if kind == "gated":
        w = s["w"].view(e4).float()
        gu = (s["a"].view(e4).float() @ (w if s["in_out"] else w.T)) * (s["a_inv"] * s["w_inv"])
        g, u = gu[:, :s["n"]], gu[:, s["n"]:]
        h = g * torch.sigmoid(_gate(g, s["act"])[0]) * u
        gu = gu.to(torch.bfloat16) if s["keep"] else None
        if s["out"] == "bf16":
            return dict(gu=gu, h=h.to(torch.bfloat16))
        return dict(gu=gu, q=(h * s["scale"]).clamp(-448, 448).to(e4), amax=h.abs().amax().reshape(1), scale_inv=1.0 / s["scale"])
    if kind == "back":
        dh = (s["a"].view(e5).float() @ s["w"].view(e4).float().T) * (s["a_inv"] * s["w_inv"])
        g, u = s["gu"][:, :s["n"]].float(), s["gu"][:, s["n"]:].float()
        w, dw = _gate(g, s["act"])
        sg = torch.sigmoid(w)
        d = torch.cat((dh * u * (sg + g * sg * (1 - sg) * dw), dh * (g * sg)), 1)
        if s["out"] == "bf16":
            return d.to(torch.bfloat16)
        return dict(q=(d * s["scale"]).clamp(-57344, 57344).to(e5), amax=d.abs().amax().reshape(1), scale_inv=1.0 / s["scale"])
    if kind == "orth":
        return _newton_schulz(s["x"].float()).to(torch.bfloat16)
    if kind == "muon":
        for p, m, g, w in zip(s["p"], s["m"], s["g"], s["w"]):
            g = g.float() / LOSS_SCALE
            m.mul_(BETA).add_(g)
            o = _newton_schulz(g + BETA * m)
            p.mul_(1 - LR * WD).sub_(o, alpha=LR * RMS * math.sqrt(max(p.shape)))
            w.copy_(p)
        return dict(p=s["p"], m=s["m"], w=s["w"])
    y = s["x"].float() @ _fp4_values(s, torch.float32).T * s["w_inv"]
    if s["act"] != "none":
        g, u = y[:, :s["n"]], y[:, s["n"]:]
        y = g * torch.sigmoid(_gate(g, s["act"])[0]) * u
    return y.to(torch.bfloat16)


def work(case):
    kind = case["kind"]
    if kind in ("gated", "back"):
        M, K, N = case["rows"], case["k"], case["n"]
        out = 1 if case["out"] == "fp8" else 2
        if kind == "gated":
            return dict(bytes=M * K + 2 * N * K + M * N * (out + (4 if case["keep"] else 0)), flops=4 * M * N * K)
        return dict(bytes=M * K + N * K + M * N * (4 + 2 * out), flops=2 * M * N * K)
    if kind in ("orth", "muon"):
        shapes = [(case["rows"], case["cols"])] if kind == "orth" else _shapes(case)
        each = (6 if case.get("dtype") == "f32" else 4) if kind == "orth" else 20
        # the two symmetric products need one half each
        flops = sum(STEPS * (3 * min(v) ** 2 * max(v) + min(v) ** 3) for v in shapes)
        return dict(bytes=sum(r * c for r, c in shapes) * each, flops=flops)
    M, K, N = case["rows"], case["k"], case["n"]
    outs = N if case["act"] == "none" else 2 * N
    held = 0.5 + (1 / 32 if case["fmt"] == "mxfp4" else 1 / 16)
    return dict(bytes=int(outs * K * held) + 2 * M * (K + N), flops=2 * M * outs * K)


# ------------------------------------------------------------------ in 64 bits
def _fp8_values(mantissa, bias, top):
    """The non-negative values of an 8-bit format with `mantissa` bits, up to `top`."""
    m = 2 ** mantissa
    v = [i / m * 2.0 ** (1 - bias) for i in range(m)]
    e = 1
    while v[-1] < top:
        v += [(1 + i / m) * 2.0 ** (e - bias) for i in range(m)]
        e += 1
    return [x for x in v if x <= top]


def _nearest(v, values):
    """v rounded to the nearest of the sorted non-negative `values` with v's sign, ties to the even index."""
    values = torch.tensor(values, dtype=torch.float64, device=v.device)
    half = (values[1:] + values[:-1]) / 2
    up, down = torch.bucketize(v.abs(), half, right=True), torch.bucketize(v.abs(), half)
    at = torch.where(up == down, up, torch.where(up % 2 == 0, up, down))
    return torch.copysign(values[at], v)


def _exact_orth(x):
    """Through the Gram matrix's other side: p(X) = X (a + b X^T X + c (X^T X)^2), on the smaller of the two sides."""
    a, b, c = NS
    x = x.double()
    norm = x.square().sum().sqrt()
    x = x / norm if norm > 0 else x
    wide = x.shape[1] >= x.shape[0]
    eye = torch.eye(min(x.shape), dtype=torch.float64, device=x.device)
    for _ in range(STEPS):
        gram = x.matmul(x.mT) if wide else x.mT.matmul(x)
        p = a * eye + gram.matmul(b * eye + c * gram)
        x = p.matmul(x) if wide else x.matmul(p)
    return x


def exact(case, seed):
    s = dict(case, **_inputs(case, seed))
    kind = case["kind"]
    e4, e5 = torch.float8_e4m3fn, torch.float8_e5m2
    if kind in ("gated", "back"):
        a, w = s["a"].view(e4 if kind == "gated" else e5).double(), s["w"].view(e4).double()
        unit = s["a_inv"].double() * s["w_inv"].double()
        n, sc = case["n"], s["scale"].double()

        def act(g):            # value and derivative, from tanh
            if case["act"] == "silu":
                t, dt = torch.tanh(g / 2), 0.5
            else:
                r = math.sqrt(2 / math.pi)
                t, dt = torch.tanh(r * (g + 0.044715 * g * g * g)), r * (1 + 0.134145 * g * g)
            return g * (1 + t) / 2, (1 + t) / 2 + g / 2 * (1 - t * t) * dt
    if kind == "gated":
        gu = torch.einsum("mk,kn->mn" if case["in_out"] else "mk,nk->mn", a, w) * unit
        h = act(gu[:, :n])[0] * gu[:, n:]
        gu = gu if case["keep"] else None
        if case["out"] == "bf16":
            return dict(gu=gu, h=h)
        return dict(gu=gu, q=_nearest(h * sc, _fp8_values(3, 7, 448.0)), amax=h.abs().max().reshape(1), scale_inv=1 / sc)
    if kind == "back":
        dh = torch.einsum("mk,nk->mn", a, w) * unit
        gu = s["gu"].double()
        v, dv = act(gu[:, :n])
        d = torch.cat((dh * dv * gu[:, n:], dh * v), 1)
        if case["out"] == "bf16":
            return d
        return dict(q=_nearest(d * sc, _fp8_values(2, 15, 57344.0)), amax=d.abs().max().reshape(1), scale_inv=1 / sc)
    if kind == "orth":
        return _exact_orth(s["x"])
    if kind == "muon":
        out = dict(p=[], m=[], w=[])
        for p, m, g in zip(s["p"], s["m"], s["g"]):
            g = g.double() / LOSS_SCALE
            m = BETA * m.double() + g
            o = _exact_orth(g + BETA * m)
            p = (1 - LR * WD) * p.double() - LR * RMS * max(p.shape) ** 0.5 * o
            for k, v in (("p", p), ("m", m), ("w", p)):
                out[k].append(v)
        return out
    y = torch.einsum("mk,nk->mn", s["x"].double(), _fp4_values(s, torch.float64)) * s["w_inv"].double()
    if case["act"] != "none":
        g, u = y.chunk(2, 1)
        z = g / 2 if case["act"] == "silu" else math.sqrt(2 / math.pi) * (g + 0.044715 * g * g * g)
        y = g * (1 + torch.tanh(z)) / 2 * u
    return y
