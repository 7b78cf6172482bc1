"""Plain 64-bit forms of the gated feed-forward block, the 4-bit matrix-vector product and the Newton-Schulz steps, and
the bounds that the kernels are held to. Everything works on torch float64 tensors of any device."""
import math

import torch

BF16, E4M3, E5M2 = 2.0 ** -8, 2.0 ** -4, 2.0 ** -3           # half a step, relative
SUBNORMAL = {torch.float8_e4m3fn: 2.0 ** -10, torch.float8_e5m2: 2.0 ** -17}   # half a step below the normal range
HALF = {torch.float8_e4m3fn: E4M3, torch.float8_e5m2: E5M2}
TOP = {torch.float8_e4m3fn: 448.0, torch.float8_e5m2: 57344.0}
ACCUMULATE = 1e-5                                            # of sum |a b|: FP32 accumulation on the tensor cores
C = math.sqrt(2 / math.pi)


def gate(g, act):
    """w(g), w'(g) of act(g) = g * sigmoid(w)."""
    if act == "silu":
        return g, torch.ones_like(g)
    return 2 * C * (g + 0.044715 * g ** 3), 2 * C * (1 + 3 * 0.044715 * g * g)


def act_of(g, act):
    return g * torch.sigmoid(gate(g, act)[0])


def slope_of(g, act):
    w, dw = gate(g, act)
    s = torch.sigmoid(w)
    return s + g * s * (1 - s) * dw


def sigmoid_error(g, act):
    """Relative error of the kernel's sigmoid s = 1 / (1 + 2^(-w log2 e)): the power is good to 2 ulp, its argument's roundings
    and w's own four move it by less than 5.2 |w| ulp, and of both 1 - s arrives in s; the sum and the reciprocal add 3 ulp."""
    w = gate(g, act)[0]
    return ((2 + 5.2 * w.abs()) * torch.sigmoid(-w) + 6) * 2.0 ** -23


def gated(a, b, unit, act):
    """G, U, h in 64 bits and what the kernel's values may be off before they are rounded; b: [2N, K]."""
    gu, mass = (a @ b.T) * unit, (a.abs() @ b.abs().T) * unit
    n = b.shape[0] // 2
    off = ACCUMULATE * mass + 2.0 ** -22 * gu.abs()          # alpha's and the product's rounding
    g, u, og, ou = gu[:, :n], gu[:, n:], off[:, :n], off[:, n:]
    v = act_of(g, act)
    h = v * u
    oh = 1.2 * og * (u.abs() + ou) + v.abs() * ou + h.abs() * (sigmoid_error(g, act) + 2.0 ** -22) + 1e-37
    return gu, off, h, oh


def gated_backward(a, b, unit, gu, act):
    """[dG | dU] in 64 bits and their error before rounding; b: [N, K]."""
    dh, mass = (a @ b.T) * unit, (a.abs() @ b.abs().T) * unit
    n = b.shape[0]
    g, u = gu[:, :n], gu[:, n:]
    off = ACCUMULATE * mass + 2.0 ** -22 * dh.abs()
    v, d = act_of(g, act), slope_of(g, act)
    w, dw = gate(g, act)
    s = torch.sigmoid(w)
    # the slope's two terms may cancel, so their errors are of the terms; 1 - s is off by s's error and a rounding
    e = sigmoid_error(g, act) + 2.0 ** -21
    od = e * (s + 2 * (g * s * (1 - s) * dw).abs()) + (g * s * dw).abs() * (s * e + 2.0 ** -24)
    out = torch.cat((dh * u * d, dh * v), 1)
    err = torch.cat((u.abs() * (off * (d.abs() + od) + dh.abs() * od), off * v.abs() + dh.abs() * v.abs() * e), 1)
    return out, err + out.abs() * 2.0 ** -21 + 1e-37


def within(got, want, off, half):
    """got is `want` moved by at most `off` and rounded (relative half step)."""
    got = got.double()
    return bool(((got - want).abs() <= off + half * (want.abs() + off)).all())


def codes_within(got, want, off, scale, kind):
    """got: codes of a value within `off` of `want`, under scale, saturated."""
    top = TOP[kind]
    v, o = (want * scale), off * scale + 2.0 ** -23 * (want * scale).abs()
    v = v.clamp(-top, top)
    err = (got.view(kind).double() - v).abs()
    return bool((err <= o + HALF[kind] * (v.abs() + o) + SUBNORMAL[kind]).all())


NS = (3.4445, -4.7750, 2.0315)


def newton_schulz(x, steps=5, fp16=False):
    """Newton-Schulz in 64 bits; with fp16 X, A and B are rounded to FP16 under a factor of 1024 where the kernel does."""
    def r(v):
        return (v * 1024).to(torch.float16).to(v.dtype) / 1024 if fp16 else v
    a, b, c = NS
    norm = x.square().sum().sqrt()
    tall = x.shape[0] > x.shape[1]
    x = r((x.T if tall else x) / (norm if norm > 0 else 1.0))
    eye = torch.eye(x.shape[0], dtype=x.dtype, device=x.device)
    for _ in range(steps):
        g = r(x @ x.T)
        x = r(r(a * eye + b * g + c * (g @ g)) @ x)
    return x.T if tall else x


def orth_bounds(x, steps=5):
    """The exact factor, and how far a result may be from it: (2-norm of the difference, largest element). The kernel's
    roundings to FP16 are those of the 64-bit form above at the same places, but fall otherwise where its FP32 sums differ
    by an ulp, so its error is another draw of the same size: four times that draw's, in norm and by element."""
    want = newton_schulz(x, steps)
    d = newton_schulz(x, steps, fp16=True) - want
    rms = d.square().mean().sqrt()
    floor = 2.0 ** -11 * want.square().mean().sqrt()          # one rounding of X, where the draw happens to be smaller
    return want, 4 * (d.norm() + floor * math.sqrt(x.numel())), 4 * (d.abs().max() + 4 * rms + 4 * floor)


def fp4_values(q, sf, rows, k, nv):
    """What 4-bit codes and their scale atoms stand for."""
    table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64, device=q.device)
    v = table[torch.stack((q & 15, q >> 4), -1).reshape(rows, -1).int()]
    block, per = (16, 4) if nv else (32, 2)
    n = k // block
    R, N = -(-rows // 128) * 128, -(-n // (4 * per)) * 4 * per
    s = sf.reshape(R // 128, N // 4, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(R, N)[:rows, :n].contiguous()
    if nv:
        s = s.view(torch.float8_e4m3fn).double()
    else:
        s = torch.where(s == 255, torch.full((), math.nan, dtype=torch.float64, device=s.device), torch.exp2(s.double() - 127))
    return (v.reshape(rows, n, block) * s[..., None]).reshape(rows, k)


def atoms(codes, nv):
    """Scale codes [rows, n] (uint8) as atoms, K padded to 256 values with zero bytes."""
    rows, n = codes.shape
    per = 4 if nv else 2
    R, N = -(-rows // 128) * 128, -(-n // (4 * per)) * 4 * per
    out = torch.zeros(R, N, dtype=torch.uint8, device=codes.device)
    out[:rows, :n] = codes
    return out.reshape(R // 128, 4, 32, N // 4, 4).permute(0, 3, 2, 1, 4).contiguous().reshape(-1)


def guarded(rows, cols, dtype, device="cuda"):
    """A [rows, cols] view with 64 untouched elements before and after it, and the check that they are untouched."""
    size = torch.empty((), dtype=dtype).element_size()
    whole = torch.full(((rows * cols + 128) * size,), 0x5A, dtype=torch.uint8, device=device)
    view = whole.view(dtype)[64:64 + rows * cols].view(rows, cols)

    def check():
        assert bool((whole[:64 * size] == 0x5A).all()) and bool((whole[(rows * cols + 64) * size:] == 0x5A).all())
    return view, check
