"""The quantising RMSNorm and its backward pass through the C ABI against the 64-bit formulas.

Bounds (u = 2^-24, half an f32 step): a row's sum of squares is a chain of at most 32 fused multiply-adds in
a thread and at most 10 additions over the threads, so it is off by at most 42 u of itself, its mean by
43 u, rstd by half of that and three roundings more, y by two more: 27 u. D = 2^-19 = 32 u covers all of them.
A code is checked against what the exact encoder gives for the value and its scale moved by D either way
(encoding is monotone), so a code may differ from the exact one only where rounding is that close."""
import numpy as np
import pytest
import torch

from tests import _block_quant as bq
from tests._gpu import bf16_bits, bf16_from_bits, u8
from tests._pins import gemm_within_tolerance

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
D = 2.0 ** -19
FP8, MXFP8, MXFP4, NVFP4 = 1, 2, 3, 4


def bf(a):
    return bf16_bits(torch.from_numpy(np.asarray(a, np.float32)).to(torch.bfloat16))


def make(rows, cols, seed, scale=1.0):
    """BF16 patterns of x, residual (with a few large columns) and gamma."""
    rng = np.random.default_rng(seed)
    x, r = rng.standard_normal((rows, cols)) * scale, rng.standard_normal((rows, cols)) * scale
    r[:, rng.integers(0, cols, 3)] *= 100
    return bf(x), bf(r), bf(1 + 0.2 * rng.standard_normal(cols))


def guarded(rows, cols, dtype):
    """A [rows, cols] view with untouched rows around it, and the check that they are untouched."""
    whole = torch.full(((rows + 2) * cols,), 0x5A, dtype=torch.uint8, device="cuda").repeat_interleave(
        torch.empty((), dtype=dtype).element_size()).view(dtype).reshape(rows + 2, cols)
    keep = whole.clone().view(torch.uint8)

    def check():
        now = whole.view(torch.uint8)
        assert torch.equal(now[0], keep[0]) and torch.equal(now[-1], keep[-1])
    return whole[1:rows + 1], check


def run(fp8, x, res, gamma, eps, quant, fmt=0, scale=1.0, want_y=False, want_rstd=True):
    rows, cols = x.shape
    o = dict(rstd=torch.empty(rows, dtype=torch.float32, device="cuda") if want_rstd else None)
    checks = []
    if res is not None:
        o["h"], c = guarded(rows, cols, torch.bfloat16)
        checks.append(c)
    if want_y or quant == 0:
        o["y"], c = guarded(rows, cols, torch.bfloat16)
        checks.append(c)
    kw = {}
    if quant:
        o["q"], c = guarded(rows, cols // 2 if quant in (MXFP4, NVFP4) else cols, torch.uint8)
        checks.append(c)
        if quant in (FP8, NVFP4):
            o["scale"] = torch.tensor([scale], dtype=torch.float32, device="cuda")
            o["amax"], o["scale_inv"] = torch.zeros(1, device="cuda"), torch.zeros(1, device="cuda")
        if quant != FP8:
            n = fp8.fp4_scale_bytes(rows, cols, quant) if quant != MXFP8 else -(-rows // 128) * -(-cols // 128) * 512
            o["sf"] = torch.full((n,), 0xEE, dtype=torch.uint8, device="cuda")
        kw = dict(quant=quant, fmt=fmt, **{k: o[k] for k in ("q", "sf", "scale", "amax", "scale_inv") if k in o})
    fp8.fp8_rmsnorm_cast(bf16_from_bits(x), bf16_from_bits(gamma), eps,
                         residual=None if res is None else bf16_from_bits(res), h=o.get("h"), rstd=o["rstd"],
                         y=o.get("y"), **kw)
    torch.cuda.synchronize()
    for c in checks:
        c()
    return o


def signed_encode(v, d, values, bit):
    """The codes of v moved by the relative d either way, as signed numbers (monotone in v)."""
    lo, hi = bq.encode(np.abs(v) * (1 - d), values, bit), bq.encode(np.abs(v) * (1 + d), values, bit)
    return lo, hi


def check(o, x, res, gamma, eps, quant, fmt=0, scale=1.0):
    rows, cols = x.shape
    h, rstd, y = bq.rmsnorm(bq.bf16_f64(x), None if res is None else bq.bf16_f64(res), bq.bf16_f64(gamma), eps)
    if res is not None:
        assert np.array_equal(bq.bf16_f64(bf16_bits(o["h"])), h)
    if o["rstd"] is not None:
        assert (np.abs(o["rstd"].cpu().numpy() - rstd) <= D * rstd).all()
    if "y" in o:
        assert (np.abs(bq.bf16_f64(bf16_bits(o["y"])) - y) <= np.abs(y) * (2.0 ** -8 + D)).all()
    if not quant:
        return
    q = u8(o["q"])
    if quant in (FP8, NVFP4):
        top = np.abs(y).max()
        assert abs(o["amax"].item() - top) <= D * top
        assert o["scale_inv"].item() == np.float32(1) / np.float32(scale)
    if quant == FP8:
        vals = bq.E4M3 if fmt == 0 else bq.E5M2
        lo, hi = signed_encode(y * np.float64(np.float32(scale)), D, vals, 128)
        mag = q & 0x7F
        assert ((lo <= mag) & (mag <= hi)).all()
        assert ((np.signbit(y) == (q >= 128)) | (mag == 0)).all()
        return
    B = 16 if quant == NVFP4 else 32
    sf, pad = bq.from_atoms(u8(o["sf"]), rows, cols // B, quant)
    assert not pad.any()                              # K's padding
    blocks = y.reshape(rows, cols // B, B)
    amax = np.abs(blocks).max(-1)
    g = np.float64(np.float32(scale))
    if quant == NVFP4:
        lo, hi = signed_encode(amax * g / 6, D, bq.E4M3, 128)
        s = bq.E4M3[sf]
        v = np.where(s[..., None] > 0, blocks * g / np.where(s > 0, s, 1)[..., None], 0)
    else:
        emax = 2 if quant == MXFP4 else 8 if fmt == 0 else 15
        lo, hi = (bq.e8m0_exponent(amax * f, emax) + 127 for f in (1 - D, 1 + D))
        v = blocks * np.exp2(127.0 - sf.astype(np.float64))[..., None]
    assert ((lo <= sf) & (sf <= hi)).all()
    if quant == MXFP8:
        vals, bit, codes = (bq.E4M3 if fmt == 0 else bq.E5M2), 128, q
    else:
        vals, bit, codes = bq.E2M1, 8, bq.unpack(q)
    lo, hi = signed_encode(v.reshape(rows, cols), 2 * D, vals, bit)      # the scale's own rounding too
    mag = codes & (bit - 1)
    assert ((lo <= mag) & (mag <= hi)).all()
    assert ((np.signbit(y) == (codes >= bit)) | (mag == 0)).all()


@pytest.mark.parametrize("quant,fmt,scale", [(0, 0, 1.0), (FP8, 0, 20.0), (FP8, 1, 300.0), (MXFP8, 0, 1.0), (MXFP8, 1, 1.0),
                                             (MXFP4, 0, 1.0), (NVFP4, 0, 130.0)])
@pytest.mark.parametrize("rows,cols,residual", [(1, 32, True), (5, 64, False), (130, 96, True), (3, 1024, True),
                                                (700, 1056, False), (1, 4096, True), (257, 4096, True), (2, 11008, True),
                                                (200, 2080, True), (33, 16384, False), (150, 16384, True)])
def test_forward(cuda_lib, quant, fmt, scale, rows, cols, residual):
    x, r, gamma = make(rows, cols, rows * 7 + cols)
    r = r if residual else None
    o = run(cuda_lib, x, r, gamma, 1e-5, quant, fmt, scale, want_y=rows % 2 == 0)
    check(o, x, r, gamma, 1e-5, quant, fmt, scale)


@pytest.mark.parametrize("cols", [16, 48, 1040, 4112])
@pytest.mark.parametrize("quant", [0, FP8])
def test_forward_columns_that_no_block_divides(cuda_lib, cols, quant):
    x, r, gamma = make(37, cols, cols)
    o = run(cuda_lib, x, r, gamma, 1e-6, quant, 0, 15.0, want_rstd=False)
    check(o, x, r, gamma, 1e-6, quant, 0, 15.0)


@pytest.mark.parametrize("quant", [0, FP8, MXFP8, MXFP4, NVFP4])
@pytest.mark.parametrize("cols", [256, 2048])
def test_forward_special_rows(cuda_lib, quant, cols):
    """A zero row (y = 0, zero scales), tiny rows, a NaN row and an infinite one beside ordinary ones."""
    x, _, gamma = make(6, cols, 3)
    x[1] = 0
    x[2] = bf(np.full(cols, 1e-30))
    x[4, 7] = 0x7FC1                                  # NaN
    x[5, 9] = 0xFF80                                  # -infinity
    o = run(cuda_lib, x, None, gamma, 1e-5, quant, 0, 10.0, want_y=True)
    y = bq.bf16_f64(bf16_bits(o["y"]))
    assert (y[1] == 0).all() and np.isnan(y[4]).all() and np.isnan(y[5, 9])
    assert (np.delete(y[5], 9) == 0).all()            # finite / infinity
    for i in (0, 2, 3):
        want = bq.rmsnorm(bq.bf16_f64(x[i:i + 1]), None, bq.bf16_f64(gamma), 1e-5)[2]
        assert (np.abs(y[i] - want) <= np.abs(want) * (2.0 ** -8 + D)).all()
    if quant == FP8:
        assert np.isnan(o["amax"].item()) and (u8(o["q"])[4] == 0x7F).all() and u8(o["q"])[5, 9] == 0x7F
    if quant in (MXFP8, MXFP4, NVFP4):
        n = 16 if quant == NVFP4 else 32
        sf, _ = bq.from_atoms(u8(o["sf"]), 6, cols // n, quant)
        assert (sf[1] == 0).all() and (sf[4] == (0x7F if quant == NVFP4 else 0xFF)).all()
        nan_block = sf[5] == (0x7F if quant == NVFP4 else 0xFF)
        assert nan_block[9 // n] and nan_block.sum() == 1


def test_residual_may_be_overwritten(cuda_lib):
    x, r, gamma = make(300, 1024, 8)
    for target in ("x", "residual"):
        t = dict(x=bf16_from_bits(x), residual=bf16_from_bits(r))
        y = torch.empty(300, 1024, dtype=torch.bfloat16, device="cuda")
        cuda_lib.fp8_rmsnorm_cast(t["x"], bf16_from_bits(gamma), 1e-5, residual=t["residual"], h=t[target], y=y)
        h, _, want = bq.rmsnorm(bq.bf16_f64(x), bq.bf16_f64(r), bq.bf16_f64(gamma), 1e-5)
        assert np.array_equal(bq.bf16_f64(bf16_bits(t[target])), h)
        assert (np.abs(bq.bf16_f64(bf16_bits(y)) - want) <= np.abs(want) * (2.0 ** -8 + D)).all()


def test_amax_is_max_accumulated(cuda_lib):
    x, _, gamma = make(9, 64, 2)
    a = torch.full((1,), 1e6, device="cuda")
    q = torch.empty(9, 64, dtype=torch.uint8, device="cuda")
    cuda_lib.fp8_rmsnorm_cast(bf16_from_bits(x), bf16_from_bits(gamma), 1e-5, quant=FP8, q=q,
                              scale=torch.ones(1, device="cuda"), amax=a)
    assert a.item() == 1e6


# ------------------------------------------------------------------ backward
def backward(fp8, dy, h, gamma, rstd, dres, ws=None):
    rows, cols = dy.shape
    dh, c = guarded(rows, cols, torch.bfloat16)
    dgamma = torch.full((cols,), float("nan"), device="cuda")
    dgamma16 = torch.full((cols,), float("nan"), dtype=torch.bfloat16, device="cuda")
    fp8.fp8_rmsnorm_backward(bf16_from_bits(dy), bf16_from_bits(h), bf16_from_bits(gamma),
                             torch.from_numpy(rstd.astype(np.float32)).cuda(), dh,
                             dres=None if dres is None else bf16_from_bits(dres), dgamma=dgamma,
                             dgamma_bf16=dgamma16, workspace=ws)
    torch.cuda.synchronize()
    c()
    return dh, dgamma, dgamma16


@pytest.mark.parametrize("rows,cols,residual", [(1, 16, True), (1, 32, False), (3, 64, True), (130, 96, False),
                                                (512, 256, True), (601, 512, True), (77, 1024, True), (1999, 1024, False),
                                                (5, 1040, True), (2000, 4096, True), (149, 11008, True), (300, 16384, False)])
def test_backward(cuda_lib, rows, cols, residual):
    """dh: the formula's terms each rounded a few times in f32 and a row sum whose chain has at most 42
    additions: (2^-8 |dh| + 64 u (terms)). dgamma: a chain of at most rows additions per column."""
    h, r, gamma = make(rows, cols, rows + cols)
    rng = np.random.default_rng(rows)
    dy = bf(rng.standard_normal((rows, cols)) * 1e-3)
    dres = bf(rng.standard_normal((rows, cols)) * 1e-3) if residual else None
    H, G, DY = bq.bf16_f64(h), bq.bf16_f64(gamma), bq.bf16_f64(dy)
    rstd = bq.rmsnorm(H, None, G, 1e-5)[1].astype(np.float32).astype(np.float64)
    DR = None if dres is None else bq.bf16_f64(dres)
    dh, dgamma, dgamma16 = backward(cuda_lib, dy, h, gamma, rstd, dres)
    want, wantg = bq.rmsnorm_grad(DY, H, G, rstd, DR)
    xh = H * rstd[:, None]
    terms = rstd[:, None] * (np.abs(DY * G) + np.abs(xh) * np.abs(DY * G * xh).mean(1, keepdims=True))
    if DR is not None:
        terms = terms + np.abs(DR)
    got = bq.bf16_f64(bf16_bits(dh))
    assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 64 * U * terms).all()
    bound = (min(rows, 64 + rows // 148 + 592 // 16) + 8) * U * np.abs(DY * xh).sum(0)
    assert (np.abs(dgamma.cpu().numpy() - wantg) <= bound).all()
    assert torch.equal(dgamma16, dgamma.to(torch.bfloat16))


def test_backward_against_differences(cuda_lib):
    """Central differences of the 64-bit loss sum(w * y): the formula's own error is O(d^2), so what is left
    is the BF16 rounding of dh and f32 rounding of dgamma."""
    rows, cols = 4, 64
    h, _, gamma = make(rows, cols, 12)
    w = bf(np.random.default_rng(5).standard_normal((rows, cols)))
    H, G, W = bq.bf16_f64(h), bq.bf16_f64(gamma), bq.bf16_f64(w)
    rstd = bq.rmsnorm(H, None, G, 1e-3)[1]
    dh, dgamma, _ = backward(cuda_lib, w, h, gamma, rstd, None)
    got, d = bq.bf16_f64(bf16_bits(dh)), 1e-5

    def loss(H, G):
        return (bq.rmsnorm(H, None, G, 1e-3)[2] * W).sum()
    for i, j in ((0, 0), (1, 33), (3, 63)):
        e = np.zeros_like(H)
        e[i, j] = d
        diff = (loss(H + e, G) - loss(H - e, G)) / (2 * d)
        assert abs(got[i, j] - diff) <= 2.0 ** -8 * abs(diff) + 1e-6
    for j in (0, 31, 50):
        e = np.zeros(cols)
        e[j] = d
        diff = (loss(H, G + e) - loss(H, G - e)) / (2 * d)
        assert abs(dgamma[j].item() - diff) <= 1e-6 * (1 + abs(diff))


@pytest.mark.parametrize("cols", [256, 4096])
def test_backward_in_place_and_same_every_run(cuda_lib, cols):
    rows = 700
    h, _, gamma = make(rows, cols, 4)
    rng = np.random.default_rng(0)
    dy, dres = bf(rng.standard_normal((rows, cols))), bf(rng.standard_normal((rows, cols)))
    rstd = bq.rmsnorm(bq.bf16_f64(h), None, bq.bf16_f64(gamma), 1e-5)[1]
    a = backward(cuda_lib, dy, h, gamma, rstd, dres)
    b = backward(cuda_lib, dy, h, gamma, rstd, dres)
    for p, q in zip(a, b):
        assert torch.equal(p.view(torch.uint8), q.view(torch.uint8))
    for which in ("dy", "dres"):
        t = dict(dy=bf16_from_bits(dy), dres=bf16_from_bits(dres))
        cuda_lib.fp8_rmsnorm_backward(t["dy"], bf16_from_bits(h), bf16_from_bits(gamma),
                                      torch.from_numpy(rstd.astype(np.float32)).cuda(), t[which], dres=t["dres"])
        assert torch.equal(t[which].view(torch.int16), a[0].view(torch.int16))


def test_backward_without_dgamma_needs_no_workspace(cuda_lib):
    h, _, gamma = make(20, 64, 4)
    dh = torch.empty(20, 64, dtype=torch.bfloat16, device="cuda")
    t = bf16_from_bits(h)
    cuda_lib.fp8_rmsnorm_backward(t, t, bf16_from_bits(gamma), torch.ones(20, device="cuda"), dh)
    want = bq.rmsnorm_grad(bq.bf16_f64(h), bq.bf16_f64(h), bq.bf16_f64(gamma), np.ones(20))[0]
    xh = bq.bf16_f64(h)
    terms = np.abs(xh) * (1 + (xh * xh).mean(1, keepdims=True)) * 2
    assert (np.abs(bq.bf16_f64(bf16_bits(dh)) - want) <= 2.0 ** -8 * np.abs(want) + 64 * U * terms).all()


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("quant,scale", [(MXFP4, 1.0), (NVFP4, 130.0)])
@pytest.mark.parametrize("rows", [1, 16, 300])
def test_norm_feeds_the_4_bit_product(cuda_lib, quant, scale, rows):
    """Serving: the norm's codes and scales go straight into the product (captured and replayed)."""
    cols, n = 1024, 520
    x, r, gamma = make(rows, cols, rows)
    wcodes, wsf = bq.quantise(bf(np.random.default_rng(1).standard_normal((n, cols)) * 0.02), quant, 5000.0)
    B, bsf = torch.from_numpy(bq.pack(wcodes)).cuda(), torch.from_numpy(bq.atoms(wsf, quant)).cuda()
    inv_w = torch.full((1,), 1 / 5000.0 if quant == NVFP4 else 1.0, device="cuda")
    q = torch.empty(rows, cols // 2, dtype=torch.uint8, device="cuda")
    sf = torch.full((cuda_lib.fp4_scale_bytes(rows, cols, quant),), 0x7F, dtype=torch.uint8, device="cuda")
    t = dict(x=bf16_from_bits(x), r=bf16_from_bits(r), g=bf16_from_bits(gamma))
    s = torch.tensor([scale], device="cuda")
    inv = torch.ones(1, device="cuda")
    y = torch.empty(rows, n, dtype=torch.bfloat16, device="cuda")
    extra = dict(scale=s, scale_inv=inv) if quant == NVFP4 else {}

    def go():
        cuda_lib.fp8_rmsnorm_cast(t["x"], t["g"], 1e-5, residual=t["r"], quant=quant, q=q, sf=sf, **extra)
        cuda_lib.fp4_gemm_multi([dict(A=q, a_sf=sf, B=B, b_sf=bsf, quant=quant, D=y, a_scale_inv=inv, b_scale_inv=inv_w)])
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        go()
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            go()
    y.zero_()
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    cuda_lib.fp8t_check_device_error()
    blk = 16 if quant == NVFP4 else 32
    a = bq.values(bq.unpack(u8(q)), bq.from_atoms(u8(sf), rows, cols // blk, quant)[0], quant)
    b = bq.values(wcodes, wsf, quant)
    alpha = np.float64(inv.item()) * np.float64(inv_w.item())
    R = bf16_bits(torch.from_numpy((a @ b.T) * alpha).float().to(torch.bfloat16))
    assert gemm_within_tolerance(bf16_bits(y), R, (np.abs(a) @ np.abs(b).T) * alpha).all()


def test_training_chain(cuda_lib):
    """Norm (FP8 codes for fprop and wgrad) -> FP8 products -> the norm's backward pass on dX -> AdamW on
    dW and dgamma, in a captured graph on a side stream; the replay equals the eager run bit for bit."""
    from optimizer_fp8_cast_b200 import E4M3, E5M2
    T, fin, fout = 512, 256, 256
    rng = np.random.default_rng(2)
    bfc = dict(dtype=torch.bfloat16, device="cuda")
    x, r, gamma = (bf16_from_bits(v) for v in make(T, fin, 1))
    W = bf16_from_bits(bf(rng.standard_normal((fin, fout)) * 0.02))
    dY = bf16_from_bits(bf(rng.standard_normal((T, fout)) * 1e-3))
    dres = bf16_from_bits(bf(rng.standard_normal((T, fin)) * 1e-3))

    def state():
        u8_ = lambda *s: torch.zeros(*s, dtype=torch.uint8, device="cuda")  # noqa: E731
        one = lambda v=0.0: torch.full((1,), v, device="cuda")  # noqa: E731
        s = dict(h=torch.empty(T, fin, **bfc), rstd=torch.empty(T, device="cuda"), xq=u8_(T, fin), wq=u8_(fin, fout),
                 dyq=u8_(T, fout), y=torch.empty(T, fout, **bfc), dx=torch.empty(T, fin, **bfc),
                 dw=torch.empty(fin, fout, **bfc), dh=torch.empty(T, fin, **bfc), dg=torch.empty(fin, **bfc),
                 gam=gamma.clone(), W=W.clone(), ws=torch.empty(
                     cuda_lib.fp8_rmsnorm_backward_workspace_bytes(T, fin), dtype=torch.uint8, device="cuda"))
        for k, v in (("x", 20.0), ("w", 4000.0), ("dy", 1e6)):
            s["s" + k], s["a" + k], s["i" + k] = one(v), one(), one()
        s["master"] = [s["W"].float(), s["gam"].float()]
        s["m"], s["v"] = [torch.zeros_like(t) for t in s["master"]], [torch.zeros_like(t) for t in s["master"]]
        s["aws"] = torch.empty(cuda_lib.fused_adamw_workspace_bytes([fin * fout, fin]), dtype=torch.uint8, device="cuda")
        s["norm"] = one()
        return s

    def step(s):
        cuda_lib.fp8_rmsnorm_cast(x, s["gam"], 1e-5, residual=r, h=s["h"], rstd=s["rstd"], quant=FP8, q=s["xq"],
                                  scale=s["sx"], amax=s["ax"], scale_inv=s["ix"])
        cuda_lib.fp8_cast_transpose_amax_multi([
            dict(x=s["W"], fmt=E4M3, scale=s["sw"], q=s["wq"], amax=s["aw"], scale_inv=s["iw"]),
            dict(x=dY, fmt=E5M2, scale=s["sdy"], q=s["dyq"], amax=s["ady"], scale_inv=s["idy"])])
        cuda_lib.fp8_gemm_multi([
            dict(A=s["xq"], a_fmt=E4M3, B=s["wq"], b_mn=True, b_fmt=E4M3, a_scale_inv=s["ix"], b_scale_inv=s["iw"], D=s["y"]),
            dict(A=s["dyq"], a_fmt=E5M2, B=s["wq"], b_fmt=E4M3, a_scale_inv=s["idy"], b_scale_inv=s["iw"], D=s["dx"]),
            dict(A=s["xq"], a_mn=True, a_fmt=E4M3, B=s["dyq"], b_mn=True, b_fmt=E5M2, a_scale_inv=s["ix"],
                 b_scale_inv=s["idy"], D=s["dw"])])
        cuda_lib.fp8_rmsnorm_backward(s["dx"], s["h"], s["gam"], s["rstd"], s["dh"], dres=dres, dgamma_bf16=s["dg"],
                                      workspace=s["ws"])
        cuda_lib.fused_adamw_multi_tensor(s["master"], s["m"], s["v"], [s["dw"], s["dg"]], [s["W"], s["gam"]], lr=1e-3,
                                          beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0, step=1, loss_scale=1.0,
                                          max_grad_norm=1.0, grad_norm=s["norm"], workspace=s["aws"])
    eager = state()
    step(eager)
    torch.cuda.synchronize()
    s = state()
    start = {k: s[k].clone() for k in ("W", "gam")}
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            step(s)
    assert torch.equal(s["W"], start["W"])            # capturing runs nothing
    graph.replay()
    torch.cuda.synchronize()
    cuda_lib.fp8t_check_device_error()
    for k in ("h", "rstd", "xq", "y", "dx", "dw", "dh", "dg", "W", "gam", "norm"):
        assert torch.equal(s[k].view(torch.uint8), eager[k].view(torch.uint8)), k
    # the norm's gradient against the 64-bit formula on the dX that the product gave
    H, G = bq.bf16_f64(bf16_bits(s["h"])), bq.bf16_f64(bf16_bits(gamma.reshape(1, -1)))[0]
    DX, DR = bq.bf16_f64(bf16_bits(s["dx"])), bq.bf16_f64(bf16_bits(dres))
    rs = s["rstd"].cpu().numpy().astype(np.float64)
    want, wantg = bq.rmsnorm_grad(DX, H, G, rs, DR)
    xh = H * rs[:, None]
    terms = rs[:, None] * (np.abs(DX * G) + np.abs(xh) * np.abs(DX * G * xh).mean(1, keepdims=True)) + np.abs(DR)
    assert (np.abs(bq.bf16_f64(bf16_bits(s["dh"])) - want) <= 2.0 ** -8 * np.abs(want) + 64 * U * terms).all()
    dg = bq.bf16_f64(bf16_bits(s["dg"].reshape(1, -1)))[0]
    assert (np.abs(dg - wantg) <= 2.0 ** -8 * np.abs(wantg) + 128 * U * np.abs(DX * xh).sum(0)).all()


def test_two_streams_at_once(cuda_lib):
    """Two calls at the same time, each with its own buffers, give what each gives alone."""
    x, r, gamma = make(2000, 4096, 1)
    alone = run(cuda_lib, x, r, gamma, 1e-5, MXFP4)
    t = [bf16_from_bits(v) for v in (x, r, gamma)]
    outs = []
    for s in (torch.cuda.Stream(), torch.cuda.Stream()):
        s.wait_stream(torch.cuda.current_stream())
        o = dict(h=torch.empty_like(t[0]), q=torch.empty(2000, 2048, dtype=torch.uint8, device="cuda"),
                 sf=torch.full_like(alone["sf"], 0xEE))
        cuda_lib.fp8_rmsnorm_cast(t[0], t[2], 1e-5, residual=t[1], h=o["h"], quant=MXFP4, q=o["q"], sf=o["sf"], stream=s)
        outs.append(o)
    torch.cuda.synchronize()
    for o in outs:
        for k in ("h", "q", "sf"):
            assert torch.equal(o[k].view(torch.uint8), alone[k].contiguous().view(torch.uint8))
