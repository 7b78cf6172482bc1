"""A gated feed-forward block as it is used: trained for a step in FP8 (norm, gated product, down projection, gradient,
Muon) and then served in 4 bits for a few tokens, each part against 64 bits from its actual inputs."""
import pytest
import torch

from tests import _feed_forward as ff
from tests.test_gpu_muon import check_step

pytestmark = pytest.mark.gpu
E4, E5 = torch.float8_e4m3fn, torch.float8_e5m2


def one(v=0.0):
    return torch.full((1,), v, device="cuda")


def cast(fp8, x, kind):
    """Codes under the scale of x's own amax, and the inverse scale."""
    q, inv, amax = torch.empty(x.shape, dtype=torch.uint8, device="cuda"), one(), one()
    scale = ff.TOP[kind] / x.float().abs().amax().reshape(1)
    fp8.fp8_cast_transpose_amax(x, 0 if kind == E4 else 1, scale, q, None, amax, inv)
    return q, inv


def product(fp8, A, af, ai, B, bf, bi, M, N, a_mn=False, b_mn=False):
    D = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    fp8.fp8_gemm_multi([dict(A=A, a_fmt=af, B=B, b_fmt=bf, a_scale_inv=ai, b_scale_inv=bi, D=D, a_mn=a_mn, b_mn=b_mn)])
    return D


def val(q, inv, kind):
    return q.view(kind).double() * inv.double()


def close(got, a, b):
    """One FP8 product (within 2 BF16 steps and the accumulation)."""
    want = a @ b
    return ff.within(got, want, ff.ACCUMULATE * (a.abs() @ b.abs()), 4 * ff.BF16)


def test_block(cuda_lib):
    fp8 = cuda_lib
    T, D, F = 304, 256, 704
    gen = torch.Generator(device="cuda").manual_seed(0)
    rnd = lambda r, c, s: (torch.randn(r, c, generator=gen, device="cuda") * s)  # noqa: E731
    x, gamma = rnd(T, D, 1).to(torch.bfloat16), torch.ones(D, dtype=torch.bfloat16, device="cuda")
    pw, pd = rnd(D, 2 * F, 0.06), rnd(F, D, 0.04)
    w, wd = pw.to(torch.bfloat16), pd.to(torch.bfloat16)
    # forward: norm to FP8, both projections with the gate to FP8, down projection
    xq, xi, amax, rstd = torch.empty(T, D, dtype=torch.uint8, device="cuda"), one(), one(), torch.empty(T, device="cuda")
    fp8.fp8_rmsnorm_cast(x, gamma, 1e-5, rstd=rstd, quant=fp8.Q_FP8, q=xq, scale=one(90.0), amax=amax, scale_inv=xi)
    wq, wi = cast(fp8, w, E4)
    gu = torch.empty(T, 2 * F, dtype=torch.bfloat16, device="cuda")
    hq, hi, hmax = torch.empty(T, F, dtype=torch.uint8, device="cuda"), one(), one()
    fp8.fp8_gated_gemm(xq, 0, wq, 0, xi, wi, b_mn=True, gu=gu, q=hq, scale=one(40.0), amax=hmax, scale_inv=hi)
    unit = float(xi * wi)
    _, _, h, oh = ff.gated(xq.view(E4).double(), wq.view(E4).double().T, unit, "silu")
    assert ff.codes_within(hq, h, oh, 40.0, E4)
    wdq, wdi = cast(fp8, wd, E4)
    y = product(fp8, hq, 0, hi, wdq, 0, wdi, T, D, b_mn=True)
    assert close(y, val(hq, hi, E4), val(wdq, wdi, E4))
    # backward: the gate's gradient in the down projection's dgrad, then one product each for dX and dW
    dy = rnd(T, D, 1e-3).to(torch.bfloat16)
    dyq, dyi = cast(fp8, dy, E5)
    dq, di, dmax = torch.empty(T, 2 * F, dtype=torch.uint8, device="cuda"), one(), one()
    fp8.fp8_gated_gemm_backward(dyq, 1, wdq, 0, dyi, wdi, gu, q=dq, scale=one(4e6), amax=dmax, scale_inv=di)
    d, od = ff.gated_backward(dyq.view(E5).double(), wdq.view(E4).double(), float(dyi * wdi), gu.double(), "silu")
    assert ff.codes_within(dq, d, od, 4e6, E5)
    dx = product(fp8, dq, 1, di, wq, 0, wi, T, D)
    assert close(dx, val(dq, di, E5), val(wq, wi, E4).T)
    dw = product(fp8, xq, 0, xi, dq, 1, di, D, 2 * F, a_mn=True, b_mn=True)
    dwd = product(fp8, hq, 0, hi, dyq, 1, dyi, F, D, a_mn=True, b_mn=True)
    assert close(dw, val(xq, xi, E4).T, val(dq, di, E5)) and close(dwd, val(hq, hi, E4).T, val(dyq, dyi, E5))
    # the whole gradient is that of the unquantised block but for FP8's roundings
    xd = (x.double() * rstd.double()[:, None])
    w64, wd64 = w.double().requires_grad_(), wd.double().requires_grad_()
    g, u = (xd @ w64).chunk(2, 1)
    (((ff.act_of(g, "silu") * u) @ wd64) * dy.double()).sum().backward()
    for got, want in ((dw, w64.grad), (dwd, wd64.grad)):
        assert float((got.double() - want).norm() / want.norm()) < 0.2
    # Muon over both matrices
    s = dict(p=[pw, pd], m=[torch.zeros_like(pw), torch.zeros_like(pd)], g=[dw, dwd], w=[w, wd])
    old = {k: [t.clone() for t in v] for k, v in s.items()}
    fp8.fused_muon_multi_tensor(s["p"], s["m"], s["g"], s["w"], lr=0.01, beta=0.95, weight_decay=0.0)
    check_step(s, old, lr=0.01, beta=0.95, wd=0.0, S=1.0)
    # serving: the new weights in 4 bits, a few tokens through gate, up and down
    tokens = x[:3].contiguous()
    for quant, nv in ((fp8.Q_MXFP4, False), (fp8.Q_NVFP4, True)):
        held = []
        for m in (w, wd):
            q = torch.empty(m.shape[1], m.shape[0] // 2, dtype=torch.uint8, device="cuda")
            sf = torch.empty(fp8.fp4_scale_bytes(m.shape[1], m.shape[0], quant), dtype=torch.uint8, device="cuda")
            inv = one() if nv else None
            extra = dict(scale=2688.0 / m.float().abs().amax().reshape(1), scale_inv=inv) if nv else {}
            fp8.fp4_cast_multi([dict(x=m, quant=quant, q_col=q, sf_col=sf, **extra)])
            held.append((q, sf, inv))
        q, sf, inv = held[0]
        out = torch.empty(3, F, dtype=torch.bfloat16, device="cuda")
        fp8.fp4_matvec(tokens, q, sf, quant, out, w_scale_inv=inv, act=fp8.ACT_SILU)
        v = ff.fp4_values(q, sf, 2 * F, D, nv)
        _, _, want, off = ff.gated(tokens.double(), v, float(inv) if nv else 1.0, "silu")
        assert ff.within(out, want, off, ff.BF16)
        q, sf, inv = held[1]
        last = torch.empty(3, D, dtype=torch.bfloat16, device="cuda")
        fp8.fp4_matvec(out, q, sf, quant, last, w_scale_inv=inv)
        v = ff.fp4_values(q, sf, D, F, nv) * (inv.double() if nv else 1.0)
        assert ff.within(last, out.double() @ v.T, ff.ACCUMULATE * (out.double().abs() @ v.abs().T), ff.BF16)
    fp8.fp8t_check_device_error()
