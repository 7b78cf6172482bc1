"""The plain forms that the kernels are held to: the gate's gradient against differences, the FP16 Newton-Schulz steps
against the exact ones, and that a planted mistake fails the bounds."""
import pytest
import torch

from tests import _feed_forward as ff


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_activation_and_its_slope(act):
    g = torch.linspace(-12, 12, 4001, dtype=torch.float64)
    want = torch.nn.functional.silu(g) if act == "silu" else torch.nn.functional.gelu(g, approximate="tanh")
    assert torch.allclose(ff.act_of(g, act), want, atol=1e-14, rtol=1e-13)
    e = 1e-5
    diff = (ff.act_of(g + e, act) - ff.act_of(g - e, act)) / (2 * e)
    assert torch.allclose(ff.slope_of(g, act), diff, atol=1e-9)


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gradient_against_differences(act):
    gen = torch.Generator().manual_seed(1)
    M, N, K = 3, 4, 5
    dy, wd = (torch.randn(s, generator=gen, dtype=torch.float64) for s in ((M, K), (N, K)))
    gu = torch.randn(M, 2 * N, generator=gen, dtype=torch.float64)

    def loss(v):
        return ((ff.act_of(v[:, :N], act) * v[:, N:]) * (dy @ wd.T)).sum()
    got, _ = ff.gated_backward(dy, wd, 1.0, gu, act)
    for i in range(M):
        for j in range(2 * N):
            p, m = gu.clone(), gu.clone()
            p[i, j] += 1e-6
            m[i, j] -= 1e-6
            assert abs((loss(p) - loss(m)) / 2e-6 - got[i, j]) < 1e-7


@pytest.mark.parametrize("rows,cols", [(40, 40), (17, 60), (60, 17), (1, 5)])
def test_newton_schulz_reaches_the_band(rows, cols):
    gen = torch.Generator().manual_seed(rows)
    x = torch.randn(rows, cols, generator=gen, dtype=torch.float64)
    u, s, vh = torch.linalg.svd(x, full_matrices=False)
    y, norm, most = ff.orth_bounds(x, 10)
    # the same singular vectors, and the values in the polynomial's band
    d = u.T @ y @ vh.T
    assert (d - torch.diag(torch.diagonal(d))).abs().max() < 1e-10
    assert 0.65 < float(torch.diagonal(d).min()) and float(torch.diagonal(d).max()) < 1.25
    assert float(norm) < 0.05 * float(y.norm()) and float(most) < 0.2


def test_bounds_see_a_wrong_coefficient():
    gen = torch.Generator().manual_seed(3)
    x = torch.randn(48, 64, generator=gen, dtype=torch.float64)
    want, norm, most = ff.orth_bounds(x)
    keep = ff.NS
    try:
        ff.NS = (3.4445, -4.7750, 2.05)
        wrong = ff.newton_schulz(x)
    finally:
        ff.NS = keep
    assert (wrong - want).norm() > norm


def test_fp4_atoms_round_trip():
    gen = torch.Generator().manual_seed(4)
    for nv, k in ((True, 288), (False, 288), (False, 32)):
        rows = 130
        codes = torch.randint(100, 120, (rows, k // (16 if nv else 32)), generator=gen, dtype=torch.uint8)
        q = torch.full((rows, k // 2), 0x22, dtype=torch.uint8)                # every value 1
        v = ff.fp4_values(q, ff.atoms(codes, nv), rows, k, nv)
        s = codes.view(torch.float8_e4m3fn).double() if nv else torch.exp2(codes.double() - 127)
        assert torch.equal(v.reshape(rows, codes.shape[1], -1)[..., 0], s)
