"""The two measures of tests/_newton_schulz.py against one another."""
import pytest
import torch

from tests import _feed_forward as ff
from tests import _newton_schulz as ns


def rounded(x, dtype):
    """Steps whose X, A and B are rounded to a type; 64 bits otherwise."""
    a, b, c = ff.NS
    r = lambda v: v.to(dtype).double()  # noqa: E731
    x = r(x / x.norm())
    for _ in range(5):
        g = r(x @ x.T)
        x = r(r(a * torch.eye(len(x), dtype=x.dtype) + b * g + c * (g @ g)) @ x)
    return x


@pytest.mark.parametrize("rows,cols", [(48, 48), (128, 200), (200, 128)])
@pytest.mark.parametrize("power", [0.5, 1, 1.5, 2, 3])
def test_expected_error_covers_rounded_steps(rows, cols, power):
    x = ns.falling(rows, cols, power, 1, "cpu")
    assert (ff.newton_schulz(x, fp16=True) - ff.newton_schulz(x)).norm() <= ns.rounding_error(x)


@pytest.mark.parametrize("power", [2, 3])
def test_expected_error_sees_three_bits_fewer(power):
    """Planted: BF16 in the place of FP16, where the noise of X0 decides."""
    x = ns.falling(64, 96, power, 1, "cpu")
    want = ff.newton_schulz(x)
    assert (rounded(x, torch.float32) - want).norm() < 1e-3 < ns.rounding_error(x) < (rounded(x, torch.bfloat16) - want).norm()


def test_rounding_of_fp16():
    """RHO is the root mean square over values spread over their logarithm."""
    v = torch.exp2(torch.linspace(0, 4, 100001, dtype=torch.float64)[:-1])
    rms = ((v.to(torch.float16).double() - v) / v).square().mean().sqrt()
    assert abs(float(rms) / ns.RHO - 1) < 0.01


def test_spectrum():
    s = torch.linalg.svdvals(ns.falling(20, 30, 1.5, 2, "cpu"))
    assert torch.allclose(s, torch.arange(1, 21, dtype=torch.float64) ** -1.5)
