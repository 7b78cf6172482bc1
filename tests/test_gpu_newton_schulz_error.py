"""How far the Newton-Schulz calls are from the exact factor, on spectra that fall as gradients' do: no further than the
documented roundings (X, A and B to FP16, the result to BF16) put them, in both forms of the kernel."""
import pytest
import torch

from tests import _newton_schulz as ns

pytestmark = pytest.mark.gpu
# held by one CTA pair (up to 256 a side), and grid-wide
SIZES = [(200, 256), (256, 200), (256, 256), (64, 250), (300, 520), (520, 300), (600, 640)]


def error(fp8, x):
    out = torch.empty(x.shape, dtype=torch.bfloat16, device="cuda")
    fp8.muon_orthogonalize([x], [out])
    fp8.fp8t_check_device_error()
    return out


@pytest.mark.parametrize("power", [0, 0.5, 1, 1.5, 2])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_error_is_that_of_its_roundings(cuda_lib, rows, cols, power):
    """The kernel's roundings are the same as those of the 64-bit form, at the same places, but some fall otherwise where the FP32
    sums differ by an ulp. Both errors are sums of more than 3 s^2 of them a step (12 thousand and more here), so their norms
    differ by a percent or two where all are independent; a quarter leaves room for what the few strong directions share."""
    x = ns.falling(rows, cols, power, rows + cols, "cuda").float()
    want, norm = ns.same_roundings(x.double())
    assert float((error(cuda_lib, x).double() - want).norm()) <= 1.25 * float(norm)


@pytest.mark.parametrize("power", [1, 2, 3])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_error_by_the_formula(cuda_lib, rows, cols, power):
    """The same without any emulation of roundings: their expected size, carried through the steps, and the result's to BF16."""
    x = ns.falling(rows, cols, power, rows * cols, "cuda").float()
    want, _ = ns.same_roundings(x.double())
    off = (error(cuda_lib, x).double() - want).norm()
    assert float(off) <= float(ns.rounding_error(x.double())) + 2.0 ** -8 * float(want.norm())
