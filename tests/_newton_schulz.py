"""Matrices of a given spectrum, and two measures of how far Newton-Schulz steps in FP16 may be from exact ones. Both work on
float64 tensors of any device."""
import math

import torch

from tests import _feed_forward as ff

# Root mean square of an FP16 rounding relative to the value: the error is uniform within half a step, at most 2^-11 of the value
# 1 and 2^-12 of the value 2; over a binade, its values spread over their logarithm, that is 2^-11 sqrt(1 / 3) sqrt(3 / (8 ln 2)).
RHO = 2.0 ** -11 * math.sqrt(1 / 3) * math.sqrt(3 / (8 * math.log(2)))
# a = 3.4445 under 2^10 lies in [2048, 4096), where a step is 2: the diagonal of B is off by at most this, alike in every row
DIAGONAL = 1.0 / (1024 * ff.NS[0])


def falling(rows, cols, power, seed, device):
    """Singular values k^-power (k = 1 ..), random singular vectors."""
    gen = torch.Generator(device=device).manual_seed(seed)
    s = min(rows, cols)
    q = [torch.linalg.qr(torch.randn(n, s, generator=gen, device=device, dtype=torch.float64))[0] for n in (rows, cols)]
    return (q[0] * torch.arange(1, s + 1, device=device, dtype=torch.float64) ** -power) @ q[1].T


def same_roundings(x, steps=5):
    """The exact factor and the error, in norm, of the 64-bit form that rounds where the kernels do (X, A, B to FP16, the result to
    BF16)."""
    want, draw = ff.newton_schulz(x, steps), ff.newton_schulz(x, steps, fp16=True)
    return want, (draw.to(torch.bfloat16).double() - want).norm()


def rounding_error(x, steps=5):
    """The expected norm of the error from the roundings alone, each independent of the others, by the formula and not by rounding
    anything: what a step's roundings of A, B and X add up to in the step's result, and what the steps after it make of that. A
    step moves an error by at most a = 3.4445, its slope at zero (the directions that are still small, which is where nearly all
    of a noise lies; those that are there already move by less)."""
    a, b, c = ff.NS
    x = x.T if x.shape[0] > x.shape[1] else x
    x = x / x.norm()
    noise, alike = RHO * x.norm(), torch.zeros((), dtype=x.dtype, device=x.device)
    for _ in range(steps):
        g = x @ x.T
        y = b * g + c * (g @ g)                             # B but for a I
        top = torch.linalg.matrix_norm(g, 2)
        of_a = (abs(b) + 2 * c * top) * ((g * g) @ (x * x)).sum().sqrt()
        of_b = ((y * y) @ (x * x)).sum().sqrt()
        after = a * x + y @ x
        noise = ((a * noise) ** 2 + RHO ** 2 * (of_a ** 2 + of_b ** 2 + after.norm() ** 2)).sqrt()
        alike = a * alike + DIAGONAL * a * x.norm()
        x = after
    return noise + alike
