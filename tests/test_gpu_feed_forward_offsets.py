"""Weights, activations and outputs of more than 2^31 bytes or elements: what lies behind that is read and written where it is."""
import pytest
import torch

from tests import _feed_forward as ff
from tests.test_gpu_gated import E4, codes, scalar, value

pytestmark = pytest.mark.gpu


def clean(big):
    """Random FP8 codes without NaN in place."""
    return big.random_(0, 0x78).bitwise_or_((torch.arange(big.shape[-1], device="cuda") % 3 == 0).to(torch.uint8) * 0x80)


@pytest.mark.parametrize("b_mn", [False, True])
@pytest.mark.parametrize("M", [3, 40])
def test_gated_weights(cuda_lib, M, b_mn):
    """2N x K = 2.3 10^9 codes; the last outputs against the formula."""
    K, N, tail = 8192, 140016, 96
    w = torch.empty((K, 2 * N) if b_mn else (2 * N, K), dtype=torch.uint8, device="cuda")
    for part in w.split(1024):
        clean(part)
    a = codes((M, K), E4, 1)
    h, inv = torch.empty(M, N, dtype=torch.bfloat16, device="cuda"), scalar(2.0 ** -9)
    cuda_lib.fp8_gated_gemm(a, 0, w, 0, inv, inv, b_mn=b_mn, h=h)
    cuda_lib.fp8t_check_device_error()
    rows = torch.cat((torch.arange(N - tail, N), torch.arange(2 * N - tail, 2 * N))).cuda()
    part = w[:, rows].T if b_mn else w[rows]
    _, _, want, off = ff.gated(value(a, E4), value(part.contiguous(), E4), 2.0 ** -18, "silu")
    assert ff.within(h[:, -tail:], want, off, ff.BF16)


def test_gated_rows(cuda_lib):
    """[G | U] and its gradient of 2.2 10^9 elements, codes of 1.1 10^9: the last rows."""
    M, K, N, tail = 70003, 16, 15664, 200
    a, w, inv = codes((M, K), E4, 1), codes((2 * N, K), E4, 2), scalar(0.25)
    gu = torch.empty(M, 2 * N, dtype=torch.bfloat16, device="cuda")
    o = dict(q=torch.empty(M, N, dtype=torch.uint8, device="cuda"), scale=scalar(16.0), scale_inv=scalar(0), amax=scalar(0))
    cuda_lib.fp8_gated_gemm(a, 0, w, 0, inv, inv, gu=gu, **o)
    cuda_lib.fp8t_check_device_error()
    want = ff.gated(value(a[-tail:], E4), value(w, E4), 0.0625, "silu")
    assert ff.within(gu[-tail:], want[0], want[1], ff.BF16) and ff.codes_within(o["q"][-tail:], want[2], want[3], 16.0, E4)
    kept = gu[-tail:].double()
    cuda_lib.fp8_gated_gemm_backward(a, 0, w[:N], 0, inv, inv, gu, dgu=gu)
    cuda_lib.fp8t_check_device_error()
    d, off = ff.gated_backward(value(a[-tail:], E4), value(w[:N], E4), 0.0625, kept, "silu")
    assert ff.within(gu[-tail:], d, off, ff.BF16)


@pytest.mark.parametrize("nv", [False, True])
def test_matvec_weights(cuda_lib, nv):
    """4.3 10^9 weights, 2.1 10^9 bytes of codes: the last outputs, and the up rows of a gated product."""
    K, N, tail = 8192, 262152, 136
    q = torch.empty(2 * N, K // 2, dtype=torch.uint8, device="cuda")
    for part in q.split(8192):
        part.random_(0, 256)
    n = cuda_lib.fp4_scale_bytes(2 * N, K, 4 if nv else 3)
    sf = torch.empty(n, dtype=torch.uint8, device="cuda").random_(*((0x30, 0x40) if nv else (120, 126)))
    x = torch.randn(2, K, device="cuda").to(torch.bfloat16)
    y = torch.empty(2, N, dtype=torch.bfloat16, device="cuda")
    inv = scalar(2.0 ** -6)
    cuda_lib.fp4_matvec(x, q, sf, 4 if nv else 3, y, w_scale_inv=inv, act=1)
    torch.cuda.synchronize()
    # the tail's rows with the scales of their own row blocks
    block = n // ((2 * N + 127) // 128)
    part = []
    for last in (N, 2 * N):
        first = (last - tail) // 128
        rows = last - first * 128
        v = ff.fp4_values(q[first * 128:last], sf[first * block:(first + (rows + 127) // 128) * block], rows, K, nv)
        part.append(v[-tail:])
    _, _, want, off = ff.gated(x.double(), torch.cat(part), 2.0 ** -6, "silu")
    assert ff.within(y[:, -tail:], want, off, ff.BF16)
