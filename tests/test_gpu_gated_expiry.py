"""What a gated product leaves behind where its waits expired: the same in the form for few rows and in pair tiles."""
import pytest
import torch

from tests.test_gpu_gated import E4, E5, codes, scalar
from tests.test_gpu_timeout import _run_expired

pytestmark = pytest.mark.gpu


def check(o):
    assert o["amax"].isnan().item()                            # a scale update keeps its scale
    assert o["scale_inv"].item() == (1.0 / torch.tensor(12.0)).item()


# W as [K][2N]: its few rows wait for their loads too (as [2N][K] they wait for nothing)
@pytest.mark.parametrize("M,b_mn", [(1, True), (8, True), (600, True), (600, False)])
def test_forward(cuda_lib, M, b_mn):
    K, N = 512, 400
    a, w = codes((M, K), E4, 1), codes((K, 2 * N) if b_mn else (2 * N, K), E4, 2)
    o = dict(q=torch.empty(M, N, dtype=torch.uint8, device="cuda"), scale=scalar(12), scale_inv=scalar(7), amax=scalar(0))
    _run_expired(cuda_lib, 1, lambda: cuda_lib.fp8_gated_gemm(a, 0, w, 0, scalar(1), scalar(1), b_mn=b_mn, **o))
    check(o)


@pytest.mark.parametrize("M", [1, 600])
def test_backward(cuda_lib, M):
    K, N = 512, 400
    a, w = codes((M, K), E5, 1), codes((N, K), E4, 2)
    gu = torch.ones(M, 2 * N, dtype=torch.bfloat16, device="cuda")
    o = dict(q=torch.empty(M, 2 * N, dtype=torch.uint8, device="cuda"), scale=scalar(12), scale_inv=scalar(7), amax=scalar(0))
    _run_expired(cuda_lib, 1, lambda: cuda_lib.fp8_gated_gemm_backward(a, 1, w, 0, scalar(1), scalar(1), gu, **o))
    check(o)
