"""Bounded waits of the 4-bit kernels, without a fault: with the test hook every wait (mode 1), or only the
epilogue's (mode 2: loads and MMAs are in flight), runs out after 1 ms, the kernel records FP8T_ERR_TIMEOUT,
drains and returns, and the next call is right."""
import numpy as np
import pytest
import torch

from tests import _block_quant as bq
from tests._gpu import bf16_bits
from tests._pins import gemm_within_tolerance
from tests.test_gpu_fp4 import cast, check_cast, operand, random_bits, reference
from tests.test_gpu_timeout import _run_expired

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("mode", [1, 2])
@pytest.mark.parametrize("kind", [bq.MXFP4, bq.NVFP4])
@pytest.mark.parametrize("M,N,K", [(1, 4096, 4096), (50, 1024, 4096), (128, 256, 2048), (900, 1024, 4096), (2100, 4104, 544)])
def test_gemm_waits_expire_and_context_survives(cuda_lib, mode, kind, M, N, K):
    """The K split over a cluster (apart and over the stages), 256- and 384-column tiles."""
    A, sa, a = operand(M, K, kind, 1)
    B, sb, b = operand(N, K, kind, 2)
    D = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    g = [dict(A=A, a_sf=sa, B=B, b_sf=sb, quant=kind, D=D)]
    _run_expired(cuda_lib, mode, lambda: cuda_lib.fp4_gemm_multi(g))
    cuda_lib.fp4_gemm_multi(g)
    cuda_lib.fp8t_check_device_error()
    rows = np.unique(np.random.default_rng(0).integers(0, M, 40))
    R, ab = reference(a[rows], b, 1.0)
    assert gemm_within_tolerance(bf16_bits(D)[rows], R, ab).all()


def test_cast_waits_expire_and_context_survives(cuda_lib):
    bits = random_bits(1024, 2048, 3)
    d = cast(cuda_lib, bits, bq.MXFP4, 1.0)
    _run_expired(cuda_lib, 1, lambda: cuda_lib.fp4_cast_multi([d]))
    cuda_lib.fp4_cast_multi([d])
    cuda_lib.fp8t_check_device_error()
    check_cast(d, bits, bq.MXFP4, 1.0)
