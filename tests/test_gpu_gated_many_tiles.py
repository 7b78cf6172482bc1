"""Gated products whose clusters have three tiles and more each: accumulators handed back and chunks fetched ahead from tile to
tile (74 CTA pairs)."""
import pytest

from tests.test_gpu_gated import backward, check_backward, check_forward, forward

pytestmark = pytest.mark.gpu


# 9 x 33 tiles of 256 columns, or 9 x 43 of 192; 17 x 18; 3 x 86
@pytest.mark.parametrize("M,K,N", [(2100, 144, 8208), (4353, 144, 4368), (700, 272, 21984)])
@pytest.mark.parametrize("b_mn", [False, True])
@pytest.mark.parametrize("inplace", [False, True])
def test_backward(cuda_lib, M, K, N, b_mn, inplace):
    check_backward(*backward(cuda_lib, M, K, N, "gelu" if inplace else "silu", b_mn, inplace=inplace, outs="d" if inplace else "dq"))


@pytest.mark.parametrize("M,K,N", [(2100, 144, 4112), (4353, 272, 2192), (10000, 16, 1040)])
@pytest.mark.parametrize("b_mn", [False, True])
def test_forward(cuda_lib, M, K, N, b_mn):
    check_forward(*forward(cuda_lib, M, K, N, "gelu" if b_mn else "silu", b_mn))
