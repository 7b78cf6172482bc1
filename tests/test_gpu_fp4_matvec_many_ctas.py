"""fp4_matvec without an activation where it has more CTAs (of 32 outputs) than the GPU has SMs: eight warps, three CTAs an SM."""
import pytest
import torch

from tests import _feed_forward as ff
from tests.test_gpu_fp4_matvec import run

pytestmark = pytest.mark.gpu


# N that ends inside a CTA, a group and a group's first eight rows; several chunks a warp, idle warps, a last chunk of 32
@pytest.mark.parametrize("nv", [False, True])
@pytest.mark.parametrize("M,K,N", [(1, 4096, 4760), (8, 2080, 11016), (3, 32, 4744), (5, 288, 14232), (2, 1056, 9488)])
def test_product(cuda_lib, M, K, N, nv):
    y, want, off = run(cuda_lib, M, K, N, nv, "none", seed=N)
    assert ff.within(y, want, off, ff.BF16)


@pytest.mark.parametrize("nv", [False, True])
def test_the_same_bits_twice(cuda_lib, nv):
    """Twice the same."""
    y, _, _ = run(cuda_lib, 8, 544, 9496, nv, "none", seed=1)
    again, _, _ = run(cuda_lib, 8, 544, 9496, nv, "none", seed=1)
    assert torch.equal(y, again)
