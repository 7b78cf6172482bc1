"""A buffer in shared memory that a warp has read and fills again by an asynchronous copy: the reads may still be queued behind
a __syncwarp, so the source orders them (a proxy fence by every lane) and sees an arrival that it queued behind them."""
import re

import pytest

from tests.test_early_launch_cpu import body
from tests.test_feed_forward_abi_cpu import code


@pytest.mark.parametrize("name,head", [("gemm_pair.cuh", r"void fetch\(")])
def test_reads_are_over_before_the_copy(name, head):
    f = body(code(name), head)
    order = [f.index(s) for s in ("fence_proxy_async_smem()", "__syncwarp()", "mbar_arrive(", "mbar_wait(", "mbar_arrive_expect_tx(",
                                  "tma_load_2d(")]
    assert order == sorted(order)
    assert len(re.findall(r"tma_load_2d\(", f)) >= 1
