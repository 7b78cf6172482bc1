"""A buffer in shared memory that a warp has read and fills again by an asynchronous copy: the reads may still be queued behind
a __syncwarp, so lane 0 sees an arrival that it queued behind them before it starts the copy."""
import re

import pytest

from tests.test_early_launch_cpu import body
from tests.test_feed_forward_abi_cpu import code


@pytest.mark.parametrize("name,head,copy", [("gemm_pair.cuh", r"void fetch\(", "tma_load_2d("),
                                            ("gated_rows.cuh", r"auto refill = ", "fetch(")])
def test_reads_are_over_before_the_copy(name, head, copy):
    f = body(code(name), head)
    order = [f.index(s) for s in ("__syncwarp()", "mbar_arrive(", "mbar_wait(", copy)]
    assert order == sorted(order)


def test_slots_are_filled_again_in_one_place():
    text = code("gated_rows.cuh")
    kernel = text[text.index("k_gated_rows_mn("):]
    loop = body(kernel, r"for \(int c0 = warp;")
    assert "refill(" in loop and not re.search(r"\bfetch\(", loop)
