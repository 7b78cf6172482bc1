"""The rules of kernels that begin while the kernel before them still runs, for the sources that launch so: each of them, so
that a new file is not left out."""
import os
import re

import pytest

from optimizer_fp8_cast_b200 import build
from tests.test_feed_forward_abi_cpu import code

EARLY = sorted(f for f in os.listdir(build.SRC_DIR) if f.endswith(".cuh") and f != "ptx.cuh" and "pdl_enter()" in code(f))


def test_the_files_are_found():
    assert EARLY == ["fp4_matvec.cuh", "gated_rows.cuh", "gemm_pair.cuh", "muon.cuh"]


@pytest.mark.parametrize("name", EARLY + ["gated.cuh"])
def test_no_non_coherent_loads(name):
    text = code(name)
    assert "__ldg(" not in text and "__restrict__" not in text and "ld.global.nc" not in text


@pytest.mark.parametrize("name", EARLY)
def test_every_kernel_waits_for_the_one_before(name):
    text = code(name)
    kernels = [m.start() for m in re.finditer(r"__global__", text)]
    for a, b in zip(kernels, kernels[1:] + [len(text)]):
        assert text[a:b].count("pdl_enter();") == 1
        # nothing is loaded, and no load of a tensor is issued, before it
        before = text[a:a + text[a:b].index("pdl_enter();")]
        assert "ld_dep(" not in before and "tma_load" not in before
