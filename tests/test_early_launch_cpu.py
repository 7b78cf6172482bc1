"""What the sources of kernels that start before their predecessor has ended (programmatic launch) have to keep."""
import os
import re

import pytest

from optimizer_fp8_cast_b200 import build

SOURCES = ("fp4_cast.cuh", "gemm_fp4.cuh", "rmsnorm.cuh")


def code(name):
    with open(os.path.join(build.SRC_DIR, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_the_list_is_complete():
    early = [f for f in sorted(os.listdir(build.SRC_DIR))
             if f.endswith(".cuh") and f != "ptx.cuh" and "pdl_wait()" in code(f)]
    assert tuple(early) == SOURCES


@pytest.mark.parametrize("name", SOURCES)
def test_no_non_coherent_loads(name):
    """ld.global.nc needs memory that is read-only for the kernel's whole life; here the kernel before writes scales,
    scale inverses, rstd and partial rows while this one is resident."""
    text = code(name)
    assert "__ldg(" not in text and "__restrict__" not in text and "ld.global.nc" not in text
