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


def body(text, head):
    """The braces after the first place that `head` matches."""
    at = text.index("{", re.search(head, text).end())
    depth, i = 1, at + 1
    while depth:
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        i += 1
    return text[at:i]


@pytest.mark.parametrize("name", ["cluster_sync", "cluster_arrive", "cluster_wait"])
def test_cluster_barriers_converge_their_warps(name):
    """barrier.cluster in its .aligned forms is undefined for a warp whose lanes come one by one."""
    assert re.match(r"\{\s*__syncwarp\(\);\s*asm", body(code("ptx.cuh"), r"void " + name + r"\(\)"))


def test_split_product_waits_as_whole_warps():
    """tcgen05.ld.sync.aligned follows these waits, so a lane may not leave one alone."""
    split = body(code("gemm_fp4.cuh"), r"k_fp4_gemm_split\(const __grid_constant__ SplitGroup g\)")
    assert "warp_wait(" in split and not re.search(r"\bmbar_wait\(", split)


def test_tile_product_converges_before_each_chunk():
    tile = body(code("gemm_fp4.cuh"), r"k_fp4_gemm\(const __grid_constant__ G g\)")
    assert re.search(r"__syncwarp\(\);\s*tmem_ld_32x32b_x32\(t_base \+ c \* 32, r\);", tile)


@pytest.mark.parametrize("head,alloc", [(r"k_fp4_gemm\(const __grid_constant__ G g\)", "tmem_alloc_pair("),
                                        (r"k_fp4_gemm_split\(const __grid_constant__ SplitGroup g\)", "tmem_alloc(")])
def test_tensor_memory_is_taken_before_the_next_kernel_may_start(head, alloc):
    """A dependent kernel waits for this grid's end with what it has allocated: if it could take an SM's tensor
    memory before this grid's CTA there, neither would go on."""
    text = body(code("gemm_fp4.cuh"), head)
    assert text.count("pdl_trigger()") == 1 and text.index(alloc) < text.index("pdl_trigger()")
