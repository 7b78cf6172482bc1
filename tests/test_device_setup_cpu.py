"""A call sets up its own kernels only: what every call runs first names none of the norm's and the 4-bit ones'."""
import os
import re

import pytest

from optimizer_fp8_cast_b200 import build


def function(name):
    with open(build.MAIN) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    at = text.index("{", re.search(r"^\w[^;{}]*\b%s\([^;{}]*\)\s*\{" % name, text, re.M).end() - 1)
    depth, i = 1, at + 1
    while depth:
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        i += 1
    return text[at:i]


def test_common_set_up_is_that_of_the_8_bit_calls():
    body = function("current_device")
    assert "k_fp8_gemm" in body and not re.search(r"fp4|norm::", body)


@pytest.mark.parametrize("call,ready", [("fp4_cast_multi", "ready_fp4_cast"), ("fp4_gemm_multi", "ready_fp4_gemm"),
                                        ("fp8_rmsnorm_backward", "ready_norm_backward")])
def test_calls_set_up_their_kernels_before_they_launch(call, ready):
    body = function(call)
    launch = re.search(r"launch_pdl\(|fp4_gemm_split\(|fp4_gemm_tiles\(", body).start()
    assert body.index("current_device(") < body.index(ready + "(") < launch
