"""A Muon step whose call fails on the host: what the source does in which order (no launch can be made to fail here)."""
import os
import re

from optimizer_fp8_cast_b200 import build
from tests.test_early_launch_cpu import body


def source(name):
    with open(os.path.join(build.SRC_DIR, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_tensor_maps_come_before_the_first_kernel_that_writes_momentum():
    text = source("fp8train.cu")
    call = body(text, r"fp8t_status muon_call\(")
    scale = call.index("k_muon_scale<MODE>")
    after = call[scale:]
    # behind that kernel there are launches only: no function that encodes a tensor map or allocates
    for name in ("launch_table", "newton_schulz"):
        b = body(text, r"fp8t_status " + name + r"\(")
        assert "encode" not in b and "fill_muon_matrix" not in b and "vector" not in b
    assert "prepare" not in after and "encode" not in after and "launch_table(" in after
    assert "prepare_table(" in call[:scale]


def test_only_the_last_pass_clears_skipped():
    text = source("muon.cuh")
    scale, apply = body(text, r"k_muon_scale\("), body(text, r"k_muon_apply\(")
    assert re.findall(r"\*t\.skipped = (\d)", scale) == ["1"] and re.findall(r"\*t\.skipped = (\d)", apply) == ["0"]
