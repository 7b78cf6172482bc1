"""The scales of an NVFP4 step's first step keep gradients of the repository's own sizes (no kernel runs: the
reference quantisation of tests/_block_quant.py under the scales that the step driver starts with)."""
import numpy as np
import pytest
import torch

from optimizer_fp8_cast_b200 import synth
from optimizer_fp8_cast_b200.step import ROLE_DY, Fp8LinearStep
from tests import _block_quant as bq


@pytest.mark.parametrize("wl", [synth.LINEAR256, synth.STRESS1024, synth.LINEAR4096], ids=lambda w: w.name)
def test_first_dy_is_represented(wl):
    """A block of amax m has the scale s = e4m3(m g / 6), off by 2^-4 of it at most where it is a normal number, and E2M1's
    steps are 2 at most, so a value is off by s / g <= m / 6 * (1 + 2^-4), f32 roundings aside (2^-20)."""
    _, fin, fout = wl.layers[0]
    rows = 64                                            # of the workload's dY
    st = Fp8LinearStep([(fin, fout)], rows, wl.history_len, adamw=wl.adamw, w_init=[torch.zeros(fin, fout)], device="cpu",
                       recipe="nvfp4")
    dy = synth.bf16_bits(synth.linear_inputs(wl, 0, 0)[1][:rows])
    g = np.float32(st.scale[ROLE_DY].item())
    codes, sf = bq.quantise(dy, bq.NVFP4, g)
    got, x = bq.values(codes, sf, bq.NVFP4) / np.float64(g), bq.bf16_f64(dy)
    m = np.repeat(np.abs(x).reshape(rows, -1, 16).max(2), 16, axis=1)
    assert (np.abs(got - x) <= m / 6 * (1 + 2.0 ** -4) * (1 + 2.0 ** -20)).all()
    assert (got.reshape(rows, -1, 16) != 0).any(2).all()


def test_only_the_recipe_with_delayed_4_bit_scales_is_primed():
    def make(recipe):
        return Fp8LinearStep([(64, 32)], 32, 4, adamw=synth.LINEAR256.adamw, w_init=[torch.zeros(64, 32)], device="cpu",
                             recipe=recipe)
    assert make("nvfp4").scale.tolist() == [1.0, 1.0, 512.0] and make("nvfp4").scale_inv[2] == 1 / 512
    for recipe in ("mxfp4", "delayed"):
        assert make(recipe).scale.tolist() == [1.0, 1.0, 1.0]
        with pytest.raises(ValueError, match="prime_scales"):
            make(recipe).prime_scales([], [])
