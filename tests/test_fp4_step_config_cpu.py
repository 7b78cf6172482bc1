"""Host-side logic of the step driver's 4-bit recipes (no kernel runs)."""
import torch

from optimizer_fp8_cast_b200 import FP4_MAX, fp4_scale_bytes
from tests.test_step_config_cpu import HP
from optimizer_fp8_cast_b200.step import Fp8LinearStep


def make(recipe, layers=1):
    return Fp8LinearStep([(256, 160)] * layers, 192, 16, adamw=HP, w_init=[torch.zeros(256, 160)] * layers,
                         device="cpu", recipe=recipe)


def test_launches_and_buffers():
    st = make("mxfp4")
    assert st.kernels_per_step() == 4 and not st.fused_norm and not st.fused_wcast   # cast, products, AdamW x 2
    assert make("nvfp4").kernels_per_step() == 5                                     # + scale update
    assert make("mxfp4", 3).kernels_per_step() == 5                                  # 9 casts: two launches
    L = st.layers[0]
    assert L.fp4["W"]["q_row"].shape == (256, 80) and L.fp4["W"]["q_col"].shape == (160, 128)
    assert L.fp4["X"]["sf_col"].numel() == fp4_scale_bytes(256, 192, st.quant)
    assert (make("nvfp4").fp8_max == FP4_MAX).all()


def test_products_of_few_rows_take_launches_of_their_own():
    def n(fin, tokens, layers=1):
        st = Fp8LinearStep([(fin, 160)] * layers, tokens, 16, adamw=HP, w_init=[torch.zeros(fin, 160)] * layers,
                           device="cpu", recipe="mxfp4")
        return st.kernels_per_step() - (3 * layers + 7) // 8 - 2
    assert n(256, 192) == 1 and n(96, 192) == 2 and n(256, 64) == 2 and n(96, 64) == 1
    assert n(96, 64, 2) == 2                          # six products of few rows: four and two
    assert n(256, 192, 9) == 2                        # 27 products
