"""The first step of the NVFP4 recipe: its scales, and gradients that are not zero."""
import numpy as np
import pytest
import torch

from optimizer_fp8_cast_b200.step import NVFP4_FIRST_DY, ROLE_DY, ROLE_W, ROLE_X
from tests import _block_quant as bq
from tests._gpu import bf16_bits, u8
from tests.test_gpu_fp4_step import inputs, make

pytestmark = pytest.mark.gpu
SHAPES, TOKENS = [(256, 160), (64, 288)], 192


def amax(t):
    return np.float32(t.float().abs().max().item())


def test_first_step_without_priming(cuda_lib):
    """dY of standard deviation 1e-3: under a scale of 1 every code of it is zero."""
    st = make("nvfp4", SHAPES, TOKENS)
    for k, L in enumerate(st.layers):
        s = st.scale[3 * k:3 * k + 3].tolist()
        assert s[ROLE_W] == np.float32(2688) / amax(L.W) and s[ROLE_X] == 1.0 and s[ROLE_DY] == NVFP4_FIRST_DY
    assert not st.amax.any()
    xs, dys = inputs(SHAPES, TOKENS, 0)
    st.step(xs, dys)
    torch.cuda.synchronize()
    cuda_lib.fp8t_check_device_error()
    for L in st.layers:
        assert (L.dX != 0).any(1).all() and (L.dW != 0).any(1).all()
    assert st.grad_norm.item() > 0


def test_primed_scales_are_those_of_the_tensors(cuda_lib):
    st = make("nvfp4", SHAPES, TOKENS)
    xs, dys = inputs(SHAPES, TOKENS, 1)
    st.prime_scales(xs, dys)
    for k, L in enumerate(st.layers):
        for role, t in ((ROLE_X, xs[k]), (ROLE_W, L.W), (ROLE_DY, dys[k])):
            assert st.scale[3 * k + role].item() == np.float32(2688) / amax(t)
            assert st.history[3 * k + role, 0].item() == amax(t)
    scale = st.scale.clone()
    st.step(xs, dys)
    torch.cuda.synchronize()
    cuda_lib.fp8t_check_device_error()
    assert torch.equal(st.scale, scale)                  # the step's own amax is the primed one
    for k, L in enumerate(st.layers):
        codes, sf = bq.quantise(bf16_bits(dys[k]), bq.NVFP4, np.float32(scale[3 * k + ROLE_DY].item()))
        assert np.array_equal(bq.unpack(u8(L.fp4["dY"]["q_row"])), codes)
        assert np.array_equal(u8(L.fp4["dY"]["sf_row"]), bq.atoms(sf, bq.NVFP4))
        assert (L.dX != 0).any(1).all() and (L.dW != 0).any(1).all()
