"""Whole 4-bit training steps of the step driver, stage by stage against the 64-bit reference (each stage's
reference input is what the GPU's own earlier stage gave), and their replay from a CUDA graph."""
import numpy as np
import pytest
import torch

import oracle
from optimizer_fp8_cast_b200 import synth
from optimizer_fp8_cast_b200.step import Fp8LinearStep
from tests import _block_quant as bq
from tests._gpu import bf16_bits, u8
from tests._pins import gemm_within_tolerance

pytestmark = pytest.mark.gpu
KIND = {"mxfp4": bq.MXFP4, "nvfp4": bq.NVFP4}


def make(recipe, shapes, tokens, **kw):
    wl = synth.LINEAR256
    ws = [(torch.randn(fi, fo, generator=torch.Generator().manual_seed(7 + i)) * 0.02).to(torch.bfloat16)
          for i, (fi, fo) in enumerate(shapes)]
    return Fp8LinearStep(shapes, tokens, 4, "max", 0, wl.adamw, ws, "cuda", recipe=recipe, **kw)


def inputs(shapes, tokens, seed):
    g = torch.Generator().manual_seed(seed)
    xs = [torch.randn(tokens, fi, generator=g).to(torch.bfloat16).cuda() for fi, _ in shapes]
    dys = [(torch.randn(tokens, fo, generator=g) * 1e-3).to(torch.bfloat16).cuda() for _, fo in shapes]
    return xs, dys


@pytest.mark.parametrize("recipe", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("shapes,tokens", [([(256, 256)], 512), ([(160, 416), (288, 64)], 352)])
def test_fp4_steps(cuda_lib, recipe, shapes, tokens):
    st, kind = make(recipe, shapes, tokens), KIND[recipe]
    for step in range(3):
        xs, dys = inputs(shapes, tokens, step)
        before = dict(scale=st.scale.cpu().numpy().copy(), history=st.history.cpu().numpy().copy(),
                      W=[bf16_bits(L.W) for L in st.layers],
                      opt=[[t.cpu().numpy().reshape(-1).copy() for t in (L.master, L.m, L.v)] for L in st.layers])
        st.step(xs, dys)
        torch.cuda.synchronize()
        cuda_lib.fp8t_check_device_error()
        for k, L in enumerate(st.layers):
            v = {}
            for role, (name, b) in enumerate((("X", bf16_bits(xs[k])), ("W", before["W"][k]), ("dY", bf16_bits(dys[k])))):
                g = before["scale"][3 * k + role] if kind == bq.NVFP4 else np.float32(1)
                for way, bb in (("row", b), ("col", np.ascontiguousarray(b.T))):
                    codes, sf = bq.quantise(bb, kind, g)
                    assert np.array_equal(bq.unpack(u8(L.fp4[name]["q_" + way])), codes)
                    assert np.array_equal(u8(L.fp4[name]["sf_" + way]), bq.atoms(sf, kind))
                    v[name, way] = bq.values(codes, sf, kind) / np.float64(g)
                if kind == bq.NVFP4:                     # the delayed scale: 448 * 6 over the window's largest amax
                    h = st.history[3 * k + role].cpu().numpy()
                    assert h[0] == bq.bf16_f64(b & 0x7FFF).max()
                    assert np.array_equal(h[1:], before["history"][3 * k + role][:-1])
                    assert st.scale[3 * k + role].item() == np.float32(2688) / h.max()
            for D, a, b in ((L.Y, v["X", "row"], v["W", "col"]), (L.dX, v["dY", "row"], v["W", "row"]),
                            (L.dW, v["X", "col"], v["dY", "col"])):
                R, ab = a @ b.T, np.abs(a) @ np.abs(b).T
                R = bf16_bits(torch.from_numpy(R).float().to(torch.bfloat16))
                assert gemm_within_tolerance(bf16_bits(D), R, ab).all()
        master, m, v_ = ([o[i] for o in before["opt"]] for i in range(3))
        oracle.fused_adamw(master, m, v_, [bf16_bits(L.dW).reshape(-1) for L in st.layers],
                           [np.zeros(L.W.numel(), np.uint16) for L in st.layers], dict(synth.LINEAR256.adamw, step=step + 1))
        for k, L in enumerate(st.layers):
            assert np.allclose(L.master.cpu().numpy().reshape(-1), master[k], rtol=2.0 ** -21, atol=0)


@pytest.mark.parametrize("recipe", ["mxfp4", "nvfp4"])
def test_fp4_step_in_a_graph(cuda_lib, recipe):
    """Two replays of a captured step equal two eager ones bit for bit."""
    shapes, tokens = [(256, 128)], 160
    xs, dys = inputs(shapes, tokens, 3)
    eager = make(recipe, shapes, tokens, device_step=True)
    for _ in range(2):
        eager.step(xs, dys)
    st = make(recipe, shapes, tokens, device_step=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            st.step(xs, dys, stream=s)
    torch.cuda.synchronize()
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    cuda_lib.fp8t_check_device_error()
    for a, b in zip(eager.layers, st.layers):
        for n in ("Y", "dX", "dW", "W", "master", "m", "v"):
            assert torch.equal(getattr(a, n).view(torch.uint8), getattr(b, n).view(torch.uint8)), n
    for n in ("scale", "history", "amax", "grad_norm"):
        assert torch.equal(getattr(eager, n), getattr(st, n)), n
