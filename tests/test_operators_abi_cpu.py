"""Refusals of the norm and 4-bit entry points: every invalid argument is found on the host, before any
CUDA call (addresses here are dummies that nothing dereferences)."""
import ctypes as C
import os
import subprocess
import sys

import pytest
import torch

import optimizer_fp8_cast_b200 as fp8
from optimizer_fp8_cast_b200 import _abi, build

P = 16 * 1024            # aligned dummy address
U = P + 4                # 4- but not 16-byte aligned
O = P + 2                # 2-byte aligned


@pytest.fixture(scope="module")
def lib():
    build.build()
    return fp8.load()


def test_fp4_scale_bytes(lib):
    f = lib.fp4_scale_bytes
    assert f(1, 32, 3) == 2 * 512 and f(128, 256, 3) == 2 * 512 and f(129, 256, 3) == 4 * 512
    assert f(1, 32, 4) == 4 * 512 and f(128, 257, 4) == 8 * 512
    assert f(0, 32, 3) == 0 and f(1, 0, 3) == 0 and f(1, 32, 2) == 0 and f(1, 1 << 31, 3) == 0


def test_fp4_cast_refusals(lib):
    def call(n=1, **kw):
        a = dict(x_bf16=P, rows=128, cols=128, quant=3, d_scale=None, q_row=P, scales_row=P, q_col=P,
                 scales_col=P, d_amax_inout=None, d_scale_inv_out=None)
        a.update(kw)
        arr = (_abi.Fp4CastTensor * 1)(_abi.Fp4CastTensor(**a))
        return lib.fp4_cast_multi(arr, n, None)
    assert lib.fp4_cast_multi(None, 1, None) == 1 and call(n=0) == 1 and call(n=4097) == 1
    assert call(x_bf16=None) == 1 and call(q_row=None, q_col=None) == 1
    assert call(scales_row=None) == 1 and call(scales_col=None) == 1
    assert call(quant=2) == 1 and call(quant=5) == 1
    assert call(quant=4) == 1                                        # NVFP4 without its scale
    assert call(d_scale=P) == 1 and call(d_amax_inout=P) == 1 and call(d_scale_inv_out=P) == 1
    assert call(rows=0) == 1 and call(cols=-32) == 1
    assert call(cols=48) == 2 and call(rows=16) == 2                 # rows: only with a column-wise copy
    assert call(rows=1 << 31) == 2 and call(rows=1 << 25, cols=1 << 15) == 2
    for k in ("x_bf16", "q_row", "q_col", "scales_row", "scales_col"):
        assert call(**{k: U}) == 3
    assert call(quant=4, d_scale=O) == 3 and b"misaligned" in lib.fp8t_last_error_message()


def test_fp4_gemm_refusals(lib):
    def call(n=1, **kw):
        a = dict(A=P, A_scales=P, B=P, B_scales=P, quant=3, M=5, N=8, K=32, d_a_scale_inv=None,
                 d_b_scale_inv=None, D_bf16=P)
        a.update(kw)
        return lib.fp4_gemm_multi((_abi.Fp4GemmDesc * 1)(_abi.Fp4GemmDesc(**a)), n, None)
    assert lib.fp4_gemm_multi(None, 1, None) == 1 and call(n=0) == 1 and call(n=5000) == 1
    for k in ("A", "A_scales", "B", "B_scales", "D_bf16"):
        assert call(**{k: None}) == 1 and call(**{k: U}) == 3
    assert call(quant=0) == 1 and call(quant=2) == 1
    assert call(M=0) == 1 and call(N=0) == 1 and call(K=0) == 1
    assert call(N=12) == 2 and call(K=48) == 2 and call(M=1 << 31) == 2
    assert call(M=(1 << 31) - 1, K=1 << 24) == 2                     # scale rows past 32 bits
    assert call(d_a_scale_inv=O) == 3


def test_rmsnorm_refusals(lib):
    def call(**kw):
        a = dict(x_bf16=P, residual_bf16=P, gamma_bf16=P, rows=3, cols=64, eps=1e-5, h_bf16=P, d_rstd_out=P,
                 y_bf16=P, quant=0, fmt=0, q=None, scales=None, d_scale=None, d_amax_inout=None,
                 d_scale_inv_out=None)
        a.update(kw)
        return lib.fp8_rmsnorm_cast(C.byref(_abi.RmsNorm(**a)), None)
    assert lib.fp8_rmsnorm_cast(None, None) == 1
    assert call(x_bf16=None) == 1 and call(gamma_bf16=None) == 1
    assert call(rows=0) == 1 and call(cols=0) == 1
    assert call(eps=-1.0) == 1 and call(eps=float("nan")) == 1 and call(eps=float("inf")) == 1
    assert call(quant=5) == 1 and call(quant=-1) == 1
    assert call(residual_bf16=None) == 1                             # h without a residual
    assert call(y_bf16=None) == 1                                    # nothing asked for
    assert call(q=P) == 1                                            # codes without a quant
    assert call(quant=1, q=P) == 1 and call(quant=1, q=P, d_scale=P) == 1          # no amax slot
    assert call(quant=1, d_scale=P, d_amax_inout=P) == 1             # no codes
    assert call(quant=1, q=P, d_scale=P, d_amax_inout=P, scales=P) == 1
    assert call(quant=1, q=P, d_scale=P, d_amax_inout=P, fmt=2) == 1
    assert call(quant=2, q=P) == 1 and call(quant=2, q=P, scales=P, d_scale=P) == 1
    assert call(quant=3, q=P, scales=P, d_amax_inout=P) == 1
    assert call(quant=4, q=P, scales=P) == 1                         # NVFP4 without its scale
    assert call(cols=24) == 2 and call(cols=16400) == 2 and call(rows=1 << 31) == 2
    assert call(quant=3, q=P, scales=P, cols=48) == 2                # 48 is fine without block scales
    for k in ("x_bf16", "residual_bf16", "gamma_bf16", "h_bf16", "y_bf16"):
        assert call(**{k: U}) == 3
    assert call(d_rstd_out=O) == 3 and call(quant=3, q=U, scales=P) == 3 and call(quant=3, q=P, scales=U) == 3


def test_rmsnorm_backward_refusals(lib):
    need = lib.fp8_rmsnorm_backward_workspace_bytes(3, 64)
    assert need > 0 and need % 4 == 0
    assert lib.fp8_rmsnorm_backward_workspace_bytes(0, 64) == 0
    assert lib.fp8_rmsnorm_backward_workspace_bytes(3, 24) == 0
    assert lib.fp8_rmsnorm_backward_workspace_bytes(3, 16400) == 0

    def call(ws=P, n=need, **kw):
        a = dict(dy_bf16=P, h_bf16=P, gamma_bf16=P, d_rstd=P, dres_bf16=P, rows=3, cols=64, dh_bf16=P,
                 dgamma_f32=P, dgamma_bf16=P)
        a.update(kw)
        return lib.fp8_rmsnorm_backward(C.byref(_abi.RmsNormGrad(**a)), ws, n, None)
    assert lib.fp8_rmsnorm_backward(None, P, need, None) == 1
    for k in ("dy_bf16", "h_bf16", "gamma_bf16", "d_rstd", "dh_bf16"):
        assert call(**{k: None}) == 1
    assert call(rows=0) == 1 and call(cols=0) == 1 and call(cols=24) == 2 and call(cols=16400) == 2
    assert call(ws=None) == 1 and call(n=need - 1) == 1
    for k in ("dy_bf16", "h_bf16", "gamma_bf16", "dres_bf16", "dh_bf16"):
        assert call(**{k: U}) == 3
    assert call(ws=U) == 3 and call(d_rstd=O) == 3 and call(dgamma_f32=O) == 3
    assert call(dgamma_bf16=P + 1) == 3


def test_python_binding_checks_sizes_and_types(lib):
    """The binding refuses what the C side cannot see: wrong types and shapes, CPU tensors, unknown names."""
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    g = torch.ones(64, dtype=torch.bfloat16)
    u = torch.zeros(1, 16, dtype=torch.uint8)
    with pytest.raises(ValueError, match="x: must be a CUDA tensor"):
        fp8.fp8_rmsnorm_cast(x, g, 1e-5, y=torch.empty_like(x))
    with pytest.raises(ValueError, match="x: must be a bfloat16 matrix"):
        fp8.fp8_rmsnorm_cast(x.float(), g, 1e-5, y=torch.empty_like(x))
    with pytest.raises(ValueError, match="x: must be a matrix"):
        fp8.fp8_rmsnorm_cast(g, g, 1e-5, y=g)
    with pytest.raises(TypeError, match="unexpected argument 'bias'"):
        fp8.fp8_rmsnorm_cast(x, g, 1e-5, bias=x)
    with pytest.raises(TypeError, match="two values for argument 'eps'"):
        fp8.fp8_rmsnorm_cast(x, g, 1e-5, eps=1e-5)
    with pytest.raises(TypeError, match="missing argument 'gamma'"):
        fp8.fp8_rmsnorm_cast(x)
    with pytest.raises(TypeError, match="at most 3 positional"):
        fp8.fp8_rmsnorm_cast(x, g, 1e-5, x)
    with pytest.raises(TypeError, match="x: must be a tensor"):
        fp8.fp8_rmsnorm_cast(3, g, 1e-5)
    with pytest.raises(ValueError, match="dy: must be a bfloat16"):
        fp8.fp8_rmsnorm_backward(x.float(), x, g, torch.empty(4), x)
    with pytest.raises(TypeError, match="missing argument"):
        fp8.fp8_rmsnorm_backward(x, x, g, torch.empty(4))
    with pytest.raises(ValueError, match="matrix"):
        fp8.fp4_cast_multi([dict(x=x[0], quant=fp8.Q_MXFP4)])
    with pytest.raises(TypeError, match="list of dicts"):
        fp8.fp4_cast_multi([x])
    with pytest.raises(TypeError, match="list of dicts"):
        fp8.fp4_gemm_multi(dict(A=u))
    with pytest.raises(ValueError, match="one K"):
        fp8.fp4_gemm_multi([dict(A=u, a_sf=None, B=torch.zeros(8, 32, dtype=torch.uint8), b_sf=None,
                                 quant=fp8.Q_MXFP4, D=None)])


def test_binding_documents_its_calls(lib):
    for f in (fp8.fp8_rmsnorm_cast, fp8.fp8_rmsnorm_backward, fp8.fp4_cast_multi, fp8.fp4_gemm_multi):
        assert f.__doc__ and f.__text_signature__
    assert all(hasattr(fp8, n) for n in fp8.__all__)


def test_binding_refuses_integers_that_would_wrap(lib):
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="constant of the package"):
        fp8.fp8_rmsnorm_cast(x, x[0], 1e-5, quant=(1 << 32) + fp8.Q_FP8)
    with pytest.raises(ValueError, match="constant of the package"):
        fp8.fp4_cast_multi([dict(x=x, quant=(1 << 32) + fp8.Q_MXFP4)])


def test_importing_the_step_driver_loads_no_library():
    code = ("import sys, optimizer_fp8_cast_b200.step as s, optimizer_fp8_cast_b200 as p;"
            "assert p._lib is None and not any(m.endswith('._binding') for m in sys.modules)")
    subprocess.run([sys.executable, "-c", code], check=True, cwd=os.path.dirname(os.path.dirname(__file__)))
