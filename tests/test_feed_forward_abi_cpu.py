"""Refusals of the gated, Muon and 4-bit matrix-vector entry points: every invalid argument is found on the host, before
any CUDA call (addresses here are dummies that nothing dereferences); and what their sources have to keep."""
import ctypes as C
import os
import re

import pytest
import torch

import optimizer_fp8_cast_b200 as fp8
from optimizer_fp8_cast_b200 import _abi, build

P = 16 * 1024            # aligned dummy address
U = P + 4                # 4- but not 16-byte aligned
O = P + 2                # 2-byte aligned
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    build.build()
    return fp8.load()


def test_gated_refusals(lib):
    def call(**kw):
        a = dict(A=P, a_fmt=0, B=P, b_fmt=0, b_layout=0, M=3, N=16, K=32, d_a_scale_inv=P, d_b_scale_inv=P, act=1,
                 gu_bf16=None, h_bf16=None, q=P, q_fmt=0, d_scale=P, d_amax_inout=P, d_scale_inv_out=P)
        a.update(kw)
        return lib.fp8_gated_gemm(C.byref(_abi.Gated(**a)), None)
    assert lib.fp8_gated_gemm(None, None) == 1
    for k in ("A", "B", "d_a_scale_inv", "d_b_scale_inv"):
        assert call(**{k: None}) == 1
    assert call(q=None, d_scale=None, d_scale_inv_out=None) == 1 and b"no output" in lib.fp8t_last_error_message()
    assert call(d_scale=None) == 1 and call(q=None, h_bf16=P) == 1
    assert call(q=None, h_bf16=P, d_scale=None) == 1                 # an inverse of no scale
    for k in ("a_fmt", "b_fmt", "q_fmt"):
        assert call(**{k: 2}) == 1 and call(**{k: -1}) == 1
    assert call(act=0) == 1 and call(act=3) == 1 and call(b_layout=2) == 1
    for k in ("M", "N", "K"):
        assert call(**{k: 0}) == 1 and call(**{k: -16}) == 1 and call(**{k: 1 << 30}) == 2
    assert call(N=24) == 2 and call(K=40) == 2
    assert call(M=1 << 29, N=1 << 20) == 2                           # tiles past 32 bits
    for k in ("A", "B", "gu_bf16", "h_bf16", "q"):
        assert call(**{k: U}) == 3
    for k in ("d_a_scale_inv", "d_b_scale_inv", "d_scale", "d_amax_inout", "d_scale_inv_out"):
        assert call(**{k: O}) == 3


def test_gated_backward_refusals(lib):
    def call(**kw):
        a = dict(A=P, a_fmt=1, B=P, b_fmt=0, b_layout=0, M=3, N=16, K=32, d_a_scale_inv=P, d_b_scale_inv=P, act=2,
                 gu_bf16=P, dgu_bf16=None, q=P, q_fmt=1, d_scale=P, d_amax_inout=P, d_scale_inv_out=P)
        a.update(kw)
        return lib.fp8_gated_gemm_backward(C.byref(_abi.GatedGrad(**a)), None)
    assert lib.fp8_gated_gemm_backward(None, None) == 1
    for k in ("A", "B", "d_a_scale_inv", "d_b_scale_inv", "gu_bf16"):
        assert call(**{k: None}) == 1
    assert call(q=None, d_scale=None, d_scale_inv_out=None) == 1
    assert call(d_scale=None) == 1 and call(q=None, dgu_bf16=P) == 1
    assert call(act=0) == 1 and call(q_fmt=2) == 1 and call(b_layout=-1) == 1
    assert call(M=0) == 1 and call(N=8) == 2 and call(K=24) == 2
    for k in ("A", "B", "gu_bf16", "dgu_bf16", "q"):
        assert call(**{k: U}) == 3
    assert call(d_amax_inout=O) == 3


def test_matvec_refusals(lib):
    def call(**kw):
        a = dict(x_bf16=P, rows=1, N=8, K=32, q=P, scales=P, quant=3, d_w_scale_inv=None, act=0, y_bf16=P)
        a.update(kw)
        return lib.fp4_matvec(C.byref(_abi.Fp4Matvec(**a)), None)
    assert lib.fp4_matvec(None, None) == 1
    for k in ("x_bf16", "q", "scales", "y_bf16"):
        assert call(**{k: None}) == 1 and call(**{k: U}) == 3
    assert call(quant=2) == 1 and call(quant=5) == 1 and call(act=3) == 1 and call(act=-1) == 1
    assert call(rows=0) == 1 and call(N=0) == 1 and call(K=-32) == 1
    assert call(rows=9) == 2 and call(N=12) == 2 and call(K=48) == 2 and call(N=1 << 30) == 2 and call(K=1 << 30) == 2
    assert call(d_w_scale_inv=O) == 3


def test_muon_refusals(lib):
    ws = 1 << 24

    def step(n=1, lr=1e-3, beta=0.9, wd=0.1, rms=0.2, scale=1.0, steps=5, skipped=None, w=P, size=ws, **kw):
        a = dict(master=P, momentum=2 * P, grad_bf16=3 * P, weight_bf16=4 * P, rows=4, cols=4)
        a.update(kw)
        arr = (_abi.MuonTensor * 2)(_abi.MuonTensor(**a), _abi.MuonTensor(5 * P, 6 * P, 7 * P, 8 * P, 4, 4))
        return lib.fused_muon_multi_tensor(arr, n, lr, beta, wd, rms, scale, 1, steps, skipped, w, size, None)
    assert lib.fused_muon_multi_tensor(None, 1, 0, 0, 0, 0, 1, 0, 5, None, P, ws, None) == 1
    assert step(n=0) == 1 and step(n=4097) == 1
    for k in ("master", "momentum", "grad_bf16", "weight_bf16"):
        assert step(**{k: None}) == 1 and step(**{k: U}) == 3
    for bad in (NAN, INF):
        assert step(lr=bad) == 1 and step(beta=bad) == 1 and step(wd=bad) == 1 and step(rms=bad) == 1 and step(scale=bad) == 1
    assert step(scale=0.0) == 1 and step(scale=-1.0) == 1
    assert step(steps=0) == 1 and step(steps=17) == 1
    assert step(rows=0) == 2 and step(cols=-1) == 2 and step(rows=65537) == 2
    assert step(w=None) == 1 and step(size=100) == 1 and step(w=P + 16) == 3 and step(skipped=O) == 3
    assert step(n=2, master=5 * P) == 1 and b"twice" in lib.fp8t_last_error_message()
    assert step(momentum=P) == 1
    assert step(n=2, grad_bf16=8 * P) == 1                           # another tensor's weight, or this one's master
    assert step(grad_bf16=P) == 1

    def orth(n=1, f32=0, steps=5, w=P, size=ws, **kw):
        a = dict(x=P, out_bf16=2 * P, rows=4, cols=4)
        a.update(kw)
        arr = (_abi.OrthMatrix * 2)(_abi.OrthMatrix(**a), _abi.OrthMatrix(3 * P, 4 * P, 4, 4))
        return lib.muon_orthogonalize(arr, n, f32, steps, w, size, None)
    assert lib.muon_orthogonalize(None, 1, 0, 5, P, ws, None) == 1
    assert orth(n=0) == 1 and orth(x=None) == 1 and orth(out_bf16=None) == 1 and orth(steps=0) == 1
    assert orth(x=U) == 3 and orth(out_bf16=U) == 3 and orth(rows=0) == 2 and orth(size=10) == 1
    assert orth(f32=1, out_bf16=P) == 1                              # an f32 matrix has no room for itself in BF16
    assert orth(n=2, out_bf16=4 * P) == 1
    assert orth(n=2, out_bf16=3 * P) == 1 and b"another matrix" in lib.fp8t_last_error_message()


def test_muon_workspace_bytes(lib):
    def need(*shapes):
        return fp8.muon_workspace_bytes(shapes)
    assert need((0, 4)) == 0 and need((4, 65537)) == 0 and need((-1, 4)) == 0
    # X twice, A and B in FP16, a partial sum per 8192 elements, a norm
    copies = 2 * 256 * 512 * 2 + 2 * 256 * 256 * 2
    assert need((256, 512)) == need((512, 256)) == copies + 256 + 256
    assert need((256, 512), (256, 512)) == 2 * copies + 512
    # a table of 24 at a time: 48 matrices need the copies of 24, and 48 norms
    assert need(*[(256, 512)] * 48) - need(*[(256, 512)] * 24) == 48 * 16 + 256 - (24 * 16 + 128)
    assert need((7, 9)) == 2 * 256 + 2 * 256 + 512                   # pitches of 16 and 8 elements


def test_python_calls_refuse(lib):
    m = fp8._load_binding()
    z = torch.zeros(4, 32, dtype=torch.uint8)
    f = torch.ones(1)
    with pytest.raises(ValueError, match="CUDA tensor"):
        m.fp8_gated_gemm(z, 0, torch.zeros(32, 32, dtype=torch.uint8), 0, f, f)
    with pytest.raises(ValueError, match="B: must be"):
        m.fp8_gated_gemm(z, 0, torch.zeros(32, 16, dtype=torch.uint8), 0, f, f)
    with pytest.raises(ValueError, match="B: must be"):
        m.fp8_gated_gemm(z, 0, torch.zeros(33, 32, dtype=torch.uint8), 0, f, f)      # an odd number of features
    with pytest.raises(ValueError, match="codes"):
        m.fp8_gated_gemm(f.reshape(1, 1), 0, z, 0, f, f)
    with pytest.raises(TypeError, match="missing"):
        m.fp8_gated_gemm_backward(z, 0, z, 0, f, f)
    with pytest.raises(TypeError, match="unexpected"):
        m.fp4_matvec(z, z, z, 3, z, gate=1)
    with pytest.raises(ValueError, match="q: must be"):
        m.fp4_matvec(torch.zeros(1, 32, dtype=torch.bfloat16), torch.zeros(8, 8, dtype=torch.uint8), f, 3, z)
    x = torch.zeros(4, 4)
    with pytest.raises(ValueError, match="same length"):
        fp8.muon_orthogonalize([], [])
    with pytest.raises(ValueError, match="bfloat16"):
        fp8.muon_orthogonalize([x], [x])
    with pytest.raises(ValueError, match="shapes"):
        fp8.fused_muon_multi_tensor([x], [x[:2]], [x.bfloat16()], [x.bfloat16()], lr=0.1)
    with pytest.raises(ValueError, match="float32"):
        fp8.fused_muon_multi_tensor([x.double()], [x], [x.bfloat16()], [x.bfloat16()], lr=0.1)


def code(name):
    with open(os.path.join(build.SRC_DIR, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


@pytest.mark.parametrize("name", ["gemm_pair.cuh", "gated.cuh", "muon.cuh", "fp4_matvec.cuh"])
def test_no_non_coherent_loads(name):
    """These kernels begin while the kernel before them still runs, so nothing that it writes is read-only for them."""
    text = code(name)
    assert "__ldg(" not in text and "__restrict__" not in text and "ld.global.nc" not in text


@pytest.mark.parametrize("name", ["gemm_pair.cuh", "muon.cuh", "fp4_matvec.cuh"])
def test_every_kernel_waits_for_the_one_before(name):
    text = code(name)
    kernels = len(re.findall(r"__global__", text))
    assert kernels > 0 and text.count("pdl_enter();") == kernels


@pytest.mark.parametrize("name", ["fp8_gated_gemm", "fp8_gated_gemm_backward", "fp4_matvec"])
def test_declaration_and_compiled_function_say_the_same(lib, name):
    import inspect
    declared, compiled = getattr(fp8, name), getattr(fp8._load_binding(), name)
    assert inspect.getdoc(declared) == inspect.getdoc(compiled)
    assert list(inspect.signature(getattr(declared, "__wrapped__", declared)).parameters) == \
        list(inspect.signature(compiled).parameters)
