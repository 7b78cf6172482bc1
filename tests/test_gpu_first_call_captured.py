"""The library's very first calls of a process may be captured ones: setting up kernels is allowed while a stream
captures. Each case runs in a process of its own."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SET_UP = """
import torch, optimizer_fp8_cast_b200 as fp8
R, C = 160, 512
x = torch.randn(R, C, device="cuda").to(torch.bfloat16)
gamma = torch.ones(C, dtype=torch.bfloat16, device="cuda")
u8 = dict(dtype=torch.uint8, device="cuda")
def operand():
    return torch.zeros(R, C // 2, **u8), torch.zeros(fp8.fp4_scale_bytes(R, C, fp8.Q_MXFP4), **u8)
q, sf = operand()
y, dh = torch.zeros_like(x), torch.zeros_like(x)
D, few = torch.zeros(R, R, dtype=torch.bfloat16, device="cuda"), torch.zeros(32, R, dtype=torch.bfloat16, device="cuda")
rstd, dg = torch.zeros(R, device="cuda"), torch.zeros(C, device="cuda")
outs = [q, sf, y, dh, D, few, rstd, dg]
"""
CALLS = {
    "cast": "fp8.fp4_cast_multi([dict(x=x, quant=fp8.Q_MXFP4, q_row=q, sf_row=sf)])",
    "two-way cast": """fp8.fp4_cast_multi([dict(x=x, quant=fp8.Q_MXFP4, q_row=q, sf_row=sf, q_col=qc, sf_col=sfc)])""",
    "product": """fp8.fp4_gemm_multi([dict(A=q, a_sf=sf, B=q, b_sf=sf, quant=fp8.Q_MXFP4, D=D)])""",
    "product of few rows": """fp8.fp4_gemm_multi([dict(A=q[:32], a_sf=sf, B=q, b_sf=sf, quant=fp8.Q_MXFP4, D=few)])""",
    "norm": """fp8.fp8_rmsnorm_cast(x, gamma, 1e-5, rstd=rstd, y=y, quant=fp8.Q_MXFP4, q=q, sf=sf)""",
    "gradient": """fp8.fp8_rmsnorm_backward(x, x, gamma, rstd, dh, dgamma=dg)""",
}


@pytest.mark.parametrize("call", list(CALLS))
def test_first_call_of_a_process_is_captured(cuda_lib, call):
    code = SET_UP + f"""
qc, sfc = torch.zeros(C, R // 2, **u8), torch.zeros(fp8.fp4_scale_bytes(C, R, fp8.Q_MXFP4), **u8)
outs += [qc, sfc]
def call():
    {CALLS[call]}
q.random_(0, 255); sf.fill_(127); rstd.fill_(0.5)
first = [t.clone() for t in outs]
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    call()
g.replay()
torch.cuda.synchronize()
fp8.fp8t_check_device_error()
got = [t.clone() for t in outs]
for t, f in zip(outs, first):
    t.copy_(f)
call()
torch.cuda.synchronize()
assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, outs))
assert any(not torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, first))
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=240)
    assert r.returncode == 0, r.stderr[-2000:]
