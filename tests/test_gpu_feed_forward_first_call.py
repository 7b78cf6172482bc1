"""The first call of a process may be a captured one (tests/test_gpu_first_call_captured.py), for the gated, Muon and 4-bit
matrix-vector calls. Each case runs in a process of its own."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SET_UP = """
import torch, optimizer_fp8_cast_b200 as fp8
M, K, N = 300, 256, 144
codes = lambda *s: torch.randint(0x20, 0x40, s, dtype=torch.uint8, device="cuda")
bf = lambda *s: torch.randn(s, device="cuda").to(torch.bfloat16)
inv = torch.full((1,), 0.05, device="cuda")
a, w, wt = codes(M, K), codes(2 * N, K), codes(K, 2 * N)
h, few, y = bf(M, N), bf(5, N), bf(3, N)
gu = bf(M, 2 * N); dgu = bf(M, 2 * N)
q4, sf = codes(N, K // 2), torch.full((fp8.fp4_scale_bytes(N, K, fp8.Q_MXFP4),), 120, dtype=torch.uint8, device="cuda")
x, x2 = bf(3, K), bf(300, 520)
o, o2 = bf(300, 520), bf(64, 100)
small = bf(64, 100)
p, m = [torch.randn(300, 300, device="cuda")], [torch.randn(300, 300, device="cuda")]
pw, g = [bf(300, 300)], [bf(300, 300)]
outs = [h, few, y, dgu, o, o2, p[0], m[0], pw[0]]
"""
CALLS = {
    "gated": "fp8.fp8_gated_gemm(a, 0, w, 0, inv, inv, h=h)",
    "gated in x out": "fp8.fp8_gated_gemm(a, 0, wt, 0, inv, inv, b_mn=True, h=h)",
    "gated few rows": "fp8.fp8_gated_gemm(a[:5], 0, w, 0, inv, inv, h=few)",
    "gated few rows in x out": "fp8.fp8_gated_gemm(a[:5], 0, wt, 0, inv, inv, b_mn=True, h=few)",
    "gated gradient": "fp8.fp8_gated_gemm_backward(a, 0, w[:N], 0, inv, inv, gu, dgu=dgu)",
    "matvec": "fp8.fp4_matvec(x, q4, sf, fp8.Q_MXFP4, y)",
    "orthogonalize": "fp8.muon_orthogonalize([x2], [o])",
    "orthogonalize small": "fp8.muon_orthogonalize([small], [o2])",
    "muon": "fp8.fused_muon_multi_tensor(p, m, g, pw, lr=0.1)",
}


@pytest.mark.parametrize("call", list(CALLS))
def test_first_call_of_a_process_is_captured(cuda_lib, call):
    code = SET_UP + f"""
def call():
    {CALLS[call]}
first = [t.clone() for t in outs]
g_ = torch.cuda.CUDAGraph()
with torch.cuda.graph(g_):
    call()
g_.replay()
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
