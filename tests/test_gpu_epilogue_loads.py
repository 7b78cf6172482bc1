"""Products that read tensors through buffers which are filled beside the tensor cores' work: the same call gives the same bits every
time. A chunk's buffer is filled again as soon as its reads have been issued, so a fill that came before a queued read
showed as 16-byte pieces of the next chunk, in about one gradient of a hundred of these sizes."""
import pytest
import torch

from tests.test_gpu_gated import E4, E5, check_backward, backward, codes, scalar
from tests.test_gpu_muon import matrix

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,K,N,b_mn", [(2679, 640, 5440, False), (2679, 640, 5440, True), (4353, 272, 4368, False)])
def test_gradient_repeats(cuda_lib, M, K, N, b_mn):
    """Several tiles a CTA pair and few k-blocks each, so that the epilogues run beside MMAs all the time."""
    a, w = codes((M, K), E5, 1), codes((K, N) if b_mn else (N, K), E4, 2)
    gen = torch.Generator(device="cuda").manual_seed(3)
    gu = (torch.randn(M, 2 * N, generator=gen, device="cuda") * 0.1).to(torch.bfloat16)
    inv, want, d, wrong = scalar(0.1), torch.empty_like(gu), torch.empty_like(gu), 0
    check_backward(*backward(cuda_lib, M, K, N, "silu", b_mn))
    cuda_lib.fp8_gated_gemm_backward(a, 1, w, 0, inv, inv, gu, b_mn=b_mn, dgu=want)
    for i in range(800):
        if i % 2:
            d.copy_(gu)
            cuda_lib.fp8_gated_gemm_backward(a, 1, w, 0, inv, inv, d, b_mn=b_mn, dgu=d)
        else:
            cuda_lib.fp8_gated_gemm_backward(a, 1, w, 0, inv, inv, gu, b_mn=b_mn, dgu=d)
        wrong += int(not torch.equal(d.view(torch.int16), want.view(torch.int16)))
    cuda_lib.fp8t_check_device_error()
    assert wrong == 0


@pytest.mark.parametrize("rows,cols,times", [(1237, 611, 300), (2310, 2333, 200), (600, 4000, 200)])
def test_newton_schulz_repeats(cuda_lib, rows, cols, times):
    x = matrix(rows, cols, 1).to(torch.bfloat16)
    want, out, wrong = torch.empty_like(x), torch.empty_like(x), 0
    ws = torch.empty(cuda_lib.muon_workspace_bytes([x.shape]), dtype=torch.uint8, device="cuda")
    cuda_lib.muon_orthogonalize([x], [want], workspace=ws)
    for _ in range(times):
        cuda_lib.muon_orthogonalize([x], [out], workspace=ws)
        wrong += int(not torch.equal(out.view(torch.int16), want.view(torch.int16)))
    cuda_lib.fp8t_check_device_error()
    assert wrong == 0


@pytest.mark.parametrize("M,K,N", [(1, 4096, 4736), (8, 4096, 9472), (8, 1024, 11008), (24, 2048, 688), (3, 528, 40000)])
def test_few_rows_repeat(cuda_lib, M, K, N):
    """W as [K][2N] in tiles of 32 to 128 outputs; the smaller weights stay in L2, so that the next chunk comes soon."""
    a, w, inv = codes((M, K), E4, 1), codes((K, 2 * N), E4, 2), scalar(0.05)
    want, h, wrong = torch.empty(M, N, dtype=torch.bfloat16, device="cuda"), torch.empty(M, N, dtype=torch.bfloat16, device="cuda"), 0
    cuda_lib.fp8_gated_gemm(a, 0, w, 0, inv, inv, b_mn=True, h=want)
    for _ in range(1000):
        cuda_lib.fp8_gated_gemm(a, 0, w, 0, inv, inv, b_mn=True, h=h)
        wrong += int(not torch.equal(h.view(torch.int16), want.view(torch.int16)))
    cuda_lib.fp8t_check_device_error()
    assert wrong == 0
