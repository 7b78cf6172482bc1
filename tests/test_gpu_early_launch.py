"""Kernels that start before their predecessor has ended read what it leaves, not what was there when they started:
chains in which scales, scale inverses, rstd and partial rows sit in the same buffers from replay to replay and
change each time, against the same calls with the device idle between them."""
import pytest
import torch

from optimizer_fp8_cast_b200 import E4M3, Q_FP8, Q_NVFP4
from tests import _block_quant as bq
from tests.test_gpu_fp4 import operand

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [1, 9, 128, 300])
def test_scalars_rewritten_between_replays(cuda_lib, rows):
    """product -> norm -> product -> cast -> product -> gradient, on one pair of scale inverses."""
    C = 512
    g = torch.Generator().manual_seed(rows)
    x = torch.randn(rows, C, generator=g).to(torch.bfloat16).cuda()
    gamma = (1 + 0.1 * torch.randn(C, generator=g)).to(torch.bfloat16).cuda()
    W = [operand(C, C, bq.NVFP4, 20 + i)[:2] for i in range(2)]
    scales = [torch.tensor([s], device="cuda") for s in (64.0, 512.0, 8.0, 300.0, 2.0)]

    def buffers():
        bf, f32 = dict(dtype=torch.bfloat16, device="cuda"), dict(dtype=torch.float32, device="cuda")
        u8 = dict(dtype=torch.uint8, device="cuda")
        return dict(g=torch.ones(1, **f32), inv=torch.ones(1, **f32), amax=torch.zeros(1, **f32), rstd=torch.zeros(rows, **f32),
                    dg=torch.zeros(C, **f32), D=[torch.zeros(rows, C, **bf) for _ in range(3)], h=torch.zeros(rows, C, **bf),
                    dh=torch.zeros(rows, C, **bf), q8=torch.zeros(rows, C, **u8),
                    q=torch.zeros(rows, C // 2, **u8), sf=torch.zeros(cuda_lib.fp4_scale_bytes(rows, C, Q_NVFP4), **u8),
                    ws=torch.zeros(cuda_lib.fp8_rmsnorm_backward_workspace_bytes(rows, C), **u8))

    def product(b, w, D):
        cuda_lib.fp4_gemm_multi([dict(A=b["q"], a_sf=b["sf"], B=W[w][0], b_sf=W[w][1], quant=Q_NVFP4, D=D,
                                      a_scale_inv=b["inv"])])

    def calls(b):
        D = b["D"]
        return [
            lambda: cuda_lib.fp4_cast_multi([dict(x=x, quant=Q_NVFP4, q_row=b["q"], sf_row=b["sf"], scale=b["g"],
                                                  scale_inv=b["inv"])]),
            lambda: product(b, 0, D[0]),
            lambda: cuda_lib.fp8_rmsnorm_cast(D[0], gamma, 1e-5, residual=x, h=b["h"], rstd=b["rstd"], quant=Q_FP8, fmt=E4M3,
                                              q=b["q8"], scale=b["inv"], amax=b["amax"], scale_inv=b["g"]),
            lambda: cuda_lib.fp8_rmsnorm_cast(D[0], gamma, 1e-5, residual=x, h=b["h"], rstd=b["rstd"], quant=Q_NVFP4,
                                              q=b["q"], sf=b["sf"], scale=b["g"], scale_inv=b["inv"]),
            lambda: product(b, 1, D[1]),
            lambda: cuda_lib.fp8_rmsnorm_backward(D[1], b["h"], gamma, b["rstd"], b["dh"], dres=x, dgamma=b["dg"],
                                                  workspace=b["ws"]),
            lambda: cuda_lib.fp4_cast_multi([dict(x=b["dh"], quant=Q_NVFP4, q_row=b["q"], sf_row=b["sf"], scale=b["inv"],
                                                  scale_inv=b["g"])]),
            lambda: cuda_lib.fp4_gemm_multi([dict(A=b["q"], a_sf=b["sf"], B=W[0][0], b_sf=W[0][1], quant=Q_NVFP4, D=D[2],
                                                  a_scale_inv=b["g"])]),
        ]
    keep = ("dg", "rstd", "h", "dh", "q", "sf", "q8", "amax", "g", "inv")
    alone, want = buffers(), []
    for s in scales:
        alone["g"].copy_(s)
        for call in calls(alone):
            torch.cuda.synchronize()
            call()
        torch.cuda.synchronize()
        want.append([alone[k].clone() for k in keep] + [d.clone() for d in alone["D"]])
    assert not torch.equal(want[0][keep.index("inv")], want[1][keep.index("inv")])

    b = buffers()
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=stream):
        for call in calls(b):
            call()
    got = []
    b["amax"].zero_()
    for s in scales:                                     # nothing waits between the replays
        b["g"].copy_(s)
        graph.replay()
        got.append([b[k].clone() for k in keep] + [d.clone() for d in b["D"]])
    torch.cuda.synchronize()
    cuda_lib.fp8t_check_device_error()
    for w, o in zip(want, got):
        for a, c in zip(w, o):
            assert torch.equal(a.view(torch.uint8), c.view(torch.uint8))


def backward_inputs(rows, cols):
    g = torch.Generator().manual_seed(rows)
    h, dy = (torch.randn(rows, cols, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    gamma = (1 + 0.1 * torch.randn(cols, generator=g)).to(torch.bfloat16).cuda()
    rstd = (torch.rand(rows, generator=g) + 0.5).cuda()
    return dy, h, gamma, rstd, torch.empty_like(h)


def test_backward_takes_its_workspace_from_the_stream_it_runs_on(cuda_lib):
    """The allocator keeps freed blocks per stream: a block that the current stream freed may still be in use there, so
    a call on another stream must not be given it."""
    rows, cols = 700, 1024
    args = backward_inputs(rows, cols)
    need = cuda_lib.fp8_rmsnorm_backward_workspace_bytes(rows, cols)

    def bytes_reserved(stream):
        return sum(s["total_size"] for s in torch.cuda.memory_snapshot() if s["stream"] == stream.cuda_stream)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    side = next(s for s in (torch.cuda.Stream() for _ in range(64)) if bytes_reserved(s) == 0)
    cuda_lib.fp8_rmsnorm_backward(*args, dgamma=torch.empty(cols, device="cuda"), stream=side)
    torch.cuda.synchronize()
    assert bytes_reserved(side) >= need


def test_backward_beside_work_on_just_freed_memory(cuda_lib):
    """The current stream is busy with temporaries of the workspace's size that Python has freed already; neither they
    nor dgamma of the call on another stream may change."""
    rows, cols = 700, 1024
    args = backward_inputs(rows, cols)
    n = cuda_lib.fp8_rmsnorm_backward_workspace_bytes(rows, cols)
    want = torch.empty(cols, device="cuda")
    cuda_lib.fp8_rmsnorm_backward(*args, dgamma=want)
    side = torch.cuda.Stream()
    got = [torch.empty(cols, device="cuda") for _ in range(8)]
    sums = torch.zeros(8, device="cuda")
    torch.cuda.synchronize()
    for i in range(8):
        t = torch.full((n // 4,), float(i + 1), device="cuda")
        torch.cuda._sleep(2_000_000)                     # about a millisecond: t is read long after it was freed
        sums[i] = t.min() + t.max()
        del t
        cuda_lib.fp8_rmsnorm_backward(*args, dgamma=got[i], stream=side)
    torch.cuda.synchronize()
    cuda_lib.fp8t_check_device_error()
    assert sums.tolist() == [2.0 * (i + 1) for i in range(8)]
    assert all(torch.equal(g, want) for g in got)


def test_backward_captured_on_the_stream_it_is_given(cuda_lib):
    """The workspace is then the graph's; eager calls on the same stream between replays change nothing."""
    rows, cols = 700, 1024
    args, other = backward_inputs(rows, cols), backward_inputs(rows, cols)
    want, got, eager = (torch.empty(cols, device="cuda") for _ in range(3))
    cuda_lib.fp8_rmsnorm_backward(*args, dgamma=want)
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=s):
        cuda_lib.fp8_rmsnorm_backward(*args, dgamma=got, stream=s)
    for _ in range(3):
        got.fill_(float("nan"))
        graph.replay()
        s.wait_stream(torch.cuda.current_stream())
        cuda_lib.fp8_rmsnorm_backward(other[1], other[0], *other[2:], dgamma=eager, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(got, want)
