"""4-bit weights times a few tokens against 64 bits. Bounds: FP32 accumulation 1e-5 of sum |x w|, one rounding to BF16;
behind a gate as in tests/_feed_forward.py."""
import pytest
import torch

from tests import _feed_forward as ff

pytestmark = pytest.mark.gpu
ACT = {"none": 0, "silu": 1, "gelu": 2}


def weights(rows, k, nv, seed, lo=None, hi=None):
    """Random codes and scales: E8M0 near 2^-6 (or lo .. hi), E4M3 of any finite non-negative value."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    q = torch.randint(0, 256, (rows, k // 2), generator=gen, device="cuda", dtype=torch.uint8)
    lo, hi = (lo, hi) if lo is not None else ((0, 0x7F) if nv else (118, 126))
    s = torch.randint(lo, hi, (rows, k // (16 if nv else 32)), generator=gen, device="cuda", dtype=torch.uint8)
    return q, s


def run(fp8, M, K, N, nv, act, seed=0, x=None, q=None, s=None, inv=1e-4):
    outs = N if act == "none" else 2 * N
    gen = torch.Generator(device="cuda").manual_seed(seed + 7)
    x = torch.randn(M, K, generator=gen, device="cuda").to(torch.bfloat16) if x is None else x
    if q is None:
        q, s = weights(outs, K, nv, seed)
    sf = ff.atoms(s, nv)
    y, check = ff.guarded(M, N, torch.bfloat16)
    scale = torch.full((1,), inv, device="cuda") if nv else None
    fp8.fp4_matvec(x, q, sf, 4 if nv else 3, y, w_scale_inv=scale, act=ACT[act])
    torch.cuda.synchronize()
    check()
    w = ff.fp4_values(q, sf, outs, K, nv)
    unit = float(torch.tensor(inv)) if nv else 1.0
    if act == "none":
        want = (x.double() @ w.T) * unit
        off = ff.ACCUMULATE * (x.double().abs() @ w.abs().T) * unit + 2.0 ** -22 * want.abs()
        return y, want, off
    _, _, want, off = ff.gated(x.double(), w, unit, act)
    return y, want, off


@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
@pytest.mark.parametrize("nv", [False, True])
@pytest.mark.parametrize("M,K,N", [(1, 32, 8), (1, 64, 16), (2, 96, 24), (3, 160, 40), (4, 1024, 200), (5, 2080, 136), (7, 4096, 72),
                                   (8, 11008, 264), (1, 11008, 1000), (8, 288, 4096), (2, 4096, 4104)])
def test_product(cuda_lib, M, K, N, nv, act):
    y, want, off = run(cuda_lib, M, K, N, nv, act)
    assert ff.within(y, want, off, ff.BF16)


@pytest.mark.parametrize("M", range(1, 9))
@pytest.mark.parametrize("nv", [False, True])
def test_every_number_of_rows(cuda_lib, M, nv):
    y, want, off = run(cuda_lib, M, 544, 56, nv, "none", seed=M)
    assert ff.within(y, want, off, ff.BF16)


@pytest.mark.parametrize("lo,hi", [(0, 12), (126, 132), (140, 200), (1, 254)])
def test_scales_over_the_range_of_e8m0(cuda_lib, lo, hi):
    """Blocks down to 2^-127 (BF16 subnormals) and up to 2^126, on both sides of what one BF16 factor holds."""
    M, K, N = 3, 256, 64
    q, s = weights(N, K, False, 5, lo, hi)
    shift = 2.0 ** (-60 if hi > 200 else 40 if hi <= 12 else 0)
    x = (torch.randn(M, K, device="cuda") * shift).to(torch.bfloat16)
    y, want, off = run(cuda_lib, M, K, N, False, "none", x=x, q=q, s=s)
    assert ff.within(y, want, off, ff.BF16)


def test_scale_specials(cuda_lib):
    M, K, N = 2, 128, 16
    q, s = weights(N, K, False, 6)
    s[5, 2] = 255                                              # NaN block: its row alone
    y, _, _ = run(cuda_lib, M, K, N, False, "none", q=q, s=s)
    assert bool(y[:, 5].isnan().all()) and int(y.isnan().sum()) == M
    q, s = weights(N, K, True, 6)
    s[5, 2] = 0x7F
    s[3] = 0
    y, _, _ = run(cuda_lib, M, K, N, True, "none", q=q, s=s)
    assert bool(y[:, 5].isnan().all()) and int(y.isnan().sum()) == M and bool((y[:, 3] == 0).all())


def test_each_weight_alone(cuda_lib):
    """One x at a time picks one column of W exactly: every code, place and scale."""
    for nv in (False, True):
        K, N = 288, 24
        q, s = weights(N, K, nv, 8)
        w = ff.fp4_values(q, ff.atoms(s, nv), N, K, nv)
        for k0 in range(0, K, 8):
            x = torch.zeros(8, K, dtype=torch.bfloat16, device="cuda")
            x[torch.arange(8), k0 + torch.arange(8)] = 1.0
            y, _, _ = run(cuda_lib, 8, K, N, nv, "none", x=x, q=q, s=s, inv=1.0)
            assert torch.equal(y.double(), w[:, k0:k0 + 8].T.to(torch.bfloat16).double())


def test_what_the_cast_writes(cuda_lib):
    """Weights through fp4_cast_multi, with the tensor scale of NVFP4."""
    K, N = 512, 136
    w = (torch.randn(N, K, device="cuda") * 0.02).to(torch.bfloat16)
    x = torch.randn(4, K, device="cuda").to(torch.bfloat16)
    for nv in (False, True):
        quant = 4 if nv else 3
        q = torch.empty(N, K // 2, dtype=torch.uint8, device="cuda")
        sf = torch.empty(cuda_lib.fp4_scale_bytes(N, K, quant), dtype=torch.uint8, device="cuda")
        extra, inv = {}, None
        if nv:
            inv = torch.empty(1, device="cuda")
            extra = dict(scale=2688.0 / w.float().abs().amax().reshape(1), scale_inv=inv)
        cuda_lib.fp4_cast_multi([dict(x=w, quant=quant, q_row=q, sf_row=sf, **extra)])
        y = torch.empty(4, N, dtype=torch.bfloat16, device="cuda")
        cuda_lib.fp4_matvec(x, q, sf, quant, y, w_scale_inv=inv)
        v = ff.fp4_values(q, sf, N, K, nv) * (inv.double() if nv else 1.0)
        assert ff.within(y, x.double() @ v.T, ff.ACCUMULATE * (x.double().abs() @ v.abs().T), ff.BF16)
        # and near the weights themselves: a value is off by at most a quarter of its block's largest
        assert float((y.double() - x.double() @ w.double().T).norm() / (x.double() @ w.double().T).norm()) < 0.25


def test_stream_and_graph(cuda_lib):
    y, _, _ = run(cuda_lib, 3, 1024, 64, True, "silu", seed=3)
    gen = torch.Generator(device="cuda").manual_seed(10)
    x = torch.randn(3, 1024, generator=gen, device="cuda").to(torch.bfloat16)
    q, s = weights(128, 1024, True, 3)
    sf, inv = ff.atoms(s, True), torch.full((1,), 1e-4, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = torch.empty_like(y)
    cuda_lib.fp4_matvec(x, q, sf, 4, out, w_scale_inv=inv, act=1, stream=side)
    side.synchronize()
    assert torch.equal(out, y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cuda_lib.fp4_matvec(x, q, sf, 4, out, w_scale_inv=inv, act=1)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, y)
