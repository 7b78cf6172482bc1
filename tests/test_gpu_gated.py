"""The gated feed-forward product and its gradient against the 64-bit formulas (bounds in tests/_feed_forward.py)."""
import pytest
import torch

from tests import _feed_forward as ff
from tests.test_gpu_timeout import _run_expired

pytestmark = pytest.mark.gpu
E4, E5 = torch.float8_e4m3fn, torch.float8_e5m2
FMT = {E4: 0, E5: 1}
ACT = {"silu": 1, "gelu": 2}
# one row; less than a tile; edges of tiles in each direction; several tiles and runs of tiles; K below and past a k-block
SIZES = [(1, 16, 16), (5, 64, 16), (127, 272, 48), (128, 128, 128), (129, 400, 208), (257, 144, 272), (300, 1024, 320),
         (2100, 144, 400), (513, 4096, 144), (1, 4096, 1040)]


def codes(shape, kind, seed, sigma=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(shape, generator=gen, device="cuda") * sigma
    return x.clamp(-ff.TOP[kind], ff.TOP[kind]).to(kind).view(torch.uint8)


def scalar(v):
    return torch.full((1,), float(v), device="cuda")


def value(c, kind):
    return c.view(kind).double()


def forward(fp8, M, K, N, act, b_mn, kinds=(E4, E4), qk=E4, seed=0, a=None, w=None, inv=(0.5, 0.03), scale=16.0, outs="ghq"):
    a = codes((M, K), kinds[0], seed) if a is None else a
    w = codes((2 * N, K), kinds[1], seed + 1) if w is None else w
    b = w.T.contiguous() if b_mn else w
    o, checks = {}, []
    for name, key, cols, dtype in (("g", "gu", 2 * N, torch.bfloat16), ("h", "h", N, torch.bfloat16), ("q", "q", N, torch.uint8)):
        if name in outs:
            o[key], c = ff.guarded(M, cols, dtype)
            checks.append(c)
    if "q" in outs:
        o["scale"], o["scale_inv"] = scalar(scale), scalar(0)
    o["amax"] = scalar(0)
    fp8.fp8_gated_gemm(a, FMT[kinds[0]], b, FMT[kinds[1]], scalar(inv[0]), scalar(inv[1]), act=ACT[act], b_mn=b_mn,
                       q_fmt=FMT[qk], **o)
    fp8.fp8t_check_device_error()
    for c in checks:
        c()
    unit = float(torch.tensor(inv[0]) * torch.tensor(inv[1]))
    return o, ff.gated(value(a, kinds[0]), value(w, kinds[1]), unit, act)


def check_forward(o, want, qk=E4, scale=16.0):
    gu, off, h, oh = want
    if "gu" in o:
        assert ff.within(o["gu"], gu, off, ff.BF16)
    if "h" in o:
        assert ff.within(o["h"], h, oh, ff.BF16)
    if "q" in o:
        assert ff.codes_within(o["q"], h, oh, scale, qk)
        assert o["scale_inv"].item() == (1.0 / torch.tensor(scale)).item()
    at = h.abs().argmax()
    assert abs(o["amax"].item() - h.abs().max().item()) <= oh.max().item()
    assert o["amax"].item() >= (h.abs().flatten()[at] - oh.flatten()[at]).item()


@pytest.mark.parametrize("b_mn", [False, True])
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("M,K,N", SIZES)
def test_forward(cuda_lib, M, K, N, act, b_mn):
    check_forward(*forward(cuda_lib, M, K, N, act, b_mn))


@pytest.mark.parametrize("b_mn", [False, True])
@pytest.mark.parametrize("kinds", [(E4, E4), (E4, E5), (E5, E4), (E5, E5)])
@pytest.mark.parametrize("M,K,N", [(1, 16, 16), (2, 48, 48), (7, 80, 64), (8, 512, 80), (9, 96, 112), (15, 1040, 144), (16, 4096, 176),
                                   (17, 112, 96), (32, 256, 688), (33, 256, 688), (16, 4096, 1040), (3, 2064, 1008)])
def test_few_rows(cuda_lib, M, K, N, kinds, b_mn):
    """Up to 8 rows, or 32 of few weights: another kernel, with and without a transpose of W's bytes; K that ends inside a chunk, idle warps."""
    check_forward(*forward(cuda_lib, M, K, N, "silu" if N % 32 else "gelu", b_mn, kinds=kinds))


@pytest.mark.parametrize("M", [1, 8])
@pytest.mark.parametrize("N,K", [(4720, 48), (4752, 48), (9472, 272), (9488, 272), (14208, 48), (14224, 48), (18944, 144), (18960, 48),
                                 (28672, 80), (40000, 16)])
@pytest.mark.parametrize("kinds", [(E4, E4), (E5, E4)])
def test_few_rows_wide_transposed(cuda_lib, M, N, K, kinds):
    """W as [K][2N] with tiles of 32, 64, 96 and 128 outputs, in one round of the SMs and more; N that ends inside a tile."""
    o, want = forward(cuda_lib, M, K, N, "silu", True, kinds=kinds, seed=N + M)
    check_forward(o, want)


@pytest.mark.parametrize("b_mn", [False, True])
@pytest.mark.parametrize("M", [9, 17, 31, 33, 100, 127, 128])
def test_less_than_a_cta_of_rows(cuda_lib, M, b_mn):
    """Rows that fill part of a box, behind a call whose operands leave NaN codes in shared memory: none reaches an output."""
    K, N = 528, 48 if M > 32 else 40000
    a = torch.full((256, K), 0x7F, dtype=torch.uint8, device="cuda")
    forward(cuda_lib, 256, K, 4736, "silu", b_mn, a=a, w=torch.full((2 * 4736, K), 0x7F, dtype=torch.uint8, device="cuda"))
    check_forward(*forward(cuda_lib, M, K, N, "silu", b_mn))
    if N == 48:
        check_backward(*backward(cuda_lib, M, K, N, "gelu", b_mn))


@pytest.mark.parametrize("M,K,N", [(300, 256, 2768), (1237, 144, 2752), (1000, 272, 5504), (40, 144, 11008), (500, 144, 4160)])
@pytest.mark.parametrize("kinds", [(E4, E4), (E4, E5)])
def test_tiles_of_192_columns(cuda_lib, M, K, N, kinds):
    """Tiles of three quarters of the columns, where they make the clusters' rounds shorter."""
    o, want = forward(cuda_lib, M, K, N, "gelu", False, kinds=kinds, seed=N)
    check_forward(o, want)


@pytest.mark.parametrize("M,K,N", [(1000, 272, 5504), (300, 144, 11008), (1000, 144, 2768), (40, 400, 16400)])
@pytest.mark.parametrize("inplace", [False, True])
def test_backward_tiles_of_192_columns(cuda_lib, M, K, N, inplace):
    check_backward(*backward(cuda_lib, M, K, N, "silu", False, inplace=inplace))

@pytest.mark.parametrize("outs", ["g", "h", "q", "gq", "gh"])
def test_few_rows_outputs_alone(cuda_lib, outs):
    for b_mn in (False, True):
        check_forward(*forward(cuda_lib, 6, 272, 144, "silu", b_mn, outs=outs))


def test_few_rows_nan_and_infinite_operands(cuda_lib):
    for b_mn in (False, True):
        M, K, N = 11, 272, 80
        a, w = codes((M, K), E4, 5), codes((2 * N, K), E5, 6)
        a[a.view(E4).float() == 0] = 0x38
        w[3, 7] = 0x7C                                         # an infinite gate weight: column 3, or 0 where the gate is -inf
        a[9, 5] = 0x7F
        o, _ = forward(cuda_lib, M, K, N, "silu", b_mn, kinds=(E4, E5), a=a, w=w)
        good = torch.ones(M, dtype=torch.bool, device="cuda")
        good[9] = False
        assert bool(o["h"][9].isnan().all()) and bool((o["q"][9] == 0x7F).all()) and o["amax"].isnan().item()
        assert bool(o["h"][good][:, :3].isfinite().all()) and bool(o["h"][good][:, 4:].isfinite().all())
        assert not bool(o["h"][good][:, 3].isfinite().any())


@pytest.mark.parametrize("outs", ["g", "h", "q", "gq", "gh"])
def test_forward_outputs_alone(cuda_lib, outs):
    check_forward(*forward(cuda_lib, 140, 256, 144, "silu", True, outs=outs))


@pytest.mark.parametrize("kinds,qk", [((E4, E5), E5), ((E5, E4), E4), ((E5, E5), E5)])
def test_forward_formats(cuda_lib, kinds, qk):
    o, want = forward(cuda_lib, 70, 320, 80, "gelu", False, kinds=kinds, qk=qk)
    check_forward(o, want, qk)


def test_forward_saturates_and_accumulates_amax(cuda_lib):
    o, want = forward(cuda_lib, 64, 128, 64, "silu", False, scale=1e6)
    check_forward(o, want, scale=1e6)
    assert o["q"].view(E4).float().abs().max().item() == 448.0
    a, w = codes((3, 64), E4, 1), codes((32, 64), E4, 2)
    amax = scalar(1e9)
    h = torch.empty(3, 16, dtype=torch.bfloat16, device="cuda")
    cuda_lib.fp8_gated_gemm(a, 0, w, 0, scalar(1), scalar(1), h=h, amax=amax)
    assert amax.item() == 1e9


def test_forward_nan_and_infinite_operands(cuda_lib):
    M, K, N = 300, 256, 144
    a, w = codes((M, K), E4, 5), codes((2 * N, K), E5, 6)
    a[7, 3] = 0x7F                                             # NaN: row 7
    o, _ = forward(cuda_lib, M, K, N, "silu", False, kinds=(E4, E5), a=a, w=w)
    assert bool(o["h"][7].isnan().all()) and not bool(o["h"][:7].isnan().any()) and not bool(o["h"][8:].isnan().any())
    assert bool((o["q"][7] == 0x7F).all()) and o["amax"].isnan().item()
    # an infinite up weight in the last column: rows and columns past the edge hold 0 * inf, which amax must not see
    a = codes((M, K), E4, 5)
    a[a.view(E4).float() == 0] = 0x38
    w[2 * N - 1, 0] = 0x7C
    o, _ = forward(cuda_lib, M, K, N, "silu", False, kinds=(E4, E5), a=a, w=w)
    assert bool(o["h"][:, -1].isinf().all()) and bool(o["h"][:, :-1].isfinite().all()) and o["amax"].item() == float("inf")


def backward(fp8, M, K, N, act, b_mn, qk=E5, seed=0, sigma=1.5, scale=64.0, outs="dq", inplace=False, kinds=(E5, E4)):
    a, w = codes((M, K), kinds[0], seed), codes((N, K), kinds[1], seed + 1)
    gen = torch.Generator(device="cuda").manual_seed(seed + 2)
    gu, check = ff.guarded(M, 2 * N, torch.bfloat16)
    gu.copy_(torch.randn(M, 2 * N, generator=gen, device="cuda") * sigma)
    kept = gu.double()
    o, checks = {}, [check]
    if "d" in outs:
        o["dgu"], c = (gu, check) if inplace else ff.guarded(M, 2 * N, torch.bfloat16)
        checks.append(c)
    if "q" in outs:
        o["q"], c = ff.guarded(M, 2 * N, torch.uint8)
        checks.append(c)
        o["scale"], o["scale_inv"] = scalar(scale), scalar(0)
    o["amax"] = scalar(0)
    fp8.fp8_gated_gemm_backward(a, FMT[kinds[0]], w.T.contiguous() if b_mn else w, FMT[kinds[1]], scalar(0.25), scalar(0.05), gu,
                                act=ACT[act], b_mn=b_mn, q_fmt=FMT[qk], **o)
    fp8.fp8t_check_device_error()
    for c in checks:
        c()
    unit = float(torch.tensor(0.25) * torch.tensor(0.05))
    return o, ff.gated_backward(value(a, kinds[0]), value(w, kinds[1]), unit, kept, act)


def check_backward(o, want, qk=E5, scale=64.0):
    d, off = want
    if "dgu" in o:
        assert ff.within(o["dgu"], d, off, ff.BF16)
    if "q" in o:
        assert ff.codes_within(o["q"], d, off, scale, qk)
        assert o["scale_inv"].item() == (1.0 / torch.tensor(scale)).item()
    assert abs(o["amax"].item() - d.abs().max().item()) <= off.max().item()


@pytest.mark.parametrize("b_mn", [False, True])
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("M,K,N", SIZES)
def test_backward(cuda_lib, M, K, N, act, b_mn):
    check_backward(*backward(cuda_lib, M, K, N, act, b_mn))


@pytest.mark.parametrize("outs,qk", [("d", E5), ("q", E5), ("q", E4)])
def test_backward_outputs_alone(cuda_lib, outs, qk):
    o, want = backward(cuda_lib, 140, 256, 144, "silu", False, outs=outs, qk=qk)
    check_backward(o, want, qk)


def test_backward_in_place(cuda_lib):
    check_backward(*backward(cuda_lib, 600, 256, 336, "gelu", False, inplace=True))


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_backward_of_large_gates(cuda_lib, act):
    """Where the sigmoid is 0 or 1 to f32, its exponential overflows, and g's square does."""
    M, N, K = 16, 64, 32
    a, w = codes((M, K), E5, 1), codes((N, K), E4, 2)
    gu = torch.ones(M, 2 * N, dtype=torch.bfloat16, device="cuda")
    steps = torch.tensor([-3e38, -1e30, -1e20, -1e4, -200.0, -90.0, -30.0, -1e-30, 0.0, 1e-30, 30.0, 90.0, 200.0, 1e4, 1e20, 3e38])
    gu[:, :16] = steps.to(torch.bfloat16).cuda()
    d = torch.empty_like(gu)
    cuda_lib.fp8_gated_gemm_backward(a, 1, w, 0, scalar(1), scalar(1), gu, act=ACT[act], dgu=d)
    dh = value(a, E5) @ value(w, E4).T
    # dG = dh * u * act'(g): 0 for a gate far below zero, dh far above, and finite at both
    assert bool((d[:, :6].float().abs() <= 1e-30).all())
    assert ff.within(d[:, 10:16], dh[:, 10:16], 1e-4 * dh.abs()[:, 10:16] + 1e-3, ff.BF16)
    assert bool(d[:, :16].isfinite().all())


def test_streams_graph_and_repeat(cuda_lib):
    """On another stream than the inputs' own, captured and replayed, the same bits every time."""
    M, K, N = 300, 512, 272
    a, w = codes((M, K), E4, 1), codes((K, 2 * N), E4, 2)
    inv = scalar(0.1)
    want, _ = forward(cuda_lib, M, K, N, "silu", True, a=a, w=w.T.contiguous(), inv=(0.1, 0.1), outs="h")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    h = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    cuda_lib.fp8_gated_gemm(a, 0, w, 0, inv, inv, b_mn=True, h=h, stream=side)
    side.synchronize()
    assert torch.equal(h, want["h"])
    graph = torch.cuda.CUDAGraph()
    h2 = torch.zeros_like(h)
    with torch.cuda.graph(graph):
        cuda_lib.fp8_gated_gemm(a, 0, w, 0, inv, inv, b_mn=True, h=h2)
    for _ in range(2):
        h2.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(h2, want["h"])


@pytest.mark.parametrize("M,mode", [(600, 1), (600, 2), (5, 1)])
def test_waits_expire_and_context_survives(cuda_lib, M, mode):
    K, N = 512, 400
    a, w = codes((M, K), E4, 1), codes((2 * N, K), E4, 2)
    h = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    amax = scalar(0)
    wt = w.T.contiguous()
    _run_expired(cuda_lib, mode, lambda: cuda_lib.fp8_gated_gemm(a, 0, wt, 0, scalar(1), scalar(1), b_mn=True, h=h, amax=amax))
    assert amax.isnan().item()                                # a scale update keeps its scale
    check_forward(*forward(cuda_lib, M, K, N, "silu", True, a=a, w=w))
