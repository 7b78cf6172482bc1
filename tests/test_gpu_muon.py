"""Newton-Schulz steps and the Muon step against 64 bits (bounds in tests/_feed_forward.py: orth_bounds)."""
import math

import pytest
import torch

from tests import _feed_forward as ff
from tests.test_gpu_timeout import _run_expired

pytestmark = pytest.mark.gpu
SIZES = [(1, 1), (1, 7), (7, 1), (8, 8), (31, 33), (64, 200), (200, 64), (255, 257), (256, 512), (512, 256), (300, 700), (701, 333),
         (1030, 523), (520, 1031), (16, 3000), (3000, 16), (1300, 1300)]


def matrix(rows, cols, seed, scale=1.0):
    """Noise and a few strong directions."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    n = torch.randn(rows, cols, generator=gen, device="cuda")
    s = torch.randn(rows, 2, generator=gen, device="cuda") @ torch.randn(2, cols, generator=gen, device="cuda")
    return (n + 0.5 * s) * scale


def guarded(t, dtype=None):
    view, check = ff.guarded(t.shape[0], t.shape[1], dtype or t.dtype)
    view.copy_(t)
    return view, check


def check_orth(got, x, steps=5):
    want, norm, most = ff.orth_bounds(x.double(), steps)
    d = (got.double() - want).abs()
    rounding = ff.BF16 * want.abs()
    assert float(d.norm()) <= float(norm) + float(rounding.norm())
    assert bool((d <= most + rounding + ff.BF16 * most).all())


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_orthogonalize(cuda_lib, rows, cols, f32):
    x = matrix(rows, cols, rows + cols)
    x = x if f32 else x.to(torch.bfloat16)
    out, check = guarded(torch.zeros_like(x, dtype=torch.bfloat16))
    cuda_lib.muon_orthogonalize([x], [out])
    cuda_lib.fp8t_check_device_error()
    check()
    check_orth(out, x)


@pytest.mark.parametrize("steps", [1, 2, 3, 4, 8])
def test_steps(cuda_lib, steps):
    for rows, cols in ((70, 300), (300, 70)):
        x = matrix(rows, cols, steps)
        out = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
        cuda_lib.muon_orthogonalize([x], [out], steps=steps)
        check_orth(out, x, steps)


@pytest.mark.parametrize("scale", [1e-38, 1e-25, 1e25, 1e36])
def test_any_magnitude(cuda_lib, scale):
    """|x|^2 does not fit f32; its factors do."""
    x = matrix(100, 260, 1, scale)
    out = torch.empty(100, 260, dtype=torch.bfloat16, device="cuda")
    cuda_lib.muon_orthogonalize([x], [out])
    check_orth(out, x)


def test_zero_nan_infinite(cuda_lib):
    xs = [torch.zeros(40, 50, device="cuda"), matrix(40, 50, 2), matrix(40, 50, 3), matrix(40, 50, 4)]
    xs[1][3, 4] = math.nan
    xs[2][39, 49] = math.inf
    outs = [torch.empty(40, 50, dtype=torch.bfloat16, device="cuda") for _ in xs]
    cuda_lib.muon_orthogonalize(xs, outs)
    assert bool((outs[0] == 0).all()) and bool(outs[1].isnan().all()) and bool(outs[2].isnan().all())
    check_orth(outs[3], xs[3])


def test_singular_matrix(cuda_lib):
    """Rank 3 of 60: the other directions stay zero but for the roundings, which grow no faster than the rest."""
    x = (torch.randn(60, 3, device="cuda", dtype=torch.float64) @ torch.randn(3, 90, device="cuda", dtype=torch.float64)).float()
    out = torch.empty(60, 90, dtype=torch.bfloat16, device="cuda")
    cuda_lib.muon_orthogonalize([x], [out])
    check_orth(out, x)


def test_list_in_place_and_same_bits(cuda_lib):
    """30 matrices (two tables), over themselves, twice; alone they give the same."""
    shapes = [(1 + 13 * i, 400 - 11 * i) for i in range(30)]
    xs = [matrix(r, c, i).to(torch.bfloat16) for i, (r, c) in enumerate(shapes)]
    a, b = [x.clone() for x in xs], [x.clone() for x in xs]
    ws = torch.empty(cuda_lib.muon_workspace_bytes(shapes), dtype=torch.uint8, device="cuda")
    cuda_lib.muon_orthogonalize(a, a, workspace=ws)
    ws.fill_(0xFF)                                             # NaN everywhere: nothing of it may be read
    cuda_lib.muon_orthogonalize(b, b, workspace=ws)
    for i in (0, 7, 23, 24, 29):
        check_orth(a[i], xs[i])
        alone = torch.empty_like(xs[i])
        cuda_lib.muon_orthogonalize([xs[i]], [alone])
        assert torch.equal(alone, a[i])
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def state(shapes, seed=0, loss_scale=64.0):
    s = dict(p=[], m=[], g=[], w=[])
    checks = []
    for i, (r, c) in enumerate(shapes):
        for k, t in (("p", matrix(r, c, seed + 4 * i, 0.02)), ("m", matrix(r, c, seed + 4 * i + 1, 1e-3)),
                     ("g", (matrix(r, c, seed + 4 * i + 2, 1e-3) * loss_scale).to(torch.bfloat16)),
                     ("w", torch.zeros(r, c, dtype=torch.bfloat16, device="cuda"))):
            v, check = guarded(t)
            s[k].append(v)
            checks.append(check)
    return s, checks


def step(fp8, s, **kw):
    a = dict(lr=1e-2, beta=0.9, weight_decay=0.1, update_rms=0.2, loss_scale=64.0)
    a.update(kw)
    fp8.fused_muon_multi_tensor(s["p"], s["m"], s["g"], s["w"], **a)


def check_step(s, old, lr=1e-2, beta=0.9, wd=0.1, rms=0.2, S=64.0, nesterov=True, steps=5):
    f = torch.float32
    for p, m, g, w, p0, m0 in zip(s["p"], s["m"], s["g"], s["w"], old["p"], old["m"]):
        gu = g.to(f) * torch.tensor(1.0 / S, dtype=f)
        want_m = m0 * torch.tensor(beta, dtype=f) + gu
        assert torch.equal(m, want_m)
        u = want_m * torch.tensor(beta, dtype=f) + gu if nesterov else want_m
        o, norm, most = ff.orth_bounds(u.double(), steps)
        rate = lr * rms * math.sqrt(max(p.shape))
        want = p0.double() * (1 - lr * wd) - rate * o
        d = (p.double() - want).abs()
        f32 = 2.0 ** -22 * (p0.double().abs() + rate * o.abs())
        assert float(d.norm()) <= rate * float(norm) + float(f32.norm())
        assert bool((d <= rate * most + f32).all())
        assert torch.equal(w, p.to(torch.bfloat16))


@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("shapes", [[(64, 64)], [(1, 1), (3, 5), (257, 130)], [(300, 520), (520, 300), (33, 1000), (1000, 33), (128, 128)],
                                    [(8 + i, 40 - i) for i in range(27)]])
def test_step(cuda_lib, shapes, nesterov):
    s, checks = state(shapes)
    old = {k: [t.clone() for t in v] for k, v in s.items()}
    skipped = torch.full((1,), 7, dtype=torch.int32, device="cuda")
    step(cuda_lib, s, nesterov=nesterov, skipped=skipped)
    cuda_lib.fp8t_check_device_error()
    for c in checks:
        c()
    assert skipped.item() == 0
    check_step(s, old, nesterov=nesterov)


@pytest.mark.parametrize("where,value", [("g", math.nan), ("g", math.inf), ("m", math.nan)])
def test_a_non_finite_tensor_skips_the_step(cuda_lib, where, value):
    s, _ = state([(40, 60), (100, 30), (16, 16)] + [(8, 8)] * 25)
    s[where][27][7, 7] = value                                 # in the second table
    old = {k: [t.clone() for t in v] for k, v in s.items()}
    skipped = torch.zeros(1, dtype=torch.int32, device="cuda")
    step(cuda_lib, s, skipped=skipped)
    assert skipped.item() == 1
    for k in "pmw":
        for a, b in zip(s[k], old[k]):
            assert torch.equal(a.view(torch.uint8 if k == "w" else torch.int32), b.view(torch.uint8 if k == "w" else torch.int32))


def test_zero_gradient(cuda_lib):
    s, _ = state([(40, 60)])
    s["g"][0].zero_()
    s["m"][0].zero_()
    old = s["p"][0].clone()
    step(cuda_lib, s)
    assert torch.equal(s["p"][0], old * torch.tensor(1 - 1e-2 * 0.1, dtype=torch.float32)) and bool((s["m"][0] == 0).all())


def test_captured_steps(cuda_lib):
    """A graph's replays are steps; two graphs with workspaces of their own do not disturb each other."""
    shapes = [(200, 330), (64, 64)]
    a, _ = state(shapes, 1)
    b, _ = state(shapes, 1)
    c, _ = state(shapes, 2)
    n = cuda_lib.muon_workspace_bytes(shapes)
    ws = [torch.empty(n, dtype=torch.uint8, device="cuda") for _ in range(2)]
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    for graph, s, w in zip(graphs, (a, c), ws):
        with torch.cuda.graph(graph):
            step(cuda_lib, s, workspace=w)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(3):
        for graph, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                graph.replay()
    torch.cuda.synchronize()
    for _ in range(3):
        step(cuda_lib, b)
    for k in "pmw":
        assert all(torch.equal(x, y) for x, y in zip(a[k], b[k]))


def test_another_stream_allocates_there(cuda_lib):
    s, _ = state([(64, 96)], 3)
    t, _ = state([(64, 96)], 3)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(cuda_lib, s, stream=side)
    step(cuda_lib, t)
    side.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(s["p"][0], t["p"][0])


@pytest.mark.parametrize("rows,cols", [(2, 256), (256, 2), (64, 64), (65, 129), (129, 65), (128, 256), (256, 128), (255, 255), (256, 256),
                                       (200, 256), (256, 257), (257, 3)])
def test_one_pair_holds_up_to_256(cuda_lib, rows, cols):
    """The form that keeps a matrix in shared memory, at the edges of its blocks, and its neighbours past them."""
    for steps in (1, 2, 5):
        x = matrix(rows, cols, 3 * rows + cols + steps)
        out, check = guarded(torch.zeros_like(x, dtype=torch.bfloat16))
        cuda_lib.muon_orthogonalize([x], [out], steps=steps)
        cuda_lib.fp8t_check_device_error()
        check()
        check_orth(out, x, steps)


@pytest.mark.parametrize("rows,cols", [(600, 700), (200, 130)])
@pytest.mark.parametrize("mode", [1, 2])
def test_waits_expire_and_context_survives(cuda_lib, mode, rows, cols):
    """A product that gave up leaves p and w alone; the next step is right."""
    s, _ = state([(rows, cols)])
    old = {k: [t.clone() for t in v] for k, v in s.items()}
    skipped = torch.zeros(1, dtype=torch.int32, device="cuda")
    _run_expired(cuda_lib, mode, lambda: step(cuda_lib, s, skipped=skipped))
    assert skipped.item() == 1 and torch.equal(s["p"][0], old["p"][0]) and torch.equal(s["w"][0], old["w"][0])
    old = {k: [t.clone() for t in v] for k, v in s.items()}
    step(cuda_lib, s, skipped=skipped)
    cuda_lib.fp8t_check_device_error()
    assert skipped.item() == 0
    check_step(s, old)


@pytest.mark.parametrize("scale", [1e-38, 1e-25, 1.0, 1e25, 1e36])
@pytest.mark.parametrize("rows,cols", [(100, 200), (200, 100), (256, 256), (3, 5)])
def test_any_magnitude_in_shared_memory(cuda_lib, rows, cols, scale):
    """Squares past f32 in some rows, in all, and below it, beside rows of zeros."""
    for spread in (False, True):
        x = matrix(rows, cols, 7, scale)
        if spread:
            x = x * torch.logspace(-20, 0, rows, device="cuda")[:, None]
            x[rows // 2] = 0
        out = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
        cuda_lib.muon_orthogonalize([x], [out])
        cuda_lib.fp8t_check_device_error()
        check_orth(out, x)


def test_small_and_large_in_one_list(cuda_lib):
    """Matrices of both forms in every batch of a long list, some in place, and the bits that each has alone."""
    shapes = [(64, 64), (300, 70), (256, 256), (70, 300), (1, 9), (255, 257), (40, 250)] * 8
    xs = [matrix(r, c, i).to(torch.bfloat16) for i, (r, c) in enumerate(shapes)]
    alone = []
    for x in xs:
        out = torch.empty_like(x)
        cuda_lib.muon_orthogonalize([x], [out], steps=3)
        alone.append(out)
    outs = [x.clone() if i % 3 == 0 else torch.empty_like(x) for i, x in enumerate(xs)]
    cuda_lib.muon_orthogonalize([o if i % 3 == 0 else x for i, (x, o) in enumerate(zip(xs, outs))], outs, steps=3)
    cuda_lib.fp8t_check_device_error()
    for i in range(len(xs)):
        assert torch.equal(outs[i], alone[i]), shapes[i]


def test_small_ones_on_two_streams_and_captured(cuda_lib):
    """Calls at the same time on two streams, those of one replayed from a graph: each has its own results."""
    xs = [matrix(200, 256, i).to(torch.bfloat16) for i in range(4)]
    want = [torch.empty_like(x) for x in xs]
    for x, w in zip(xs, want):
        cuda_lib.muon_orthogonalize([x], [w])
    torch.cuda.synchronize()
    outs = [torch.zeros_like(x) for x in xs]
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph):
        for x, o in zip(xs[:2], outs[:2]):
            cuda_lib.muon_orthogonalize([x], [o])
    for _ in range(20):
        graph.replay()
        with torch.cuda.stream(side):
            for x, o in zip(xs[2:], outs[2:]):
                cuda_lib.muon_orthogonalize([x], [o])
    torch.cuda.synchronize()
    cuda_lib.fp8t_check_device_error()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)


@pytest.mark.parametrize("rows,cols", [(600, 700), (200, 130), (130, 200), (255, 33)])
@pytest.mark.parametrize("mode", [1, 2])
def test_orthogonalize_waits_expire(cuda_lib, mode, rows, cols):
    """The result of a product that gave up is NaN throughout; the next call is right."""
    x = matrix(rows, cols, 1)
    out, check = guarded(torch.zeros_like(x, dtype=torch.bfloat16))
    _run_expired(cuda_lib, mode, lambda: cuda_lib.muon_orthogonalize([x], [out]))
    check()
    assert bool(out.isnan().all())
    cuda_lib.muon_orthogonalize([x], [out])
    cuda_lib.fp8t_check_device_error()
    check_orth(out, x)
