"""The forms of the grid-wide Newton-Schulz kernel that model-sized matrices take. With 74 CTA pairs a list runs in tiles of 128
columns while those fit the pairs at once (all of A computed), then of 256 (all of A while it fits), then with the tiles above
the diagonal mirrored below it; past 74 tiles a pair has several in a phase; five matrices and more are another instantiation."""
import pytest
import torch

from tests import _feed_forward as ff
from tests.test_gpu_muon import check_orth, check_step, guarded, matrix, state, step

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("rows,cols", [
    (1500, 2309), (2309, 1500),                               # tiles of 256 columns, 36 of A, none mirrored
    (2100, 2050), (2050, 2100),                               # 81 of A: 45 on and above the diagonal; X in two rounds
    (2310, 2560), (2561, 2310),                               # 10 x 10 of X: rows and columns that end inside a tile, chunk and box
    (2305, 4100),                                             # a row tile of one row, 17 columns of tiles
    (4353, 2310)])
def test_orthogonalize(cuda_lib, rows, cols, f32):
    x = matrix(rows, cols, rows + cols)
    x = x if f32 else x.to(torch.bfloat16)
    out, check = guarded(torch.zeros_like(x, dtype=torch.bfloat16))
    cuda_lib.muon_orthogonalize([x], [out])
    cuda_lib.fp8t_check_device_error()
    check()
    check_orth(out, x)


@pytest.mark.parametrize("steps", [1, 2, 4])
def test_steps_mirrored(cuda_lib, steps):
    for rows, cols in ((2310, 2333), (2333, 2310)):
        x = matrix(rows, cols, steps)
        out = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
        cuda_lib.muon_orthogonalize([x], [out], steps=steps)
        check_orth(out, x, steps)


@pytest.mark.parametrize("shapes", [
    [(520, 4100), (4100, 520), (300, 333), (520, 2000), (700, 900)],                                      # 256 columns, all of A
    [(1030, 523)] * 4 + [(1100, 1200), (1200, 1100), (90, 2000), (2310, 1300), (40, 40), (256, 256)]])    # mirrored; and small ones
def test_list(cuda_lib, shapes):
    """Each as exact as alone, in place, and twice the same."""
    xs = [matrix(r, c, i).to(torch.bfloat16) for i, (r, c) in enumerate(shapes)]
    a, b = [x.clone() for x in xs], [x.clone() for x in xs]
    ws = torch.full((cuda_lib.muon_workspace_bytes(shapes),), 0xFF, dtype=torch.uint8, device="cuda")
    cuda_lib.muon_orthogonalize(a, a, workspace=ws)
    cuda_lib.muon_orthogonalize(b, b)
    cuda_lib.fp8t_check_device_error()
    for x, y, z in zip(xs, a, b):
        check_orth(y, x)
        assert torch.equal(y, z)


def test_step_with_the_weight_in_the_gradient(cuda_lib):
    """A list of every form; the new weight may take its gradient's place."""
    shapes = [(2310, 2333), (300, 1000), (200, 256), (33, 2000)]
    s, checks = state(shapes, 5)
    t, _ = state(shapes, 5)
    old = {k: [v.clone() for v in s[k]] for k in s}
    step(cuda_lib, s)
    t["w"] = t["g"]
    step(cuda_lib, t)
    cuda_lib.fp8t_check_device_error()
    for c in checks:
        c()
    check_step(s, old)
    for k in "pmw":
        assert all(torch.equal(x, y) for x, y in zip(s[k], t[k]))


@pytest.mark.parametrize("rows,cols", [(1, 65536), (65536, 1), (65536, 40), (24, 65536), (300, 65529), (65529, 300)])
def test_longest_sides(cuda_lib, rows, cols):
    x = matrix(rows, cols, 9)
    out, check = guarded(torch.zeros_like(x, dtype=torch.bfloat16))
    cuda_lib.muon_orthogonalize([x], [out])
    cuda_lib.fp8t_check_device_error()
    check()
    check_orth(out, x)


def test_captured_beside_an_eager_call(cuda_lib):
    """A replayed graph and an eager call on another stream, each with its own workspace: cooperative grids that do not fit the
    GPU together."""
    x = [matrix(2310, 2333, i).to(torch.bfloat16) for i in range(2)]
    want = [torch.empty_like(v) for v in x]
    for v, w in zip(x, want):
        cuda_lib.muon_orthogonalize([v], [w])
    torch.cuda.synchronize()
    outs = [torch.zeros_like(v) for v in x]
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph):
        cuda_lib.muon_orthogonalize([x[0]], [outs[0]])
    for _ in range(5):
        graph.replay()
        cuda_lib.muon_orthogonalize([x[1]], [outs[1]], stream=side)
    torch.cuda.synchronize()
    cuda_lib.fp8t_check_device_error()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))


def test_expected_bounds_hold_for_large_matrices():
    """The bound that the above are held to is a few thousandths of the factor, so that a tile left out or misplaced is seen."""
    x = matrix(1100, 1200, 1).double()
    want, norm, _ = ff.orth_bounds(x)
    assert float(norm) < 0.02 * float(want.norm())
