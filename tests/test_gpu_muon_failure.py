"""A Muon step that ends between its launches, as when one of them fails on the host: a captured step is replayed without its
later kernels."""
import pytest
import torch

from tests.test_gpu_muon import check_step, state, step

pytestmark = pytest.mark.gpu


def replay_until(kernel, record):
    """Captures record() and replays its graph without the first kernel of that name and those behind it; the rest's names."""
    drv = pytest.importorskip("cuda.bindings.driver")

    def ok(r):
        assert r[0] == drv.CUresult.CUDA_SUCCESS, r[0]
        return r[1] if len(r) == 2 else r[1:]
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        record()
    raw = drv.CUgraph(graph.raw_cuda_graph())
    nodes, n = ok(drv.cuGraphGetNodes(raw, 64))
    names = {}
    for node in nodes[:n]:
        p = ok(drv.cuGraphKernelNodeGetParams(node))
        name = ok(drv.cuFuncGetName(p.func)) if int(p.func) else ok(drv.cuKernelGetName(p.kern))
        names[int(node)] = name.decode()
    order = [names[int(x)] for x in nodes[:n]]                # as captured
    at = next(i for i, x in enumerate(order) if kernel in x)
    for node in reversed(nodes[at:n]):
        assert drv.cuGraphDestroyNode(node)[0] == drv.CUresult.CUDA_SUCCESS
    graph.instantiate()
    graph.replay()
    torch.cuda.synchronize()
    return order[:at]


@pytest.mark.parametrize("shapes,products", [([(300, 260)], "k_pair_gemm"), ([(64, 100)], "k_muon_small")])
def test_a_step_without_its_products_counts_as_skipped(cuda_lib, shapes, products):
    s, _ = state(shapes)
    old = {k: [t.clone() for t in v] for k, v in s.items()}
    skipped = torch.full((1,), 7, dtype=torch.int32, device="cuda")
    kept = replay_until(products, lambda: step(cuda_lib, s, skipped=skipped))
    assert len(kept) == 3 and "k_muon_scale" in kept[2]
    assert skipped.item() == 1
    assert torch.equal(s["p"][0], old["p"][0]) and torch.equal(s["w"][0], old["w"][0])
    assert not torch.equal(s["m"][0], old["m"][0])            # as documented


def test_a_step_of_two_tables_without_the_second(cuda_lib):
    shapes = [(40, 24 + i) for i in range(26)]
    s, _ = state(shapes)
    old = {k: [t.clone() for t in v] for k, v in s.items()}
    skipped = torch.full((1,), 7, dtype=torch.int32, device="cuda")
    step(cuda_lib, s, skipped=skipped)                        # whole: both tables, 0
    assert skipped.item() == 0
    check_step(s, old)
    skipped.fill_(7)
    replay_until("k_muon_apply", lambda: step(cuda_lib, s, skipped=skipped))           # up to the first table's products
    assert skipped.item() == 1
