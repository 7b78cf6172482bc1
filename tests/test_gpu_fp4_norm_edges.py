"""The norm and 4-bit calls at the edges of what their documentation allows: scales without a sign or that
are not finite, lists that mix one- and two-way casts, calls on two streams at once and replayed graphs of
several calls, matrices of more than 2^31 elements. Bounds as in test_gpu_fp4.py and test_gpu_rmsnorm.py."""
import numpy as np
import pytest
import torch

from tests import _block_quant as bq
from tests._gpu import bf16_bits, bf16_from_bits, u8
from tests._pins import gemm_within_tolerance
from tests.test_gpu_fp4 import KINDS, cast, check_cast, operand, random_bits, reference
from tests.test_gpu_rmsnorm import MXFP4, NVFP4, U, bf, check, make, run

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ scales
@pytest.mark.parametrize("g", [0.0, -0.0, -1.0, -1e30])
def test_nvfp4_scale_not_above_zero_gives_zero_codes(cuda_lib, g):
    """The block scale has no sign: every scale byte is 0 and every code +-0, one and both ways."""
    bits = random_bits(64, 96, 21)
    bits[3, 5] = 0
    sign = (bits >> 15 << 3).astype(np.uint8)
    for col in (False, True):
        d = cast(cuda_lib, bits, bq.NVFP4, g, col=col, scale_inv=None)
        cuda_lib.fp4_cast_multi([d])
        assert not u8(d["sf_row"]).any() and np.array_equal(bq.unpack(u8(d["q_row"])), sign)
        if col:
            assert not u8(d["sf_col"]).any() and np.array_equal(bq.unpack(u8(d["q_col"])), sign.T)
        assert d["amax"].item() == bq.bf16_f64(bits & 0x7FFF).max()


@pytest.mark.parametrize("g", [np.inf, np.nan])
def test_nvfp4_scale_not_finite(cuda_lib, g):
    """An infinite g saturates the block scales (NaN where the block is zero), a NaN one makes them NaN."""
    bits = random_bits(64, 96, 22)
    bits[:, :16] = 0
    d = cast(cuda_lib, bits, bq.NVFP4, g, scale_inv=None)
    cuda_lib.fp4_cast_multi([d])
    for q, sf, b in ((d["q_row"], d["sf_row"], bits), (d["q_col"], d["sf_col"], np.ascontiguousarray(bits.T))):
        codes, s = bq.quantise(b, bq.NVFP4, g)
        assert np.array_equal(bq.unpack(u8(q)), codes) and np.array_equal(u8(sf), bq.atoms(s, bq.NVFP4))


@pytest.mark.parametrize("g", [0.0, -0.0, -2.0, np.nan])
@pytest.mark.parametrize("cols", [96, 2080])
def test_norm_nvfp4_scale_without_a_positive_value(cuda_lib, g, cols):
    x, _, gamma = make(5, cols, 3)
    o = run(cuda_lib, x, None, gamma, 1e-5, NVFP4, scale=g)
    s, pad = bq.from_atoms(u8(o["sf"]), 5, cols // 16, bq.NVFP4)
    assert (s == (0x7F if g != g else 0)).all() and not pad.any()
    if g == g:
        assert not (bq.unpack(u8(o["q"])) & 7).any()


# ------------------------------------------------------------------ lists
def test_cast_list_of_one_and_two_way_tensors(cuda_lib):
    """A launch with column-wise copies also takes tensors that want one copy only, of any number of rows."""
    ds, ref = [], []
    for i, (rows, cols, row, col) in enumerate([(37, 96, True, False), (64, 160, True, True), (96, 32, False, True),
                                                (1, 64, True, False), (129, 416, True, False), (160, 288, True, True)]):
        kind = KINDS[i % 2]
        bits = random_bits(rows, cols, 300 + i)
        ds.append(cast(cuda_lib, bits, kind, 2.0 + i, row=row, col=col))
        ref.append((bits, kind, 2.0 + i))
    cuda_lib.fp4_cast_multi(ds)
    cuda_lib.fp8t_check_device_error()
    for d, r in zip(ds, ref):
        check_cast(d, *r)


def test_cast_list_of_row_wise_tensors(cuda_lib):
    """Row-wise copies alone over two launches, each tensor with an amax slot of its own: from one row (one CTA's
    work, many to fill up its atoms) to many, and an all-zero one among them."""
    ds, ref = [], []
    for i, (rows, cols) in enumerate([(1, 4096), (3, 32), (700, 288), (128, 64), (1, 32), (2049, 1056), (64, 512), (5, 96), (300, 800)]):
        kind = bq.MXFP4 if i % 4 == 1 else bq.NVFP4
        bits = random_bits(rows, cols, 400 + i)
        if i == 6:
            bits[:] = 0
        ds.append(cast(cuda_lib, bits, kind, 0.5 + i, col=False))
        ref.append((bits, kind, 0.5 + i))
    cuda_lib.fp4_cast_multi(ds)
    for d, r in zip(ds, ref):
        check_cast(d, *r)


@pytest.mark.parametrize("kind", KINDS)
def test_cast_same_tensor_twice(cuda_lib, kind):
    """One input under two descriptors (other outputs, one amax slot), and one descriptor twice."""
    bits = random_bits(96, 128, 33)
    a = cast(cuda_lib, bits, kind, 3.0)
    b = cast(cuda_lib, bits, kind, 3.0, col=False)
    b["x"] = a["x"]
    if kind == bq.NVFP4:
        b["amax"] = a["amax"]
    cuda_lib.fp4_cast_multi([a, b, a])
    check_cast(a, bits, kind, 3.0)
    check_cast(b, bits, kind, 3.0)


@pytest.mark.parametrize("kind", KINDS)
def test_gemm_operand_used_twice(cuda_lib, kind):
    """A.A^T, and one weight under two inputs in a call; K from one block to many in one launch."""
    A, sa, a = operand(40, 4096, kind, 1)
    B, sb, b = operand(72, 4096, kind, 2)
    C, sc, c = operand(24, 32, kind, 3)
    out = [torch.full(s, float("nan"), dtype=torch.bfloat16, device="cuda") for s in ((40, 40), (40, 72), (72, 72), (24, 24))]
    cuda_lib.fp4_gemm_multi([dict(A=p, a_sf=sp, B=q, b_sf=sq, quant=kind, D=D) for (p, sp, q, sq), D in
                             zip(((A, sa, A, sa), (A, sa, B, sb), (B, sb, B, sb), (C, sc, C, sc)), out)])
    cuda_lib.fp8t_check_device_error()
    for (p, q), D in zip(((a, a), (a, b), (b, b), (c, c)), out):
        assert gemm_within_tolerance(bf16_bits(D), *reference(p, q, 1.0)).all()


# ------------------------------------------------------------------ streams and graphs
@pytest.mark.parametrize("kind", KINDS)
def test_products_on_two_streams_at_once(cuda_lib, kind):
    """Pair tiles on one stream and products of few rows (K split over clusters) on another, many times over."""
    sizes = [(600, 1544, 2048), (24, 2048, 4096)]
    sets = []
    for i, (M, N, K) in enumerate(sizes):
        A, sa, a = operand(M, K, kind, i)
        B, sb, b = operand(N, K, kind, 10 + i)
        sets.append((dict(A=A, a_sf=sa, B=B, b_sf=sb, quant=kind),
                     [torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(20)], reference(a, b, 1.0)))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for i in range(20):
        for s, (d, outs, _) in zip(streams, sets):
            cuda_lib.fp4_gemm_multi([dict(d, D=outs[i])], stream=s)
    torch.cuda.synchronize()
    cuda_lib.fp8t_check_device_error()
    for _, outs, ref in sets:
        assert gemm_within_tolerance(bf16_bits(outs[0]), *ref).all()
        assert all(torch.equal(o, outs[0]) for o in outs)


@pytest.mark.parametrize("kind", KINDS)
def test_layer_chain_in_two_graphs(cuda_lib, kind):
    """norm -> product -> norm -> product, each reading what the one before wrote, captured twice with buffers of
    their own and replayed on two streams at once: every replay gives the eager call's bits (the kernels start
    before the ones they read from have ended)."""
    rows, cols, N = 9, 1024, 1024
    x, _, gamma = make(rows, cols, 7)
    x, gamma = bf16_from_bits(x), bf16_from_bits(gamma).reshape(-1)
    W = [operand(N, cols, kind, 70 + i)[:2] for i in range(2)]
    one = torch.ones(1, device="cuda")

    def buffers():
        b = dict(q=torch.empty(rows, cols // 2, dtype=torch.uint8, device="cuda"),
                 sf=torch.zeros(cuda_lib.fp4_scale_bytes(rows, cols, kind), dtype=torch.uint8, device="cuda"),
                 h=torch.empty_like(x))
        return b, [torch.empty(rows, N, dtype=torch.bfloat16, device="cuda") for _ in range(2)]

    def chain(b, D, stream=None):
        scale = dict(scale=one) if kind == bq.NVFP4 else {}
        cuda_lib.fp8_rmsnorm_cast(x, gamma, 1e-5, quant=kind, q=b["q"], sf=b["sf"], stream=stream, **scale)
        cuda_lib.fp4_gemm_multi([dict(A=b["q"], a_sf=b["sf"], B=W[0][0], b_sf=W[0][1], quant=kind, D=D[0])], stream=stream)
        cuda_lib.fp8_rmsnorm_cast(D[0], gamma, 1e-5, residual=x, h=b["h"], quant=kind, q=b["q"], sf=b["sf"], stream=stream, **scale)
        cuda_lib.fp4_gemm_multi([dict(A=b["q"], a_sf=b["sf"], B=W[1][0], b_sf=W[1][1], quant=kind, D=D[1])], stream=stream)
    b, want = buffers()
    chain(b, want)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        b, D = buffers()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            chain(b, D)
        graphs.append((g, s, D, b))
    for _ in range(20):
        for g, s, D, _b in graphs:
            with torch.cuda.stream(s):
                for d in D:
                    d.fill_(float("nan"))
                g.replay()
    torch.cuda.synchronize()
    cuda_lib.fp8t_check_device_error()
    for _, _, D, _b in graphs:
        assert torch.equal(D[0], want[0]) and torch.equal(D[1], want[1])


def test_backward_captured_with_a_workspace_of_the_call(cuda_lib):
    """The workspace that a captured call allocates belongs to its graph: eager calls between replays change nothing."""
    x, r, gamma = make(700, 1024, 9)
    h, dy, gamma = bf16_from_bits(x), bf16_from_bits(r), bf16_from_bits(gamma).reshape(-1)
    rstd = torch.rand(700, device="cuda") + 0.5

    def outs():
        return torch.empty_like(h), torch.empty(1024, device="cuda")
    dh, dg = outs()
    cuda_lib.fp8_rmsnorm_backward(dy, h, gamma, rstd, dh, dgamma=dg)
    gh, gg = outs()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        cuda_lib.fp8_rmsnorm_backward(dy, h, gamma, rstd, gh, dgamma=gg)
    eh, eg = outs()
    for _ in range(3):
        gh.fill_(float("nan"))
        gg.fill_(float("nan"))
        graph.replay()
        cuda_lib.fp8_rmsnorm_backward(h, dy, gamma, rstd, eh, dgamma=eg)
        torch.cuda.synchronize()
        assert torch.equal(gh, dh) and torch.equal(gg, dg)


# ------------------------------------------------------------------ sizes
@pytest.mark.parametrize("rows,cols", [(700, 8192), (310, 8208), (160, 12288), (333, 12304), (299, 16384), (40000, 16)])
def test_backward_of_wide_and_short_rows(cuda_lib, rows, cols):
    """Two, three and four vectors per thread with dres, and the shortest rows; dh over dy and over dres."""
    h, r, gamma = make(rows, cols, rows)
    rng = np.random.default_rng(cols)
    dy, dres = bf(rng.standard_normal((rows, cols))), bf(rng.standard_normal((rows, cols)))
    H, G, DY, DR = (bq.bf16_f64(v) for v in (h, gamma, dy, dres))
    rstd = bq.rmsnorm(H, None, G, 1e-5)[1].astype(np.float32).astype(np.float64)
    want, wantg = bq.rmsnorm_grad(DY, H, G, rstd, DR)
    xh = H * rstd[:, None]
    terms = rstd[:, None] * (np.abs(DY * G) + np.abs(xh) * np.abs(DY * G * xh).mean(1, keepdims=True)) + np.abs(DR)
    first = None
    for place in ("own", "dy", "dres"):
        t = dict(dy=bf16_from_bits(dy), dres=bf16_from_bits(dres))
        t["own"] = torch.full_like(t["dy"], float("nan"))
        dg = torch.full((cols,), float("nan"), device="cuda")
        cuda_lib.fp8_rmsnorm_backward(t["dy"], bf16_from_bits(h), bf16_from_bits(gamma),
                                      torch.from_numpy(rstd.astype(np.float32)).cuda(), t[place], dres=t["dres"], dgamma=dg)
        if first is None:
            first = t[place], dg
            assert (np.abs(bq.bf16_f64(bf16_bits(t[place])) - want) <= 2.0 ** -8 * np.abs(want) + 64 * U * terms).all()
            # a column: rows / 148 additions or fewer in a thread's chain, at most 16 groups, 148 partials
            bound = (rows // 148 + 1 + 16 + 148 // 16 + 1 + 16 + 8) * U * np.abs(DY * xh).sum(0)
            assert (np.abs(dg.cpu().numpy() - wantg) <= bound).all()
        assert torch.equal(t[place].view(torch.int16), first[0].view(torch.int16)) and torch.equal(dg, first[1])


@pytest.mark.parametrize("quant", [1, MXFP4])
def test_norm_of_many_short_rows(cuda_lib, quant):
    x, r, gamma = make(40000, 32, 6)
    check(run(cuda_lib, x, r, gamma, 1e-5, quant), x, r, gamma, 1e-5, quant)


def some_rows(rows, n=24):
    """Rows to check: the first and last, those around 2^31 elements' border and random ones."""
    rng = np.random.default_rng(rows)
    at = (1 << 31) // 16384
    return np.unique(np.concatenate(([0, 1, at - 1, at, at + 1, rows - 2, rows - 1], rng.integers(0, rows, n))))


def big(rows, cols):
    """BF16 values on the device, more than 2^31 of them."""
    t = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator("cuda").manual_seed(5)
    for i in range(0, rows, 16384):
        t[i:i + 16384].normal_(generator=g)
    return t


def test_norm_of_more_than_2_31_elements(cuda_lib):
    rows, cols = (1 << 17) + 77, 16384
    x = big(rows, cols)
    gamma = bf16_from_bits(make(1, cols, 1)[2]).reshape(-1)
    rstd = torch.empty(rows, device="cuda")
    q = torch.empty(rows, cols // 2, dtype=torch.uint8, device="cuda")
    sf = torch.empty(cuda_lib.fp4_scale_bytes(rows, cols, bq.MXFP4), dtype=torch.uint8, device="cuda")
    cuda_lib.fp8_rmsnorm_cast(x, gamma, 1e-5, rstd=rstd, quant=MXFP4, q=q, sf=sf)
    at = some_rows(rows)
    i = torch.from_numpy(at).cuda()
    words = sf.view(-1, cols // 128, 128, 4)                           # row blocks, atoms, bytes of an atom by row
    rows_sf = words[i // 128, :, (i % 32) * 4 + (i % 128) // 32, :].cpu().numpy().reshape(len(at), cols // 32)
    own = torch.zeros(cuda_lib.fp4_scale_bytes(len(at), cols, bq.MXFP4), dtype=torch.uint8)
    own.copy_(torch.from_numpy(bq.atoms(rows_sf, bq.MXFP4)))
    bits = bf16_bits(x[i])
    check(dict(rstd=rstd[i], q=q[i], sf=own), bits, None, bf16_bits(gamma.reshape(1, -1))[0], 1e-5, MXFP4)
    dh = torch.empty_like(x)
    cuda_lib.fp8_rmsnorm_backward(x, x, gamma, rstd, dh)               # dy = h: no dgamma, no workspace
    H, G = bq.bf16_f64(bits), bq.bf16_f64(bf16_bits(gamma.reshape(1, -1)))[0]
    rs = rstd[i].cpu().numpy().astype(np.float64)
    want, _ = bq.rmsnorm_grad(H, H, G, rs)
    xh = H * rs[:, None]
    terms = rs[:, None] * (np.abs(H * G) + np.abs(xh) * np.abs(H * G * xh).mean(1, keepdims=True))
    assert (np.abs(bq.bf16_f64(bf16_bits(dh[i])) - want) <= 2.0 ** -8 * np.abs(want) + 64 * U * terms).all()


@pytest.mark.parametrize("kind", KINDS)
def test_cast_of_more_than_2_31_elements(cuda_lib, kind):
    rows, cols = (1 << 17) + 96, 16384
    x = big(rows, cols)
    n = {bq.MXFP4: 32, bq.NVFP4: 16}[kind]
    q = torch.empty(rows, cols // 2, dtype=torch.uint8, device="cuda")
    sf = torch.empty(cuda_lib.fp4_scale_bytes(rows, cols, kind), dtype=torch.uint8, device="cuda")
    qc = torch.empty(cols, rows // 2, dtype=torch.uint8, device="cuda")
    sfc = torch.empty(cuda_lib.fp4_scale_bytes(cols, rows, kind), dtype=torch.uint8, device="cuda")
    scale = dict(scale=torch.full((1,), 100.0, device="cuda")) if kind == bq.NVFP4 else {}

    def rows_of(sf, at, K):
        i = torch.from_numpy(at).cuda()
        words = sf.view(-(-int(sf.numel()) // (512 * (-(-K // 256) * 256 // n // 4))), -1, 128, 4)
        return words[i // 128, :, (i % 32) * 4 + (i % 128) // 32, :].cpu().numpy().reshape(len(at), -1)
    at = some_rows(rows)
    for col in (False, True):
        q.fill_(0xEE)
        cuda_lib.fp4_cast_multi([dict(x=x, quant=kind, q_row=q, sf_row=sf, **(dict(q_col=qc, sf_col=sfc) if col else {}), **scale)])
        i = torch.from_numpy(at).cuda()
        codes, s = bq.quantise(bf16_bits(x[i]), kind, 100.0)
        assert np.array_equal(bq.unpack(u8(q[i])), codes) and np.array_equal(rows_of(sf, at, cols), s)
    cuda_lib.fp8t_check_device_error()
    cs = np.array([0, 1, 8191, cols - 1])
    codes, s = bq.quantise(np.ascontiguousarray(bf16_bits(x[:, torch.from_numpy(cs).cuda()]).T), kind, 100.0)
    assert np.array_equal(bq.unpack(u8(qc[torch.from_numpy(cs).cuda()])), codes)
    got = rows_of(sfc, cs, rows)
    assert np.array_equal(got[:, :rows // n], s) and not got[:, rows // n:].any()


@pytest.mark.parametrize("kind", KINDS)
def test_gemm_output_of_more_than_2_31_elements(cuda_lib, kind):
    M, N, K = (1 << 17) + 300, 16392, 64
    A, sa, a = operand(4096, K, kind, 1)
    B, sb, b = operand(N, K, kind, 2)
    reps = -(-M // 4096)                                                # 4096 rows are whole atoms
    per = sa.numel()
    D = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    big_a = A.repeat(reps, 1)[:M].contiguous()
    big_s = sa.repeat(reps)[:cuda_lib.fp4_scale_bytes(M, K, kind)].contiguous()
    assert per % 512 == 0
    cuda_lib.fp4_gemm_multi([dict(A=big_a, a_sf=big_s, B=B, b_sf=sb, quant=kind, D=D)])
    cuda_lib.fp8t_check_device_error()
    at = some_rows(M)
    R, ab = reference(a[at % 4096], b, 1.0)
    assert gemm_within_tolerance(bf16_bits(D[torch.from_numpy(at).cuda()]), R, ab).all()
    whole = M // 4096 * 4096
    assert all(torch.equal(D[i:i + 4096], D[:4096]) for i in range(4096, whole, 4096))
    assert torch.equal(D[whole:], D[:M - whole])
