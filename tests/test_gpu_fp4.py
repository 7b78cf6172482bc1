"""4-bit quantisation and products through the C ABI against the 64-bit reference of tests/_block_quant.py.

Codes and scales are compared bit for bit: E2M1 / E4M3 / E8M0 rounding is exact and every f32 operation of
NVFP4 is a single rounded one, repeated in numpy. GEMM outputs: 2 BF16 ulp + 1e-5 * sum |a b| scales, the
tolerance of the other GEMMs (half an ulp each for the two roundings to BF16 compared, and an FP32
accumulation over K / 64 steps, each off by at most a few 2^-24 of the running sum)."""
import numpy as np
import pytest
import torch

from tests import _block_quant as bq
from tests._gpu import bf16_bits, bf16_from_bits, u8
from tests._pins import gemm_within_tolerance

pytestmark = pytest.mark.gpu
KINDS = (bq.MXFP4, bq.NVFP4)


def zeros(n):
    return torch.zeros(n, dtype=torch.uint8, device="cuda")


def f32(v):
    return torch.tensor([v], dtype=torch.float32, device="cuda")


def random_bits(rows, cols, seed, spread=4.0):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, cols)) * 2.0 ** rng.uniform(-spread, spread, (rows, 1)) * \
        2.0 ** rng.uniform(-spread, spread, (1, cols))
    return bf16_bits(torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16))


def cast(fp8, bits, kind, g, row=True, col=True, **kw):
    rows, cols = bits.shape
    d = dict(x=bf16_from_bits(bits), quant=kind)
    if row:
        d.update(q_row=torch.full((rows, cols // 2), 0xEE, dtype=torch.uint8, device="cuda"),
                 sf_row=torch.full((fp8.fp4_scale_bytes(rows, cols, kind),), 0xEE, dtype=torch.uint8, device="cuda"))
    if col:
        d.update(q_col=torch.full((cols, rows // 2), 0xEE, dtype=torch.uint8, device="cuda"),
                 sf_col=torch.full((fp8.fp4_scale_bytes(cols, rows, kind),), 0xEE, dtype=torch.uint8, device="cuda"))
    if kind == bq.NVFP4:
        d.update(scale=f32(g), amax=f32(0.0), scale_inv=f32(0.0))
    d.update(kw)
    return d


def check_cast(d, bits, kind, g):
    """Codes, scales, and zero bytes in all of the atoms' padding (rows and K)."""
    for q, sf, b in ((d.get("q_row"), d.get("sf_row"), bits), (d.get("q_col"), d.get("sf_col"), np.ascontiguousarray(bits.T))):
        if q is None:
            continue
        codes, s = bq.quantise(b, kind, g)
        assert np.array_equal(bq.unpack(u8(q)), codes)
        assert np.array_equal(u8(sf), bq.atoms(s, kind))
    if kind == bq.NVFP4:
        a = bq.bf16_f64(bits & 0x7FFF)
        want = np.float32(np.nan if np.isnan(a).any() else a.max())
        assert np.array_equal(d["amax"].cpu().numpy(), [want], equal_nan=True)
        assert d["scale_inv"].item() == np.float32(1) / np.float32(g)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,cols", [(32, 32), (128, 128), (256, 384), (96, 160), (544, 1056), (160, 64)])
def test_cast_both_ways(cuda_lib, kind, rows, cols):
    bits = random_bits(rows, cols, rows + cols)
    d = cast(cuda_lib, bits, kind, 37.5)
    cuda_lib.fp4_cast_multi([d])
    cuda_lib.fp8t_check_device_error()
    check_cast(d, bits, kind, 37.5)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows", [1, 3, 127, 129, 301])
def test_cast_row_wise_any_number_of_rows(cuda_lib, kind, rows):
    bits = random_bits(rows, 288, rows)
    d = cast(cuda_lib, bits, kind, 3.0, col=False)
    cuda_lib.fp4_cast_multi([d])
    cuda_lib.fp8t_check_device_error()
    check_cast(d, bits, kind, 3.0)


@pytest.mark.parametrize("kind", KINDS)
def test_cast_inputs_aligned_to_16_bytes_only(cuda_lib, kind):
    """Every pointer at 16 bytes past a 32-byte boundary, one and both ways."""
    bits = random_bits(96, 320, 17)
    for col in (False, True):
        d = cast(cuda_lib, bits, kind, 3.0, col=col)
        for k, e in (("x", 8), ("q_row", 16), ("sf_row", 16), ("q_col", 16), ("sf_col", 16)):
            if k in d:
                whole = torch.empty(d[k].numel() + e, dtype=d[k].dtype, device="cuda")
                assert whole.data_ptr() % 32 == 0
                whole[e:] = d[k].reshape(-1)
                d[k] = whole[e:].view(d[k].shape)
        cuda_lib.fp4_cast_multi([d])
        check_cast(d, bits, kind, 3.0)


@pytest.mark.parametrize("kind", KINDS)
def test_cast_column_wise_only(cuda_lib, kind):
    bits = random_bits(192, 224, 5)
    d = cast(cuda_lib, bits, kind, 11.0, row=False)
    cuda_lib.fp4_cast_multi([d])
    check_cast(d, bits, kind, 11.0)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("g", [1.0, 1000.0, 1e-30])
def test_cast_every_bf16_pattern(cuda_lib, kind, g):
    """Subnormals, infinities, NaN of both signs; -0; scales that vanish and saturate."""
    bits = np.arange(65536, dtype=np.uint32).astype(np.uint16).reshape(256, 256)
    for b in (bits, np.ascontiguousarray(bits.T)):
        d = cast(cuda_lib, b, kind, g)
        cuda_lib.fp4_cast_multi([d])
        check_cast(d, b, kind, g)


def test_cast_grouped_over_two_launches(cuda_lib):
    """More tensors than a launch takes, both formats and ragged sizes among them."""
    ds, ref = [], []
    for i in range(11):
        kind = KINDS[i % 2]
        bits = random_bits(32 * (1 + i), 32 * (12 - i), 100 + i)
        ds.append(cast(cuda_lib, bits, kind, 1.0 + i))
        ref.append((bits, kind, 1.0 + i))
    cuda_lib.fp4_cast_multi(ds)
    cuda_lib.fp8t_check_device_error()
    for d, (bits, kind, g) in zip(ds, ref):
        check_cast(d, bits, kind, g)


def test_nvfp4_amax_is_max_accumulated(cuda_lib):
    bits = random_bits(64, 64, 9)
    d = cast(cuda_lib, bits, bq.NVFP4, 2.0, amax=f32(1e9))
    cuda_lib.fp4_cast_multi([d])
    assert d["amax"].item() == np.float32(1e9)


# ------------------------------------------------------------------ products
def operand(rows, K, kind, seed, spread=4.0):
    codes, sf = bq.quantise(random_bits(rows, K, seed, spread), kind, 24.0)
    return (torch.from_numpy(bq.pack(codes)).cuda(), torch.from_numpy(bq.atoms(sf, kind)).cuda(),
            bq.values(codes, sf, kind))


def reference(a, b, alpha):
    with np.errstate(invalid="ignore"):
        R, ab = (a @ b.T) * alpha, (np.abs(a) @ np.abs(b).T) * abs(alpha)
    return bf16_bits(torch.from_numpy(R).to(torch.float32).to(torch.bfloat16)), ab


def check_gemm(fp8, M, N, K, kind, seed=0):
    A, sa, a = operand(M, K, kind, seed + M)
    B, sb, b = operand(N, K, kind, seed + N + 1)
    guard = torch.full((M + 2, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    D = guard[1:M + 1]
    if D.data_ptr() % 16:                            # N = 8: every row is 16 bytes, so this never moves
        raise AssertionError("misaligned test buffer")
    fp8.fp4_gemm_multi([dict(A=A, a_sf=sa, B=B, b_sf=sb, quant=kind, D=D, a_scale_inv=f32(0.5), b_scale_inv=f32(0.75))])
    fp8.fp8t_check_device_error()
    R, ab = reference(a, b, 0.375)
    ok = gemm_within_tolerance(bf16_bits(D), R, ab)
    assert ok.all(), f"{(~ok).sum()} of {ok.size} outside tolerance"
    assert torch.isnan(guard[0]).all() and torch.isnan(guard[-1]).all()     # nothing outside D is written


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("M,N,K", [(128, 128, 256), (256, 384, 512), (256, 256, 128), (300, 520, 288), (129, 392, 32),
                                   (512, 640, 1056), (513, 1160, 96), (1000, 776, 4096), (257, 1408, 2080)])
def test_gemm_full_output(cuda_lib, kind, M, N, K):
    check_gemm(cuda_lib, M, N, K, kind)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("M", [1, 2, 7, 8, 16, 17, 31, 33, 64, 65, 127, 128])
@pytest.mark.parametrize("N,K", [(8, 32), (136, 416), (1024, 4096)])
def test_gemm_few_tokens(cuda_lib, kind, M, N, K):
    check_gemm(cuda_lib, M, N, K, kind, seed=3)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("M,N,K", [(1, 11008, 4096), (16, 4096, 11008), (192, 4096, 4096), (384, 2048, 8192), (640, 4096, 1024)])
def test_gemm_between(cuda_lib, kind, M, N, K):
    check_gemm(cuda_lib, M, N, K, kind, seed=7)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("M,N,K", [(2100, 4104, 544), (2304, 4224, 96), (2049, 4544, 32), (1281, 6536, 800)])
def test_gemm_wide_tiles(cuda_lib, kind, M, N, K):
    """Sizes that take 384-column tiles: a last column tile of 264, 384, 320 (its N = 128 MMA partly outside) and
    8 columns (without that MMA), rows that leave one row or one CTA's half of a tile."""
    check_gemm(cuda_lib, M, N, K, kind, seed=11)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("shapes", [
    [(700, 2000, 288), (900, 1544, 1088), (300, 2056, 96), (1100, 1280, 32), (200, 776, 2048)],     # 256 columns, lists
    [(1536, 4104, 64), (1300, 3864, 576), (520, 1160, 1024)],                                       # 384 columns, lists
    [(1300, 1160, 160)] * 6])                                                                       # more than four
def test_gemm_grouped_large(cuda_lib, kind, shapes):
    descs, refs = [], []
    for i, (M, N, K) in enumerate(shapes):
        A, sa, a = operand(M, K, kind, i)
        B, sb, b = operand(N, K, kind, 50 + i)
        D = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
        descs.append(dict(A=A, a_sf=sa, B=B, b_sf=sb, quant=kind, D=D, b_scale_inv=f32(0.25)))
        refs.append(reference(a, b, 0.25))
    cuda_lib.fp4_gemm_multi(descs)
    cuda_lib.fp8t_check_device_error()
    for d, (R, ab) in zip(descs, refs):
        assert gemm_within_tolerance(bf16_bits(d["D"]), R, ab).all()


@pytest.mark.parametrize("kind", KINDS)
def test_gemm_scales_missing_means_one(cuda_lib, kind):
    A, sa, a = operand(40, 256, kind, 1)
    B, sb, b = operand(64, 256, kind, 2)
    D = torch.empty(40, 64, dtype=torch.bfloat16, device="cuda")
    cuda_lib.fp4_gemm_multi([dict(A=A, a_sf=sa, B=B, b_sf=sb, quant=kind, D=D)])
    R, ab = reference(a, b, 1.0)
    assert gemm_within_tolerance(bf16_bits(D), R, ab).all()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("M", [5, 300])
def test_gemm_rows_past_the_matrix_may_hold_any_scale(cuda_lib, kind, M):
    """NaN scale bytes in the rows that fill up A's and B's last atoms change nothing."""
    N, K = 136, 512
    A, sa, a = operand(M, K, kind, 1)
    B, sb, b = operand(N, K, kind, 2)
    n = {bq.MXFP4: 32, bq.NVFP4: 16}[kind]

    def spoil(sf, rows):
        R = -(-rows // 128) * 128
        full = np.full((R, K // n), 0xFF if kind == bq.MXFP4 else 0x7F, np.uint8)
        full[:rows] = bq.from_atoms(u8(sf), rows, K // n, kind)[0]
        return torch.from_numpy(bq.atoms(full, kind)).cuda()
    D = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    cuda_lib.fp4_gemm_multi([dict(A=A, a_sf=spoil(sa, M), B=B, b_sf=spoil(sb, N), quant=kind, D=D)])
    R, ab = reference(a, b, 1.0)
    assert gemm_within_tolerance(bf16_bits(D), R, ab).all()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("M", [4, 260])
def test_gemm_nan_scale_reaches_its_row_only(cuda_lib, kind, M):
    N, K = 128, 512
    A, sa, a = operand(M, K, kind, 1)
    B, sb, b = operand(N, K, kind, 2)
    n = {bq.MXFP4: 32, bq.NVFP4: 16}[kind]
    sf = bq.from_atoms(u8(sa), M, K // n, kind)[0]
    sf[2, 1] = 0xFF if kind == bq.MXFP4 else 0x7F
    D = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    cuda_lib.fp4_gemm_multi([dict(A=A, a_sf=torch.from_numpy(bq.atoms(sf, kind)).cuda(), B=B, b_sf=sb, quant=kind, D=D)])
    d = D.float().cpu().numpy()
    assert np.isnan(d[2]).all() and np.isfinite(np.delete(d, 2, 0)).all()


def test_gemm_grouped_mixed(cuda_lib):
    """Both formats, small and large problems in one call, over more problems than a launch takes."""
    descs, refs = [], []
    for i in range(30):
        kind = KINDS[(i // 3) % 2]
        M, N, K = (1, 3, 70, 200, 300)[i % 5], 8 * (1 + 7 * (i % 6)), 32 * (1 + 5 * (i % 4))
        A, sa, a = operand(M, K, kind, i)
        B, sb, b = operand(N, K, kind, 50 + i)
        D = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
        descs.append(dict(A=A, a_sf=sa, B=B, b_sf=sb, quant=kind, D=D, a_scale_inv=f32(2.0)))
        refs.append(reference(a, b, 2.0))
    cuda_lib.fp4_gemm_multi(descs)
    cuda_lib.fp8t_check_device_error()
    for d, (R, ab) in zip(descs, refs):
        assert gemm_within_tolerance(bf16_bits(d["D"]), R, ab).all()


@pytest.mark.parametrize("kind", KINDS)
def test_gemm_same_result_every_run(cuda_lib, kind):
    for M in (3, 96, 700):
        A, sa, _ = operand(M, 4096, kind, 1)
        B, sb, _ = operand(512, 4096, kind, 2)
        out = []
        for _ in range(3):
            D = torch.empty(M, 512, dtype=torch.bfloat16, device="cuda")
            cuda_lib.fp4_gemm_multi([dict(A=A, a_sf=sa, B=B, b_sf=sb, quant=kind, D=D)])
            out.append(D)
        assert torch.equal(out[0].view(torch.int16), out[1].view(torch.int16))
        assert torch.equal(out[0].view(torch.int16), out[2].view(torch.int16))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T,fin,fout", [(512, 256, 256), (352, 160, 416), (32, 64, 32)])
def test_training_step_products(cuda_lib, kind, T, fin, fout):
    """Cast X, W, dY along both axes, then fprop, dgrad and wgrad, captured in a graph, replayed with new
    data, on a side stream."""
    g = dict(x=900.0, w=40000.0, dy=700000.0) if kind == bq.NVFP4 else dict(x=1.0, w=1.0, dy=1.0)
    shapes = dict(x=(T, fin), w=(fin, fout), dy=(T, fout))
    sigma = dict(x=1.0, w=0.02, dy=1e-3)
    rng = np.random.default_rng(4)

    def draw():
        return {k: bf16_bits(torch.from_numpy((rng.standard_normal(s) * sigma[k]).astype(np.float32)).to(torch.bfloat16))
                for k, s in shapes.items()}
    bits = draw()
    d = {k: cast(cuda_lib, bits[k], kind, g[k]) for k in shapes}
    out = dict(y=torch.empty(T, fout, dtype=torch.bfloat16, device="cuda"),
               dx=torch.empty(T, fin, dtype=torch.bfloat16, device="cuda"),
               dw=torch.empty(fin, fout, dtype=torch.bfloat16, device="cuda"))

    def gemm(a, aw, b, bw, D):
        p = dict(A=d[a]["q_" + aw], a_sf=d[a]["sf_" + aw], B=d[b]["q_" + bw], b_sf=d[b]["sf_" + bw], quant=kind, D=D)
        if kind == bq.NVFP4:
            p.update(a_scale_inv=d[a]["scale_inv"], b_scale_inv=d[b]["scale_inv"])
        return p

    def step():
        cuda_lib.fp4_cast_multi([d["x"], d["w"], d["dy"]])
        cuda_lib.fp4_gemm_multi([gemm("x", "row", "w", "col", out["y"]), gemm("dy", "row", "w", "row", out["dx"]),
                                 gemm("x", "col", "dy", "col", out["dw"])])
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()                                       # warm-up outside the capture
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            step()
    for _ in range(2):
        bits = draw()
        for k in shapes:
            d[k]["x"].copy_(bf16_from_bits(bits[k]))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        v = {}
        for k in shapes:
            for way, b in (("row", bits[k]), ("col", np.ascontiguousarray(bits[k].T))):
                v[k, way] = bq.values(*bq.quantise(b, kind, g[k]), kind) / np.float64(g[k])
        for D, a, b in ((out["y"], v["x", "row"], v["w", "col"]), (out["dx"], v["dy", "row"], v["w", "row"]),
                        (out["dw"], v["x", "col"], v["dy", "col"])):
            R, ab = reference(a, b, 1.0)
            assert gemm_within_tolerance(bf16_bits(D), R, ab).all()
    cuda_lib.fp8t_check_device_error()


def test_refusals_raise_and_launch_nothing(cuda_lib):
    """A status of the library becomes an Fp8TrainError; wrong devices and layouts a ValueError."""
    A, sa, _ = operand(16, 64, bq.MXFP4, 1)
    D = torch.full((16, 16), 7.0, dtype=torch.bfloat16, device="cuda")
    ok = dict(A=A, a_sf=sa, B=A, b_sf=sa, quant=bq.MXFP4, D=D)
    for bad in ([], [dict(ok, quant=2)], [ok, dict(ok, quant=0)]):
        with pytest.raises(cuda_lib.Fp8TrainError, match="INVALID_ARG"):
            cuda_lib.fp4_gemm_multi(bad)
    with pytest.raises(ValueError, match="a_sf"):
        cuda_lib.fp4_gemm_multi([dict(ok, a_sf=sa[:-1])])
    with pytest.raises(ValueError, match="a_sf"):
        cuda_lib.fp4_gemm_multi([dict(ok, a_sf=sa.cpu())])
    with pytest.raises(ValueError, match="D"):
        cuda_lib.fp4_gemm_multi([dict(ok, D=D.t()[:, :8])])
    with pytest.raises(ValueError, match="contiguous"):
        cuda_lib.fp4_gemm_multi([dict(ok, D=D.t())])
    with pytest.raises(cuda_lib.Fp8TrainError, match="INVALID_ARG"):          # a required operand missing
        cuda_lib.fp4_gemm_multi([dict(ok, D=None)])
    with pytest.raises(cuda_lib.Fp8TrainError, match="MISALIGNED"):
        cuda_lib.fp4_gemm_multi([dict(ok, a_sf=torch.cat([sa, sa])[4:])])
    torch.cuda.synchronize()
    assert (D == 7).all()
