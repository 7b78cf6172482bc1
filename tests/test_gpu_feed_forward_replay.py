"""Steps of a feed-forward block replayed from a graph, back to back, on buffers that every call writes and the next one reads
(each kernel begins while the one before it still runs), against the same calls with the device idle between them."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def block(fp8, T, D, F, seed):
    """Buffers of a block and its calls: norm, gated product, down projection, gradient, weights' gradients, Muon, casts; and a few
    tokens through the new weights in 4 bits."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda r, c, s: torch.randn(r, c, generator=gen, device="cuda") * s  # noqa: E731
    bf, one = torch.bfloat16, lambda v=1.0: torch.full((1,), v, device="cuda")  # noqa: E731
    u8 = lambda r, c: torch.zeros(r, c, dtype=torch.uint8, device="cuda")  # noqa: E731
    b = dict(x=rnd(T, D, 1).to(bf), gamma=torch.ones(D, dtype=bf, device="cuda"), dy=rnd(T, D, 1e-3).to(bf),
             p=[rnd(D, 2 * F, 0.06), rnd(F, D, 0.04)], rstd=torch.empty(T, device="cuda"), xq=u8(T, D), wq=u8(D, 2 * F), wdq=u8(F, D),
             gu=torch.zeros(T, 2 * F, dtype=bf, device="cuda"), hq=u8(T, F), y=torch.zeros(T, D, dtype=bf, device="cuda"), dyq=u8(T, D),
             dq=u8(T, 2 * F), dx=torch.zeros(T, D, dtype=bf, device="cuda"), few=torch.zeros(3, F, dtype=bf, device="cuda"),
             out=torch.zeros(3, D, dtype=bf, device="cuda"), fewq=torch.zeros(3, F, dtype=bf, device="cuda"), skipped=torch.zeros(1, dtype=torch.int32, device="cuda"))
    b["m"] = [torch.zeros_like(p) for p in b["p"]]
    b["w"] = [p.to(bf) for p in b["p"]]
    b["g"] = [torch.zeros_like(w) for w in b["w"]]
    for k, v in (("xs", 90.), ("ws", 800.), ("wds", 900.), ("hs", 40.), ("dys", 5e6), ("ds", 4e6)):
        b[k], b[k + "i"], b[k + "a"] = one(v), one(), one(0.0)
    held = [(u8(m.shape[1], m.shape[0] // 2), torch.zeros(fp8.fp4_scale_bytes(m.shape[1], m.shape[0], fp8.Q_MXFP4),
                                                          dtype=torch.uint8, device="cuda")) for m in b["w"]]
    b["q4"], b["sf4"] = [h[0] for h in held], [h[1] for h in held]
    ws = torch.empty(fp8.muon_workspace_bytes([p.shape for p in b["p"]]), dtype=torch.uint8, device="cuda")

    def product(A, af, ai, B, bf_, bi, D_, a_mn=False, b_mn=False):
        fp8.fp8_gemm_multi([dict(A=A, a_fmt=af, B=B, b_fmt=bf_, a_scale_inv=ai, b_scale_inv=bi, D=D_, a_mn=a_mn, b_mn=b_mn)])
    w, wd = b["w"]
    calls = [
        lambda: fp8.fp8_cast_transpose_amax(w, 0, b["ws"], b["wq"], None, b["wsa"], b["wsi"]),
        lambda: fp8.fp8_cast_transpose_amax(wd, 0, b["wds"], b["wdq"], None, b["wdsa"], b["wdsi"]),
        lambda: fp8.fp8_rmsnorm_cast(b["x"], b["gamma"], 1e-5, rstd=b["rstd"], quant=fp8.Q_FP8, q=b["xq"], scale=b["xs"],
                                     amax=b["xsa"], scale_inv=b["xsi"]),
        lambda: fp8.fp8_gated_gemm(b["xq"], 0, b["wq"], 0, b["xsi"], b["wsi"], b_mn=True, gu=b["gu"], q=b["hq"], scale=b["hs"],
                                   amax=b["hsa"], scale_inv=b["hsi"]),
        lambda: fp8.fp8_gated_gemm(b["xq"][:3], 0, b["wq"], 0, b["xsi"], b["wsi"], b_mn=True, h=b["fewq"]),
        lambda: product(b["hq"], 0, b["hsi"], b["wdq"], 0, b["wdsi"], b["y"], b_mn=True),
        lambda: fp8.fp8_cast_transpose_amax(b["dy"], 1, b["dys"], b["dyq"], None, b["dysa"], b["dysi"]),
        lambda: fp8.fp8_gated_gemm_backward(b["dyq"], 1, b["wdq"], 0, b["dysi"], b["wdsi"], b["gu"], q=b["dq"], scale=b["ds"],
                                            amax=b["dsa"], scale_inv=b["dsi"]),
        lambda: product(b["dq"], 1, b["dsi"], b["wq"], 0, b["wsi"], b["dx"]),
        lambda: product(b["xq"], 0, b["xsi"], b["dq"], 1, b["dsi"], b["g"][0], a_mn=True, b_mn=True),
        lambda: product(b["hq"], 0, b["hsi"], b["dyq"], 1, b["dysi"], b["g"][1], a_mn=True, b_mn=True),
        lambda: fp8.fused_muon_multi_tensor(b["p"], b["m"], b["g"], b["w"], lr=0.02, skipped=b["skipped"], workspace=ws),
        lambda: fp8.fp4_cast_multi([dict(x=m, quant=fp8.Q_MXFP4, q_col=q, sf_col=s) for m, q, s in zip(b["w"], b["q4"], b["sf4"])]),
        lambda: fp8.fp4_matvec(b["x"][:3], b["q4"][0], b["sf4"][0], fp8.Q_MXFP4, b["few"], act=fp8.ACT_SILU),
        lambda: fp8.fp4_matvec(b["few"], b["q4"][1], b["sf4"][1], fp8.Q_MXFP4, b["out"]),
    ]
    return b, calls


def bits(b):
    out = {}
    for k, v in b.items():
        for i, t in enumerate(v if isinstance(v, list) else [v]):
            out[k, i] = t.view(torch.uint8).clone()
    return out


# matrices of both Newton-Schulz forms: 128 x 512 and 256 x 128; 256 x 1408 and 704 x 256
@pytest.mark.parametrize("T,D,F", [(304, 256, 704), (48, 128, 256), (16, 128, 64)])
def test_replayed_block(cuda_lib, T, D, F):
    alone, calls = block(cuda_lib, T, D, F, 1)
    want = []
    for _ in range(4):
        for call in calls:
            torch.cuda.synchronize()
            call()
        torch.cuda.synchronize()
        want.append(bits(alone))
    b, calls = block(cuda_lib, T, D, F, 1)
    start = {k: [t.clone() for t in v] if isinstance(v, list) else v.clone() for k, v in b.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for call in calls:
            call()
    for k, v in start.items():
        for t, f in zip(b[k] if isinstance(v, list) else [b[k]], v if isinstance(v, list) else [v]):
            t.copy_(f)
    for _ in range(4):                                         # back to back
        graph.replay()
    torch.cuda.synchronize()
    cuda_lib.fp8t_check_device_error()
    got = bits(b)
    assert all(torch.equal(got[k], want[-1][k]) for k in got), [k for k in got if not torch.equal(got[k], want[-1][k])]
    assert any(not torch.equal(want[0][k], want[1][k]) for k in got)                       # every step was another


def test_gradient_on_another_stream_and_captured(cuda_lib):
    fp8 = cuda_lib
    M, K, N = 700, 256, 1040
    a = torch.randint(0, 0x70, (M, K), dtype=torch.uint8, device="cuda")
    w = torch.randint(0x20, 0x40, (N, K), dtype=torch.uint8, device="cuda")
    gu, inv = torch.randn(M, 2 * N, device="cuda").to(torch.bfloat16), torch.full((1,), 0.01, device="cuda")
    want = torch.empty_like(gu)
    fp8.fp8_gated_gemm_backward(a, 1, w, 0, inv, inv, gu, dgu=want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = torch.zeros_like(gu)
    fp8.fp8_gated_gemm_backward(a, 1, w, 0, inv, inv, gu, dgu=got, stream=side)
    side.synchronize()
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))
    graph, kept = torch.cuda.CUDAGraph(), gu.clone()
    with torch.cuda.graph(graph):
        fp8.fp8_gated_gemm_backward(a, 1, w, 0, inv, inv, gu, dgu=gu)                      # in place
    for _ in range(3):
        gu.copy_(kept)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(gu.view(torch.int16), want.view(torch.int16))
