"""B200-native FP8 delayed-scaling Linear training step and fused AdamW.

Thin Python binding of the C ABI in ``include/fp8train.h`` (``libfp8train.so``, built in-tree for
sm_100a). Each function takes torch CUDA tensors, passes their device pointers and the current
CUDA stream to the C entry point of the same name, and raises ``Fp8TrainError`` on a non-OK
status. Every step of the path runs in the library's kernels; there is no CPU or PyTorch
fallback, and a missing library is an error.

The norm, 4-bit and gated calls (``fp8_rmsnorm_cast``, ``fp8_rmsnorm_backward``, ``fp4_cast_multi``,
``fp4_gemm_multi``, ``fp4_matvec``, ``fp8_gated_gemm``, ``fp8_gated_gemm_backward``) are made per layer on as little as one token; their binding is compiled
(``csrc/binding.cpp``, ``_binding.so``) and is loaded when one of them is first called.
"""
import ctypes as C
import functools
import importlib.util
import inspect
import os

import torch

from . import _abi

__all__ = ["fp8_cast_transpose_amax", "fp8_cast_transpose_amax_multi",
           "fp8_cast_transpose_amax_update_multi", "fp8_cast_transpose_amax_current_multi",
           "CURRENT_WORKSPACE_BYTES", "fp8_gemm", "fp8_gemm_multi", "fp8_scale_update", "fused_adamw_multi_tensor",
           "fused_adamw_workspace_bytes", "fused_adamw_multi_tensor_noalloc",
           "fp8_gemm_multi_sumsq", "fp8_gemm_sumsq_workspace_bytes",
           "fused_adamw_multi_tensor_presummed", "fp8_mx_cast_multi", "fp8_mx_gemm_multi",
           "fp8_mx_gemm_multi_sumsq", "fp8_mx_gemm_sumsq_workspace_bytes",
           "mx_scale_bytes", "fp4_scale_bytes", "fp4_cast_multi", "fp4_gemm_multi", "fp8_rmsnorm_cast",
           "fp8_rmsnorm_backward", "fp8_rmsnorm_backward_workspace_bytes",
           "fp8_gated_gemm", "fp8_gated_gemm_backward", "fp4_matvec", "muon_orthogonalize", "fused_muon_multi_tensor",
           "muon_workspace_bytes", "ACT_NONE", "ACT_SILU", "ACT_GELU",
           "Q_NONE", "Q_FP8", "Q_MXFP8", "Q_MXFP4", "Q_NVFP4", "FP4_MAX",
           "fp8t_check_device_error", "fp8t_debug_expire_waits", "fp8t_set_wait_timeout_ns",
           "Fp8TrainError", "E4M3", "E5M2", "K_MAJOR", "MN_MAJOR", "AMAX_MAX", "AMAX_MOST_RECENT", "FP8_MAX", "load",
           "LIB_PATH"]

E4M3, E5M2 = 0, 1
AMAX_MAX, AMAX_MOST_RECENT = 0, 1
K_MAJOR, MN_MAJOR = 0, 1
Q_NONE, Q_FP8, Q_MXFP8, Q_MXFP4, Q_NVFP4 = 0, 1, 2, 3, 4
ACT_NONE, ACT_SILU, ACT_GELU = 0, 1, 2
FP8_MAX = {E4M3: 448.0, E5M2: 57344.0}
FP4_MAX = 448.0 * 6.0        # NVFP4's largest scale times its largest value (fp8_max of its scale update)
LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libfp8train.so")
BINDING_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_binding.so")


class Fp8TrainError(RuntimeError):
    def __init__(self, status, where, message):
        self.status = status
        super().__init__(f"{where}: {_abi.status_name(status)} ({message})")


_lib = None


def load():
    """Load libfp8train.so (raises if it has not been built: there is no fallback)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m optimizer_fp8_cast_b200.build`")
        _lib = _abi.declare(C.CDLL(LIB_PATH))
    return _lib


def _check(status, where):
    if status != 0:
        raise Fp8TrainError(status, where, load().fp8t_last_error_message().decode())


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return C.c_void_p(s.cuda_stream)


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensors must be CUDA tensors")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return C.c_void_p(t.data_ptr())


def fp8_cast_transpose_amax(x, fmt, scale, q=None, qT=None, amax=None, scale_inv=None,
                            counters=None, stream=None):
    """Quantise BF16 ``x`` [rows, cols] with the device scalar ``scale`` (float32 [1]).

    Writes ``q`` [rows, cols] and ``qT`` [cols, rows] (uint8, optional) and ``scale_inv``
    (float32 [1], optional); max-accumulates max|x| into ``amax`` (float32 [1]: start it at 0,
    ``fp8_scale_update`` resets it after use) and adds to ``counters`` (int64 [3], optional:
    saturated, zero, non-finite)."""
    assert x.dtype == torch.bfloat16 and x.dim() == 2
    rows, cols = x.shape
    _check(load().fp8_cast_transpose_amax(_ptr(x), rows, cols, int(fmt), _ptr(scale), _ptr(q),
                                          _ptr(qT), _ptr(amax), _ptr(scale_inv), _ptr(counters),
                                          _stream(stream)), "fp8_cast_transpose_amax")


def _cast_array(casts):
    arr = (_abi.CastTensor * len(casts))()
    for i, c in enumerate(casts):
        x = c["x"]                  # None: a scale-update-only entry (update call only)
        assert x is None or (x.dtype == torch.bfloat16 and x.dim() == 2)
        rows, cols = (0, 0) if x is None else x.shape
        arr[i] = _abi.CastTensor(_ptr(x), rows, cols, int(c["fmt"]), _ptr(c["scale"]),
                                 _ptr(c.get("q")), _ptr(c.get("qT")), _ptr(c.get("amax")),
                                 _ptr(c.get("scale_inv")), _ptr(c.get("counters")))
    return arr


def fp8_cast_transpose_amax_multi(casts, stream=None):
    """Several casts in one launch. ``casts`` is a list of dicts with the keyword arguments of
    fp8_cast_transpose_amax (x, fmt, scale and optionally q, qT, amax, scale_inv, counters)."""
    _check(load().fp8_cast_transpose_amax_multi(_cast_array(casts), len(casts), _stream(stream)),
           "fp8_cast_transpose_amax_multi")


CURRENT_WORKSPACE_BYTES = 64


def fp8_cast_transpose_amax_current_multi(casts, margin, workspace, stream=None):
    """Current scaling: each tensor's scale (written into ``casts[i]["scale"]``) comes from its
    own amax, then the casts of fp8_cast_transpose_amax_multi run with it. ``workspace``: a
    zero-filled uint8 CUDA tensor of CURRENT_WORKSPACE_BYTES, left zero."""
    assert workspace.numel() >= CURRENT_WORKSPACE_BYTES
    _check(load().fp8_cast_transpose_amax_current_multi(_cast_array(casts), len(casts), int(margin),
                                                        _ptr(workspace), _stream(stream)),
           "fp8_cast_transpose_amax_current_multi")


def fp8_cast_transpose_amax_update_multi(casts, updates, algo, margin, ticket, stream=None):
    """The casts of fp8_cast_transpose_amax_multi and, in the same launch, the scale update of
    those tensors: ``updates[i]`` holds ``history`` (this tensor's [H] float32 row, entry 0
    newest) and ``scale_inv_next`` (1 float32, distinct from the cast's ``scale_inv``); the next
    scale is written into ``casts[i]["scale"]``. ``ticket``: one zeroed int32 on the device."""
    assert len(updates) == len(casts) and ticket.dtype == torch.int32
    H = updates[0]["history"].numel()
    arr = (_abi.CastUpdate * len(updates))()
    for i, u in enumerate(updates):
        h = u["history"]
        assert h.dtype == torch.float32 and h.numel() == H and h.is_contiguous()
        arr[i] = _abi.CastUpdate(_ptr(h), _ptr(u["scale_inv_next"]))
    _check(load().fp8_cast_transpose_amax_update_multi(_cast_array(casts), arr, len(casts), H,
                                                       int(algo), int(margin), _ptr(ticket),
                                                       _stream(stream)),
           "fp8_cast_transpose_amax_update_multi")


def fp8_gemm(A, a_fmt, B, b_fmt, a_scale_inv, b_scale_inv, D, stream=None):
    """D [M, N] bf16 = (A [M, K] . B [N, K]^T) * a_scale_inv * b_scale_inv; A, B uint8 FP8 codes."""
    M, K = A.shape
    N, K2 = B.shape
    assert K == K2 and D.shape == (M, N) and D.dtype == torch.bfloat16
    _check(load().fp8_gemm(_ptr(A), int(a_fmt), _ptr(B), int(b_fmt), M, N, K, _ptr(a_scale_inv),
                           _ptr(b_scale_inv), _ptr(D), _stream(stream)), "fp8_gemm")


def _gemm_shape(g):
    """(M, N, K) of a descriptor dict; ``a_mn`` / ``b_mn`` mark operands stored MN-major
    (A as [K, M], B as [K, N])."""
    a_mn, b_mn = bool(g.get("a_mn")), bool(g.get("b_mn"))
    K, M = g["A"].shape if a_mn else g["A"].shape[::-1]
    K2, N = g["B"].shape if b_mn else g["B"].shape[::-1]
    assert K == K2, "inner dimensions differ"
    return M, N, K


def _gemm_array(gemms):
    arr = (_abi.GemmDesc * len(gemms))()
    for i, g in enumerate(gemms):
        M, N, K = _gemm_shape(g)
        D = g["D"]
        assert D.shape == (M, N) and D.dtype == torch.bfloat16
        arr[i] = _abi.GemmDesc(_ptr(g["A"]), int(g["a_fmt"]), _ptr(g["B"]), int(g["b_fmt"]), M, N, K,
                               _ptr(g["a_scale_inv"]), _ptr(g["b_scale_inv"]), _ptr(D),
                               MN_MAJOR if g.get("a_mn") else K_MAJOR,
                               MN_MAJOR if g.get("b_mn") else K_MAJOR)
    return arr


def fp8_gemm_sumsq_workspace_bytes(gemms):
    """Scratch bytes of fp8_gemm_multi_sumsq for these problems (dicts with a ``sumsq`` flag)."""
    flags = (C.c_int32 * len(gemms))(*[1 if g.get("sumsq") else 0 for g in gemms])
    arr = (_abi.GemmDesc * len(gemms))()                 # only the shapes are read
    for i, g in enumerate(gemms):
        arr[i].M, arr[i].N, arr[i].K = _gemm_shape(g)
    return int(load().fp8_gemm_sumsq_workspace_bytes(arr, len(gemms), flags))


def fp8_gemm_multi_sumsq(gemms, sumsq_out, workspace, stream=None):
    """fp8_gemm_multi that also writes into ``sumsq_out`` (float64 [1]) the FP64 sum of f32(D)^2
    over the problems whose dict has ``sumsq=True``. ``workspace``: uint8 CUDA tensor of
    fp8_gemm_sumsq_workspace_bytes, zero-filled once before its first use."""
    flags = (C.c_int32 * len(gemms))(*[1 if g.get("sumsq") else 0 for g in gemms])
    assert sumsq_out.dtype == torch.float64
    _check(load().fp8_gemm_multi_sumsq(_gemm_array(gemms), len(gemms), flags, _ptr(sumsq_out),
                                       _ptr(workspace), workspace.numel(), _stream(stream)),
           "fp8_gemm_multi_sumsq")


def fp8_gemm_multi(gemms, stream=None):
    """Several GEMMs in one persistent launch. ``gemms`` is a list of dicts with the arguments of
    fp8_gemm: A, a_fmt, B, b_fmt, a_scale_inv, b_scale_inv, D."""
    _check(load().fp8_gemm_multi(_gemm_array(gemms), len(gemms), _stream(stream)), "fp8_gemm_multi")


def mx_scale_bytes(mn, k):
    """Bytes of the scale atoms of an MX operand with mn rows (M or N) and contraction k."""
    return (mn // 128) * (k // 128) * 512


def fp8_mx_cast_multi(casts, stream=None):
    """MXFP8 quantisation. ``casts``: dicts with x (BF16 [rows, cols]), fmt and q_row / sf_row
    (row-wise copy: blocks of 32 along rows) and/or q_col / sf_col (column-wise copy: blocks of
    32 down columns); codes are uint8 [rows, cols], scales uint8 tensors of mx_scale_bytes."""
    arr = (_abi.MxCastTensor * len(casts))()
    for i, c in enumerate(casts):
        x = c["x"]
        assert x.dtype == torch.bfloat16 and x.dim() == 2
        rows, cols = x.shape
        arr[i] = _abi.MxCastTensor(_ptr(x), rows, cols, int(c["fmt"]), _ptr(c.get("q_row")),
                                   _ptr(c.get("sf_row")), _ptr(c.get("q_col")), _ptr(c.get("sf_col")))
    _check(load().fp8_mx_cast_multi(arr, len(casts), _stream(stream)), "fp8_mx_cast_multi")


def _mx_gemm_array(gemms):
    arr = (_abi.MxGemmDesc * len(gemms))()
    for i, g in enumerate(gemms):
        M, N, K = _gemm_shape(g)
        D = g["D"]
        assert D.shape == (M, N) and D.dtype == torch.bfloat16
        arr[i] = _abi.MxGemmDesc(_ptr(g["A"]), _ptr(g["a_sf"]), int(g["a_fmt"]),
                                 MN_MAJOR if g.get("a_mn") else K_MAJOR, _ptr(g["B"]), _ptr(g["b_sf"]),
                                 int(g["b_fmt"]), MN_MAJOR if g.get("b_mn") else K_MAJOR, M, N, K,
                                 _ptr(D))
    return arr


def fp8_mx_gemm_multi(gemms, stream=None):
    """Block-scaled FP8 GEMMs in one launch: dicts with A, a_sf, a_fmt, (a_mn), B, b_sf, b_fmt,
    (b_mn), D; D = bf16(A . B^T) with the operands' block scales (no per-tensor scale)."""
    _check(load().fp8_mx_gemm_multi(_mx_gemm_array(gemms), len(gemms), _stream(stream)),
           "fp8_mx_gemm_multi")


def fp8_mx_gemm_sumsq_workspace_bytes(gemms):
    """Scratch bytes of fp8_mx_gemm_multi_sumsq for these problems (dicts with a ``sumsq`` flag;
    only their shapes are read)."""
    flags = (C.c_int32 * len(gemms))(*[1 if g.get("sumsq") else 0 for g in gemms])
    arr = (_abi.MxGemmDesc * len(gemms))()
    for i, g in enumerate(gemms):
        arr[i].M, arr[i].N, arr[i].K = _gemm_shape(g)
    return int(load().fp8_mx_gemm_sumsq_workspace_bytes(arr, len(gemms), flags))


def fp8_mx_gemm_multi_sumsq(gemms, sumsq_out, workspace, stream=None):
    """fp8_mx_gemm_multi that also writes into ``sumsq_out`` (float64 [1]) the FP64 sum of
    f32(D)^2 over the problems whose dict has ``sumsq=True``. ``workspace``: uint8 CUDA tensor of
    fp8_mx_gemm_sumsq_workspace_bytes, zero-filled once before its first use."""
    flags = (C.c_int32 * len(gemms))(*[1 if g.get("sumsq") else 0 for g in gemms])
    assert sumsq_out.dtype == torch.float64
    _check(load().fp8_mx_gemm_multi_sumsq(_mx_gemm_array(gemms), len(gemms), flags, _ptr(sumsq_out),
                                          _ptr(workspace), workspace.numel(), _stream(stream)),
           "fp8_mx_gemm_multi_sumsq")


def fp4_scale_bytes(mn, k, quant):
    """Bytes of the scales of a 4-bit operand with mn rows (M or N) and contraction k; quant Q_MXFP4 or
    Q_NVFP4. Any mn > 0; K is padded to a multiple of 256."""
    return int(load().fp4_scale_bytes(int(mn), int(k), int(quant)))


def fp8_rmsnorm_backward_workspace_bytes(rows, cols):
    """Scratch bytes of fp8_rmsnorm_backward (0 on invalid input)."""
    return int(load().fp8_rmsnorm_backward_workspace_bytes(int(rows), int(cols)))


def _load_binding():
    """The calls of csrc/binding.cpp (norm, 4-bit and gated entry points), with the library's addresses."""
    how = ("run `python -c \"import __graft_entry__ as g; g.build()\"` or "
           "`python -m optimizer_fp8_cast_b200.build`")
    if not os.path.exists(BINDING_PATH):
        raise RuntimeError(f"{BINDING_PATH} is not built: {how}")
    spec = importlib.util.spec_from_file_location(__name__ + "._binding", BINDING_PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    from .build import binding_key
    if getattr(m, "built_for", None) != binding_key():
        raise RuntimeError(f"{BINDING_PATH} was built for {getattr(m, 'built_for', 'another version')!r}, this is "
                           f"{binding_key()!r}: {how}")
    lib = load()
    m.bind(*(C.cast(getattr(lib, f), C.c_void_p).value for f in
             ("fp8_rmsnorm_cast", "fp8_rmsnorm_backward", "fp8_rmsnorm_backward_workspace_bytes", "fp4_cast_multi",
              "fp4_gemm_multi", "fp8_gated_gemm", "fp8_gated_gemm_backward", "fp4_matvec")), _check)
    return m


_functions = {}


def _compiled(declared):
    """A call of the compiled binding as the package holds it until the first of them is made: that one loads the
    binding and puts its functions in the package, so naming or importing them needs no library."""
    name = declared.__name__

    @functools.wraps(declared)
    def call(*args, **kwargs):
        if not _functions:
            m = _load_binding()
            found = {f: getattr(m, f) for f in ("fp8_rmsnorm_cast", "fp8_rmsnorm_backward", "fp4_cast_multi",
                                                "fp4_gemm_multi", "fp8_gated_gemm", "fp8_gated_gemm_backward", "fp4_matvec")}
            _functions.update(found)
            globals().update(found)
        return _functions[name](*args, **kwargs)
    call.__text_signature__ = str(inspect.signature(declared))
    return call


@_compiled
def fp8_rmsnorm_cast(x, gamma, eps, *, residual=None, h=None, rstd=None, y=None, quant=Q_NONE, fmt=E4M3, q=None, sf=None,
                     scale=None, amax=None, scale_inv=None, stream=None):
    """h = bf16(x + residual); y = h / sqrt(mean(h^2) + eps) * gamma for each row of x (BF16 [rows, cols]).

    Writes h (BF16, with a residual; may be x or residual), rstd (float32 [rows], for the backward pass), y
    (BF16) and, as quant says, y's codes q (uint8): Q_FP8 with scale, amax (max-accumulated) and scale_inv
    (float32 [1] each), Q_MXFP8 / Q_MXFP4 / Q_NVFP4 with sf (uint8 scale atoms along the rows), Q_NVFP4 also
    with scale and optionally amax and scale_inv."""


@_compiled
def fp8_rmsnorm_backward(dy, h, gamma, rstd, dh, *, dres=None, dgamma=None, dgamma_bf16=None, workspace=None, stream=None):
    """Gradients of fp8_rmsnorm_cast: dh (BF16 [rows, cols]; may be dy or dres) from dy and the forward pass's h
    and rstd, with dres added where given; dgamma (float32 [cols]) and / or dgamma_bf16.

    workspace is a uint8 CUDA tensor of at least fp8_rmsnorm_backward_workspace_bytes bytes (allocated per
    call where it is missing)."""


@_compiled
def fp4_cast_multi(casts, stream=None):
    """4-bit quantisation. casts: a list of dicts with x (BF16 [rows, cols]), quant (Q_MXFP4 or Q_NVFP4), q_row
    (uint8 [rows, cols / 2]) / sf_row and / or q_col (uint8 [cols, rows / 2]: transposed) / sf_col, scales uint8
    tensors of fp4_scale_bytes; for NVFP4 also scale (float32 [1]) and optionally amax (max-accumulated) and
    scale_inv."""


@_compiled
def fp4_gemm_multi(gemms, stream=None):
    """4-bit block-scaled GEMMs: a list of dicts with A (uint8 [M, K / 2]), a_sf, B (uint8 [N, K / 2]), b_sf, quant,
    D (BF16 [M, N]) and optionally a_scale_inv, b_scale_inv (float32 [1]); D = bf16(A . B^T) with the operands'
    block scales, times the scale inverses."""


@_compiled
def fp8_gated_gemm(A, a_fmt, B, b_fmt, a_scale_inv, b_scale_inv, *, act=ACT_SILU, b_mn=False, gu=None, h=None, q=None,
                   q_fmt=E4M3, scale=None, amax=None, scale_inv=None, stream=None):
    """[G | U] = (A . B^T) * a_scale_inv * b_scale_inv; h = act(G) * U: both projections of a gated feed-forward block, its
    activation and product in one kernel.

    A: FP8 codes (uint8 [M, K], any M); B: codes of the gate's and the up projection's weights side by side, [2N, K], or [K, 2N]
    with b_mn (weights in x out). act: ACT_SILU or ACT_GELU (tanh form). Writes gu (BF16 [M, 2N], for the backward pass), h
    (BF16 [M, N]) and / or q (uint8 [M, N]: codes of h * scale in q_fmt, with scale and optionally scale_inv), and
    max-accumulates max|h| into amax (float32 [1] each)."""


@_compiled
def fp8_gated_gemm_backward(A, a_fmt, B, b_fmt, a_scale_inv, b_scale_inv, gu, *, act=ACT_SILU, b_mn=False, dgu=None,
                            q=None, q_fmt=E5M2, scale=None, amax=None, scale_inv=None, stream=None):
    """Gradient of fp8_gated_gemm inside the product that brings it: dH = (A . B^T) * a_scale_inv * b_scale_inv with A the
    output's gradient (codes [M, K]) and B the down projection (codes [N, K], or [K, N] with b_mn), then dG = dH * U * act'(G)
    and dU = dH * act(G) of gu (BF16 [M, 2N], the forward pass's).

    Writes [dG | dU] as dgu (BF16 [M, 2N]; may be gu) and / or q (uint8 [M, 2N] in q_fmt under one scale, with scale and
    optionally scale_inv), and max-accumulates its magnitude into amax (float32 [1] each)."""


@_compiled
def fp4_matvec(x, q, sf, quant, y, *, w_scale_inv=None, act=ACT_NONE, stream=None):
    """y = (x . W^T) * w_scale_inv for one to eight rows x (BF16 [rows, K]) and 4-bit weights W as fp4_cast_multi writes them
    row-wise: q (uint8 [N, K / 2]), sf, quant (Q_MXFP4 or Q_NVFP4).

    With act (ACT_SILU or ACT_GELU) W holds gate and up features, q is [2N, K / 2] and y = act(g) * u. y: BF16 [rows, N];
    w_scale_inv: float32 [1], the inverse of NVFP4's tensor scale."""


def fp8_scale_update(amax, history, fp8_max, algo, margin, scale, scale_inv, stream=None):
    """Roll ``history`` [n, H] (entry 0 newest) with ``amax`` [n] (reset to 0 afterwards) and
    write the next scales."""
    n, H = history.shape
    _check(load().fp8_scale_update(n, _ptr(amax), _ptr(history), H, _ptr(fp8_max), int(algo),
                                   int(margin), _ptr(scale), _ptr(scale_inv), _stream(stream)),
           "fp8_scale_update")


def _tensor_table(master, m, v, grads, weights):
    n = len(master)
    arr = (_abi.AdamWTensor * n)()
    for i in range(n):
        for t in (master[i], m[i], v[i]):
            assert t.dtype == torch.float32
        assert grads[i].dtype == torch.bfloat16 and weights[i].dtype == torch.bfloat16
        numel = master[i].numel()
        assert m[i].numel() == v[i].numel() == grads[i].numel() == weights[i].numel() == numel
        arr[i] = _abi.AdamWTensor(_ptr(master[i]), _ptr(m[i]), _ptr(v[i]), _ptr(grads[i]),
                                  _ptr(weights[i]), numel)
    return arr, n


def fused_adamw_workspace_bytes(numels):
    arr = (_abi.AdamWTensor * len(numels))()
    for i, n in enumerate(numels):
        arr[i].numel = int(n)
    return int(load().fused_adamw_workspace_bytes(arr, len(numels)))


def fused_adamw_multi_tensor(master, m, v, grads, weights, *, lr, beta1, beta2, eps,
                             weight_decay, step, loss_scale, max_grad_norm, grad_norm=None,
                             skipped=None, workspace=None, step_counter=None, stream=None):
    """One fused AdamW step over lists of tensors (see include/fp8train.h for the arithmetic).

    ``workspace`` is a uint8 CUDA tensor of at least ``fused_adamw_workspace_bytes`` bytes.
    ``step_counter`` (int64 [1] on the device, completed steps) replaces ``step``: the call
    performs step counter+1 and stores it back unless the update is skipped, which lets a
    captured CUDA graph replay successive steps."""
    arr, n = _tensor_table(master, m, v, grads, weights)
    need = int(load().fused_adamw_workspace_bytes(arr, n))
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=master[0].device)
    _check(load().fused_adamw_multi_tensor(arr, n, float(lr), float(beta1), float(beta2),
                                           float(eps), float(weight_decay), int(step),
                                           _ptr(step_counter), float(loss_scale),
                                           float(max_grad_norm),
                                           _ptr(grad_norm), _ptr(skipped), _ptr(workspace),
                                           workspace.numel(), _stream(stream)),
           "fused_adamw_multi_tensor")


def fused_adamw_multi_tensor_presummed(master, m, v, grads, weights, *, lr, beta1, beta2, eps,
                                       weight_decay, step, loss_scale, max_grad_norm, grad_sumsq,
                                       grad_norm=None, skipped=None, step_counter=None,
                                       ticket=None, casts=None, stream=None):
    """The AdamW step without its norm pass: ``grad_sumsq`` (float64 [1] on the device) holds
    the FP64 sum of f32(g)^2 over all gradients. ``ticket`` (zeroed int32 [1]) is required with
    ``step_counter``. ``casts``: None, or one entry per tensor, None or a dict (rows, cols, fmt,
    scale, and optionally q, amax, scale_inv) to cast that tensor's new BF16 weight (row-major
    codes)."""
    arr, n = _tensor_table(master, m, v, grads, weights)
    assert grad_sumsq.dtype == torch.float64
    carr = None
    if casts is not None:
        assert len(casts) == n
        carr = (_abi.AdamWCast * n)()
        for i, c in enumerate(casts):
            if c is not None:
                assert c.get("qT") is None, "weight casts inside AdamW write row-major codes only"
                carr[i] = _abi.AdamWCast(int(c["rows"]), int(c["cols"]), int(c["fmt"]),
                                         _ptr(c["scale"]), _ptr(c.get("q")),
                                         _ptr(c.get("amax")), _ptr(c.get("scale_inv")))
    _check(load().fused_adamw_multi_tensor_presummed(arr, carr, n, float(lr), float(beta1), float(beta2),
                                                     float(eps), float(weight_decay), int(step),
                                                     _ptr(step_counter), float(loss_scale),
                                                     float(max_grad_norm), _ptr(grad_sumsq),
                                                     _ptr(grad_norm), _ptr(skipped), _ptr(ticket),
                                                     _stream(stream)),
           "fused_adamw_multi_tensor_presummed")


def fused_adamw_multi_tensor_noalloc(master, m, v, grads, weights, *, lr, beta1, beta2, eps,
                                     weight_decay, step, loss_scale, max_grad_norm,
                                     grad_norm=None, skipped=None, step_counter=None, stream=None):
    """The same AdamW step, with no scratch buffer from the caller: for code that cannot
    allocate device memory (for instance a plugin that is handed the parameter buffers but not
    the framework's allocator). The library uses a 64 KiB array of its own instead; calls share
    it, so calls that overlap on the GPU race. Allocates nothing."""
    arr, n = _tensor_table(master, m, v, grads, weights)
    _check(load().fused_adamw_multi_tensor_noalloc(arr, n, float(lr), float(beta1), float(beta2),
                                                   float(eps), float(weight_decay), int(step),
                                                   _ptr(step_counter), float(loss_scale),
                                                   float(max_grad_norm),
                                                   _ptr(grad_norm), _ptr(skipped), _stream(stream)),
           "fused_adamw_multi_tensor_noalloc")


def _rows_cols(t, what):
    if t.dim() != 2 or t.size(0) < 1 or t.size(1) < 1:
        raise ValueError(f"{what}: must be a matrix of at least one element")
    return int(t.size(0)), int(t.size(1))


def muon_workspace_bytes(shapes):
    """Scratch bytes of muon_orthogonalize and fused_muon_multi_tensor for matrices of these (rows, cols)."""
    n = len(shapes)
    rows, cols = (C.c_int64 * n)(*[int(s[0]) for s in shapes]), (C.c_int64 * n)(*[int(s[1]) for s in shapes])
    return int(load().muon_workspace_bytes(rows, cols, n))


def _muon_call(shapes, tensors, workspace, stream, call, name):
    """Checks devices and the workspace (allocated on the call's stream where it is missing), and calls."""
    device = torch.device("cuda", torch.cuda.current_device())
    for t in tensors:
        if t.device != device:
            raise ValueError(f"{name}: tensors must be on the current device")
    if workspace is None:
        with torch.cuda.stream(torch.cuda.current_stream() if stream is None else stream):
            workspace = torch.empty(muon_workspace_bytes(shapes), dtype=torch.uint8, device=device)
    if workspace.dtype != torch.uint8 or workspace.device != device:
        raise ValueError(f"{name}: workspace must be a uint8 tensor on the current device")
    _check(call(_ptr(workspace), workspace.numel(), _stream(stream)), name)


def muon_orthogonalize(xs, outs, *, steps=5, workspace=None, stream=None):
    """The nearest-orthogonal factor of each matrix of ``xs`` (all BF16 or all float32) into ``outs`` (BF16 of the same
    shape; may be the BF16 input itself) by ``steps`` Newton-Schulz steps: X = x / |x|_F, then
    X <- aX + (bA + cA^2) X with A = X X^T and (a, b, c) = (3.4445, -4.775, 2.0315); singular values end in about 0.68 to
    1.21. X, A and aI + bA + cA^2 are held in FP16 (11 bits, FP32 accumulation) whatever the type of ``xs``: about 1.3e-3 of the result
    for most matrices, up to 4e-2 where the singular values fall as k^-3. ``workspace``: a uint8 CUDA tensor of muon_workspace_bytes (allocated per call where it is missing)."""
    if not xs or len(xs) != len(outs):
        raise ValueError("xs and outs must be lists of the same length, not empty")
    f32 = xs[0].dtype == torch.float32
    arr, shapes = (_abi.OrthMatrix * len(xs))(), []
    for i, (x, o) in enumerate(zip(xs, outs)):
        if x.dtype != (torch.float32 if f32 else torch.bfloat16) or o.dtype != torch.bfloat16:
            raise ValueError("xs must be all bfloat16 or all float32, outs bfloat16")
        shapes.append(_rows_cols(x, "xs"))
        if o.shape != x.shape:
            raise ValueError("outs must have the shapes of xs")
        arr[i] = _abi.OrthMatrix(_ptr(x), _ptr(o), *shapes[-1])
    _muon_call(shapes, [*xs, *outs], workspace, stream,
               lambda w, n, s: load().muon_orthogonalize(arr, len(xs), int(f32), int(steps), w, n, s),
               "muon_orthogonalize")


def fused_muon_multi_tensor(master, momentum, grads, weights, *, lr, beta=0.95, weight_decay=0.0, update_rms=0.2,
                            loss_scale=1.0, nesterov=True, steps=5, skipped=None, workspace=None, stream=None):
    """One Muon step over lists of matrices (float32 master and momentum, BF16 gradients and weights):

    g = grad / loss_scale; momentum <- beta * momentum + g; u = g + beta * momentum (``nesterov``) or momentum;
    master <- master * (1 - lr * weight_decay) - lr * update_rms * sqrt(max(rows, cols)) * O with O the orthogonal factor
    of u (muon_orthogonalize); weights = BF16 of master. A non-finite u changes nothing and sets ``skipped`` (int32 [1]).
    ``skipped`` is 0 only behind a whole step; where a wait expired or the call itself raised it is 1, and momentum may be new.
    ``workspace``: a uint8 CUDA tensor of muon_workspace_bytes (allocated per call where it is missing)."""
    n = len(master)
    if not n or not n == len(momentum) == len(grads) == len(weights):
        raise ValueError("master, momentum, grads and weights must be lists of the same length, not empty")
    arr, shapes = (_abi.MuonTensor * n)(), []
    for i, (p, m, g, w) in enumerate(zip(master, momentum, grads, weights)):
        if p.dtype != torch.float32 or m.dtype != torch.float32 or g.dtype != torch.bfloat16 or w.dtype != torch.bfloat16:
            raise ValueError("master and momentum must be float32, grads and weights bfloat16")
        shapes.append(_rows_cols(p, "master"))
        if not p.shape == m.shape == g.shape == w.shape:
            raise ValueError("master, momentum, grads and weights must have the same shapes")
        arr[i] = _abi.MuonTensor(_ptr(p), _ptr(m), _ptr(g), _ptr(w), *shapes[-1])
    if skipped is not None and (skipped.dtype != torch.int32 or skipped.numel() < 1):
        raise ValueError("skipped must be int32 [1]")
    _muon_call(shapes, [*master, *momentum, *grads, *weights] + ([] if skipped is None else [skipped]), workspace, stream,
               lambda ws, b, s: load().fused_muon_multi_tensor(arr, n, float(lr), float(beta), float(weight_decay),
                                                               float(update_rms), float(loss_scale), int(bool(nesterov)),
                                                               int(steps), _ptr(skipped), ws, b, s),
               "fused_muon_multi_tensor")


def fp8t_check_device_error(stream=None):
    """Synchronise the stream and raise if a bounded wait in a kernel expired."""
    _check(load().fp8t_check_device_error(_stream(stream)), "fp8t_check_device_error")


def fp8t_debug_expire_waits(mode):
    """Test hook: 1 = every bounded kernel wait expires, 2 = only the GEMM epilogue's, 0 = off."""
    _check(load().fp8t_debug_expire_waits(int(mode)), "fp8t_debug_expire_waits")


def fp8t_set_wait_timeout_ns(ns):
    _check(load().fp8t_set_wait_timeout_ns(int(ns)), "fp8t_set_wait_timeout_ns")
