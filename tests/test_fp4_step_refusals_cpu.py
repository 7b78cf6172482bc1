"""What the step driver's 4-bit recipes do not do is refused or left out, not silently empty (no kernel runs)."""
import pytest
import torch

from optimizer_fp8_cast_b200.monitor import HealthMonitor
from optimizer_fp8_cast_b200.step import Fp8LinearStep
from tests.test_step_config_cpu import HP

FOUR = ("mxfp4", "nvfp4")


def make(recipe, fin=256, fout=160, tokens=192, **kw):
    return Fp8LinearStep([(fin, fout)], tokens, 16, adamw=HP, w_init=[torch.zeros(fin, fout)], device="cpu",
                         recipe=recipe, **kw)


@pytest.mark.parametrize("recipe", FOUR)
def test_counters_are_refused(recipe):
    with pytest.raises(ValueError, match="counters"):
        make(recipe, counters=True)
    assert make(recipe).counters is None and make("delayed", counters=True).counters is not None


@pytest.mark.parametrize("recipe", FOUR)
@pytest.mark.parametrize("size", [dict(fin=144), dict(fout=48), dict(tokens=200)])
def test_sizes_are_refused_at_construction(recipe, size):
    with pytest.raises(ValueError, match="multiples of 32"):
        make(recipe, **size)
    make(recipe, fin=32, fout=96, tokens=32)


@pytest.mark.parametrize("recipe", FOUR)
@pytest.mark.parametrize("transposes", [False, True])
def test_no_8_bit_buffers(recipe, transposes):
    st = make(recipe, transposes=transposes)
    L = st.layers[0]
    assert all(getattr(L, n) is None for n in ("Xq", "Wq", "dYq", "XqT", "WqT", "dYqT"))
    assert not hasattr(st, "gemm_workspace") and L.dW.shape == (256, 160)
    assert make("delayed").layers[0].Xq.numel() == 256 * 192 and make("delayed").gemm_workspace.numel() > 0


@pytest.mark.parametrize("recipe,kept", [("mxfp4", False), ("mxfp8", False), ("nvfp4", True), ("delayed", True)])
def test_monitor_takes_no_amax_that_is_not_kept(recipe, kept):
    """The zeros of a history that nothing fills are no amax: a monitor that averages them looks as if it watched."""
    st = make(recipe)
    mon = HealthMonitor(n_tensors=3, every=1, window=2)
    for st.t in range(4):
        assert mon.maybe_check(st) == []
    assert [len(r) for r in mon.recent] == [2 * kept] * 3
    st.skipped.fill_(1)
    assert [e[0] for e in mon.maybe_check(st)] == ["skip"]
