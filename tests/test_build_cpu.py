"""The build's parts do not stand in one another's way (nothing is compiled here)."""
import os
import subprocess

import pytest

from optimizer_fp8_cast_b200 import build


@pytest.fixture
def commands(monkeypatch, tmp_path):
    """Compiler calls are recorded, not made; `missing` names a compiler that is not installed."""
    seen = []

    def run(cmd, check):
        seen.append(cmd[0])
        if cmd[0] in commands_missing:
            raise FileNotFoundError(cmd[0])
        with open(cmd[cmd.index("-o") + 1], "wb"):
            pass
    commands_missing = set()
    monkeypatch.setattr(subprocess, "run", run)
    monkeypatch.setattr(build, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "binding.so"))
    return seen, commands_missing


def test_library_is_built_where_the_extension_cannot_be(commands):
    seen, missing = commands
    missing.add(build.CXX)
    with pytest.warns(RuntimeWarning, match="norm and 4-bit calls are missing"):
        assert build.build() == build.LIB
    assert seen == [build.NVCC, build.CXX]


def test_an_extension_that_cannot_be_rebuilt_does_not_stay(commands):
    """Its calls raise then, instead of passing the new library structures of an older header."""
    _, missing = commands
    with open(build.BINDING, "wb") as f:
        f.write(b"older")
    missing.add(build.CXX)
    with pytest.warns(RuntimeWarning):
        build.build()
    assert not os.path.exists(build.BINDING)


def test_library_that_cannot_be_built_is_an_error(commands):
    seen, missing = commands
    missing.add(build.NVCC)
    with pytest.raises(FileNotFoundError):
        build.build()
    assert seen == [build.NVCC]


def test_extension_is_rebuilt_for_another_torch(commands, monkeypatch):
    """It is compiled against torch's private C++ headers: a newer file alone does not make it the right one."""
    seen, _ = commands
    build.build_binding()
    with open(build.BINDING, "wb") as f:                 # what the compiler writes holds the versions
        f.write(b"\x7fELF " + build.binding_key().encode() + b"\0")
    build.build_binding()
    assert seen == [build.CXX]                           # current: not compiled again
    import torch
    monkeypatch.setattr(torch, "__version__", torch.__version__ + ".other")
    build.build_binding()
    assert seen == [build.CXX] * 2


def test_extension_of_another_torch_is_refused(monkeypatch):
    import optimizer_fp8_cast_b200 as fp8
    build.build_library()
    build.build_binding()
    import torch
    assert fp8._load_binding().built_for == build.binding_key()
    monkeypatch.setattr(torch, "__version__", "0.0.other")
    with pytest.raises(RuntimeError, match="was built for"):
        fp8._load_binding()
