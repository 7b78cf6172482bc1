"""The build's parts do not stand in one another's way (nothing is compiled here)."""
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


def test_library_that_cannot_be_built_is_an_error(commands):
    seen, missing = commands
    missing.add(build.NVCC)
    with pytest.raises(FileNotFoundError):
        build.build()
    assert seen == [build.NVCC]
