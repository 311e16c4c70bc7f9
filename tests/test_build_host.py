"""The build without its optional parts (no compiler is run: the commands are recorded): the C library needs nvcc alone, the
torch wrappers are left out where torch or g++ is missing, and a wrapper that does not compile is reported once the C
library is linked."""
import importlib.util
import os
import shutil
import subprocess
import types

import pytest

from block_quantized_weight_pn3t_gb300 import build


@pytest.fixture
def recorded(monkeypatch, tmp_path):
    """The commands that build() runs, each made to succeed and to leave its output (unless `fails` says otherwise)."""
    rec = types.SimpleNamespace(commands=[], fails=lambda cmd: False)

    def run(cmd, **_):
        rec.commands.append(cmd)
        if rec.fails(cmd):
            return types.SimpleNamespace(returncode=1, stdout="", stderr="no")
        with open(cmd[cmd.index("-o") + 1], "w"):
            pass
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    monkeypatch.setattr(build, "BUILD_DIR", str(tmp_path / "objects"))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libpnq.so"))
    monkeypatch.setattr(build, "NATIVE", str(tmp_path / "_native.so"))
    monkeypatch.setattr(build, "nvcc", lambda: "/usr/local/cuda/bin/nvcc")
    monkeypatch.setattr(subprocess, "run", run)
    return rec


def nvcc_compiles(rec):
    return [c for c in rec.commands if c[0].endswith("nvcc") and "-c" in c]


def test_with_torch_and_gxx(recorded):
    if shutil.which("g++") is None:
        pytest.skip("g++ not found")
    build.build()
    assert len(nvcc_compiles(recorded)) == len(build.SOURCES)
    assert sum(c[0] == "g++" for c in recorded.commands) == 2  # compile and link of the wrappers
    assert os.path.exists(build.LIB) and os.path.exists(build.NATIVE)
    recorded.commands.clear()
    build.build()
    assert recorded.commands == []


@pytest.mark.parametrize("missing", ["torch", "g++"])
def test_the_c_library_needs_nvcc_alone(recorded, monkeypatch, capsys, missing):
    spec, which = importlib.util.find_spec, shutil.which
    monkeypatch.setattr(importlib.util, "find_spec", lambda n, *a: None if n == missing else spec(n, *a))
    monkeypatch.setattr(shutil, "which", lambda n, *a, **k: None if n == missing else which(n, *a, **k))
    assert build.build() == build.LIB
    assert len(nvcc_compiles(recorded)) == len(build.SOURCES) and not any(c[0] == "g++" for c in recorded.commands)
    assert os.path.exists(build.LIB) and not os.path.exists(build.NATIVE)
    assert f"{missing} not found" in capsys.readouterr().out


def test_a_failing_wrapper_leaves_the_c_library(recorded):
    if shutil.which("g++") is None:
        pytest.skip("g++ not found")
    recorded.fails = lambda cmd: any(a.endswith("pnq_torch.cpp") for a in cmd)
    with pytest.raises(RuntimeError, match="pnq_torch.cpp"):
        build.build()
    assert os.path.exists(build.LIB) and not os.path.exists(build.NATIVE)


def test_a_failing_kernel_stops_the_build(recorded):
    recorded.fails = lambda cmd: any(a.endswith("pnq_experts.cu") for a in cmd)
    with pytest.raises(RuntimeError, match="pnq_experts.cu"):
        build.build()
    assert not os.path.exists(build.LIB)
