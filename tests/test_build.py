"""The build without PyTorch: the C library needs nvcc alone, and a fault of the Python module does not
cost it (the compilers are stood in for; what they are called with is looked at)."""
import os
import subprocess
import sys

import pytest

from block_sparse_long_infllm_gb300 import build


@pytest.fixture
def elsewhere(tmp_path, monkeypatch):
    """A build into tmp_path whose compilers only leave their output files; calls are logged."""
    calls = []

    def run(cmd, **kw):
        calls.append(cmd)
        if "fail" in calls[0] and cmd[0] != build._nvcc():
            return subprocess.CompletedProcess(cmd, 1, "", "no such header")
        open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(build, "LIB_PATH", str(tmp_path / "libinfllmv2.so"))
    monkeypatch.setattr(build, "BINDING_PATH", str(tmp_path / "_binding.so"))
    monkeypatch.setattr(build, "BUILD_DIR", str(tmp_path / "objects"))
    monkeypatch.setattr(build.subprocess, "run", run)
    return calls


def test_library_builds_without_torch(elsewhere, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)  # import torch raises
    assert build.build() == build.LIB_PATH
    assert os.path.exists(build.LIB_PATH) and not os.path.exists(build.BINDING_PATH)
    assert len(elsewhere) == len(build.SOURCES) + 1 and all(c[0] == build._nvcc() for c in elsewhere)
    build.build()
    assert len(elsewhere) == len(build.SOURCES) + 1  # nothing is out of date


def test_binding_is_built_where_torch_is(elsewhere):
    build.build()
    assert os.path.exists(build.LIB_PATH) and os.path.exists(build.BINDING_PATH)
    n = len(elsewhere)
    build.build()
    assert len(elsewhere) == n
    os.remove(build.BINDING_PATH)
    build.build()
    assert os.path.exists(build.BINDING_PATH)


def test_fault_of_the_binding_leaves_the_library(elsewhere):
    elsewhere.append(["fail"])
    with pytest.raises(RuntimeError, match="binding.cpp"):
        build.build()
    assert os.path.exists(build.LIB_PATH) and not os.path.exists(build.BINDING_PATH)
