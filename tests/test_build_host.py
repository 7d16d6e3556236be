"""The build of the fused GEMMs' binding (no GPU): what makes it stale, and a binding of another torch at run time."""
import os
import sys
import types

import pytest
import torch

import block_scaled_precision_05_b200 as bsp
from block_scaled_precision_05_b200 import _native as nat
from block_scaled_precision_05_b200.csrc import build


@pytest.fixture
def compiled(monkeypatch, tmp_path):
    """The build with its outputs in an empty folder and the compiler replaced by one that writes the file it is asked for."""
    runs = []

    def run(cmd, **kw):
        runs.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").write("built")
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_fused_binding.so"))
    monkeypatch.setattr(build, "BINDING_STAMP", str(tmp_path / "stamp"), raising=False)
    monkeypatch.setattr(build.subprocess, "run", run)
    return runs


def test_binding_is_rebuilt_for_another_torch(compiled, monkeypatch):
    build._build_binding(False)
    build._build_binding(False)
    assert len(compiled) == 1  # nothing changed
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    build._build_binding(False)
    build._build_binding(False)
    assert len(compiled) == 2


def test_binding_of_another_torch_is_refused(monkeypatch):
    """A binding that still loads, but was compiled against another torch, is not run."""
    other = types.ModuleType("block_scaled_precision_05_b200._fused_binding")
    other.built_for, other.fused_gemm = "torch 0.0.1 cxx11abi=1 cpython-312", lambda *a: 0
    monkeypatch.setattr(nat, "_fused_gemm", None)
    monkeypatch.setitem(sys.modules, other.__name__, other)
    monkeypatch.setattr(bsp, "_fused_binding", other, raising=False)
    with pytest.raises(RuntimeError, match="another torch"):
        nat.fused_gemm()


def test_binding_in_place_is_this_torchs():
    assert os.path.exists(build.BINDING)
    nat.fused_gemm()
    assert sys.modules["block_scaled_precision_05_b200._fused_binding"].built_for == build.binding_target()


@pytest.mark.parametrize("lacks", ["torch", "g++", "Python.h"])
def test_library_builds_without_what_the_binding_needs(compiled, monkeypatch, capsys, tmp_path, lacks):
    """libbsp.so is for C programs too: its build needs no torch, no Python headers and no g++."""
    if lacks == "torch":
        find = build.importlib.util.find_spec
        monkeypatch.setattr(build.importlib.util, "find_spec", lambda n, *a: None if n == "torch" else find(n, *a))
    elif lacks == "g++":
        which = build.shutil.which
        monkeypatch.setattr(build.shutil, "which", lambda n, *a, **k: None if n == "g++" else which(n, *a, **k))
    else:
        monkeypatch.setattr(build.sysconfig, "get_paths", lambda *a, **k: {"include": str(tmp_path / "none")})
    monkeypatch.setattr(build, "BUILD_DIR", str(tmp_path / "build"))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libbsp.so"))
    assert build.build() == build.LIB and os.path.exists(build.LIB)
    assert not os.path.exists(build.BINDING) and lacks in capsys.readouterr().err
    assert all("g++" not in c[0] for c in compiled)
