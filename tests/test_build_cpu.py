"""What a build leaves behind, with the compilers' runs replaced by ones that
write their output file or fail."""
import os
import subprocess

import pytest

torch = pytest.importorskip("torch")

from sparse_embedding_exact_gb300 import build  # noqa: E402


class Compilers:
    """Stands in for subprocess.run: records the commands, writes each one's
    output, and fails those that `fails` names."""

    def __init__(self):
        self.commands, self.fails = [], lambda cmd: False

    def run(self, cmd, **kw):
        self.commands.append(cmd)
        if self.fails(cmd):
            return subprocess.CompletedProcess(cmd, 1, "", "fatal error: torch/extension header not found")
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("built")
        return subprocess.CompletedProcess(cmd, 0, "", "")

    def of(self, word):
        return [c for c in self.commands if any(word in a for a in c)]


@pytest.fixture
def compilers(tmp_path, monkeypatch):
    c = Compilers()
    monkeypatch.setattr(build, "BUILD", str(tmp_path))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libsparsecos.so"))
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_dense_binding.so"))
    monkeypatch.setattr(build, "nvcc", lambda: "nvcc")
    monkeypatch.setattr(build.subprocess, "run", c.run)
    return c


def test_build_makes_library_and_binding(compilers):
    assert not build.up_to_date()
    assert build.build() == build.LIB
    assert os.path.exists(build.LIB) and os.path.exists(build.BINDING) and build.up_to_date()
    n = len(compilers.commands)
    build.build()
    assert len(compilers.commands) == n  # nothing left to do


@pytest.mark.parametrize("what", ["binding.cpp", "-ltorch_python"])
def test_library_is_built_where_the_binding_cannot_be(compilers, what):
    compilers.fails = lambda cmd: any(what in a for a in cmd)
    with pytest.raises(RuntimeError, match="binding"):
        build.build()
    assert os.path.exists(build.LIB) and not os.path.exists(build.BINDING)
    # and it is not compiled again for the binding's sake
    compilers.commands.clear()
    compilers.fails = lambda cmd: False
    build.build()
    assert os.path.exists(build.BINDING) and build.up_to_date() and not compilers.of(".cu")


def test_library_failure_is_raised(compilers):
    compilers.fails = lambda cmd: "-shared" in cmd and cmd[0] == "nvcc"
    with pytest.raises(RuntimeError, match="nvcc link failed"):
        build.build()
    assert not os.path.exists(build.LIB)


def test_binding_of_another_torch_is_rebuilt(compilers, monkeypatch):
    build.build()
    compilers.commands.clear()
    monkeypatch.setattr(torch, "__version__", "0.0.1+other")
    assert not build.up_to_date()
    build.build()
    assert build.up_to_date() and not compilers.of(".cu") and compilers.of("binding.cpp")


def test_binding_of_another_torch_is_not_loaded(compilers, monkeypatch):
    from sparse_embedding_exact_gb300 import _abi, dense

    build.build()
    monkeypatch.setattr(dense, "_native", None)
    monkeypatch.setattr(_abi, "load", lambda: None)
    monkeypatch.setattr(torch, "__version__", "0.0.1+other")
    with pytest.raises(ImportError, match="0.0.1"):
        dense._load()
    os.remove(build.BINDING)
    with pytest.raises(ImportError, match="not built"):
        dense._load()
