"""The build of the library beside that of the PyTorch binding (commands are
recorded, none is run)."""
from __future__ import annotations

import importlib.machinery
import os

import pytest

from memory_bound_normalization_gb300 import build as b


@pytest.fixture
def recorded(monkeypatch, tmp_path):
    """Build folders of the test's own; what is run and linked is kept."""
    seen = {"run": [], "linked": []}
    monkeypatch.setattr(b, "BUILD_DIR", str(tmp_path / "build"))
    monkeypatch.setattr(b, "BINDING_PATH", str(tmp_path / "build" / "_binding.so"))

    def run(cmd, log):
        seen["run"].append(cmd)
        if "-o" in cmd:
            open(cmd[cmd.index("-o") + 1], "w").close()

    monkeypatch.setattr(b, "_run", run)
    monkeypatch.setattr(b, "_link", lambda objs, checked: seen["linked"].append(checked))
    return seen


def torch_at(monkeypatch, path):
    spec = importlib.machinery.ModuleSpec("torch", None, is_package=True)
    spec.submodule_search_locations.append(str(path))
    real = importlib.util.find_spec
    monkeypatch.setattr(b.importlib.util, "find_spec", lambda n: spec if n == "torch" else real(n))


def compiled_binding(seen):
    return any(b.BINDING_SOURCE in cmd for cmd in seen["run"])


def test_pytorch_without_cuda(monkeypatch, tmp_path, recorded):
    """A PyTorch that lacks CUDA has no use for the binding: the library is built
    without it."""
    (tmp_path / "torch" / "lib").mkdir(parents=True)
    torch_at(monkeypatch, tmp_path / "torch")
    b.build(force=True)
    assert recorded["linked"] == [False] and not compiled_binding(recorded)
    assert not b.binding_is_stale()


def test_binding_that_does_not_compile(monkeypatch, recorded):
    """The library is linked all the same, and the failure is raised."""
    def fail():
        raise RuntimeError("no such header")

    monkeypatch.setattr(b, "_build_binding", fail)
    with pytest.raises(RuntimeError, match="no such header"):
        b.build(force=True, both=True)
    assert recorded["linked"] == [False, True]


def test_binding_of_another_pytorch_is_stale(monkeypatch, recorded):
    if b._torch_dir() is None:
        pytest.skip("needs a PyTorch with CUDA")
    assert b.binding_is_stale()
    b.build(force=True)
    assert compiled_binding(recorded) and not b.binding_is_stale()
    made_for = b._binding_made_for()
    monkeypatch.setattr(b, "_binding_made_for", lambda: made_for + " of another version")
    assert b.binding_is_stale()
    os.remove(b.BINDING_PATH + ".info")
    monkeypatch.setattr(b, "_binding_made_for", lambda: made_for)
    assert b.binding_is_stale()
