"""The build names what failed, and does not need the Python binding's parts for the C library (no GPU is touched)."""
import os
import subprocess
import sys

import pytest

import __graft_entry__ as entry
from mixture_experts_expert_histogram_amd import _lib, build

OK = [sys.executable, "-c", "pass"]
FAIL = [sys.executable, "-c", "raise SystemExit('no such header')"]


def test_failures_are_named(capfd):
    build.run_all("anything", [("a", OK), ("b", OK)])
    with pytest.raises(RuntimeError, match="^compiling the x failed: b, c$"):
        build.run_all("compiling the x", [("a", OK), ("b", FAIL), ("c", FAIL)])
    assert "no such header" in capfd.readouterr().err


def test_library_first_and_without_torch(monkeypatch, tmp_path):
    """Commands of a build, none of them run: the library's are hipcc's alone, and it is in place before the binding's start."""
    lib, made = str(tmp_path / "lib.so"), []
    monkeypatch.setattr(build, "BUILD", str(tmp_path))
    monkeypatch.setattr(build, "LIB_PATH", lib)

    def run_all(what, jobs, verbose=False):
        made.append(what)
        for _, cmd in jobs:
            if cmd[0] == "g++":
                raise RuntimeError(what + " failed")
            open(cmd[cmd.index("-o") + 1], "w").close()
    monkeypatch.setattr(build, "run_all", run_all)
    monkeypatch.setattr(build, "binding_commands", lambda obj, out: (["g++"], ["g++"]))
    with pytest.raises(RuntimeError, match="binding"):
        build.build()
    assert os.path.exists(lib) and made == ["HIP compilation", "linking the library", "compiling the Python binding (g++)"]

    def no_torch(obj, out):
        raise AssertionError("the library asked for the binding's commands")
    monkeypatch.setattr(build, "binding_commands", no_torch)
    assert build.build_library() == lib


def test_entry_point_loads_the_binding(monkeypatch):
    loaded = []
    monkeypatch.setattr(build, "build", lambda: None)
    monkeypatch.setattr(_lib, "_block", lambda: loaded.append(1))
    entry.build()
    assert loaded


def test_module_is_loadable_by_itself():
    """In a process of its own, as a first import."""
    code = "import mixture_experts_expert_histogram_amd as m; print(m._lib._block().__name__)"
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    out = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert out.returncode == 0 and "_block" in out.stdout, out.stderr
