"""The build of the library and of its torch side: the C library needs no torch, and the
torch side is one for each torch and Python it is compiled against."""
import os
import subprocess
import sys
import types

import pytest
import torch

from exact_attention_154_b200 import _build, fa


def test_the_library_builds_without_torch(tmp_path):
    _build.build()  # (current, so the child below compiles nothing)
    code = """
import importlib.util, sys
sys.modules["torch"] = None  # as if it were not installed
spec = importlib.util.spec_from_file_location("b", sys.argv[1])
b = importlib.util.module_from_spec(spec)
spec.loader.exec_module(b)
b.BINDING = sys.argv[2]      # (none there yet)
print(b.build() == b.LIB)
"""
    r = subprocess.run([sys.executable, "-c", code, _build.__file__, str(tmp_path / "none.so")],
                       capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "True", r.stderr


def compiles(monkeypatch):
    """What the build compiles, by compiler, instead of compiling it."""
    ran = []

    def run(cmd, **kw):
        ran.append(os.path.basename(cmd[0]))
        open(cmd[cmd.index("-o") + 1], "w").close()
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    monkeypatch.setattr(_build.subprocess, "run", run)
    monkeypatch.setattr(_build.os, "replace", lambda a, b: os.remove(a))
    return ran


@pytest.mark.parametrize("change", ["torch", "abi", "python", "nothing"])
def test_the_binding_belongs_to_its_torch_and_python(monkeypatch, change):
    _build.build()
    ran = compiles(monkeypatch)
    if change == "torch":
        monkeypatch.setattr(torch, "__version__", "99.9.0")
    if change == "abi":
        monkeypatch.setattr(torch._C, "_GLIBCXX_USE_CXX11_ABI", not torch._C._GLIBCXX_USE_CXX11_ABI)
    if change == "python":
        import sysconfig
        monkeypatch.setattr(sysconfig, "get_config_var", lambda name: "cpython-399-other")
    _build.build_binding()
    assert ran == ([] if change == "nothing" else ["g++"])


def test_the_library_comes_first(monkeypatch, tmp_path):
    # a binding that does not compile leaves the library built
    ran = compiles(monkeypatch)
    monkeypatch.setattr(_build, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(_build, "check_register_split", lambda log: None)

    def fail(force=False):
        ran.append("binding")
        raise RuntimeError("g++ failed")

    monkeypatch.setattr(_build, "build_binding", fail)
    with pytest.raises(RuntimeError, match="g\\+\\+ failed"):
        _build.build()
    assert ran == ["nvcc", "binding"]


def test_a_binding_that_is_not_there_or_does_not_load_is_named(monkeypatch, tmp_path):
    _build.build()
    path = str(tmp_path / "_fa_torch-0.so")
    monkeypatch.setattr(fa, "_torch_calls", None)
    monkeypatch.setattr(_build, "binding_path", lambda: path)
    x = torch.zeros(1, 1, 8, 64, dtype=torch.float16)
    with pytest.raises(RuntimeError, match="missing for torch"):
        fa.fwd_sinks(x, x, x, 4, 1)
    with open(path, "w") as f:
        f.write("not a library")
    with pytest.raises(RuntimeError, match="does not load: .*_fa_torch-0.so"):
        fa.fwd_sinks(x, x, x, 4, 1)
