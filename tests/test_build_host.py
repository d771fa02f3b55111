"""The build on the host: what is built without torch's headers or a C++ compiler,
and that a binding of another torch or Python is neither kept nor used."""
import os
import re
import subprocess
import sys
import sysconfig

import pytest
import torch

import attention_jvp_attn_b200 as aj
from attention_jvp_attn_b200 import build, serving

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture()
def runs(monkeypatch, tmp_path):
    """Commands that a build would run; each leaves its output as an empty file."""
    seen = []

    def run(cmd, verbose):
        seen.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w"):
            pass
        return ""

    monkeypatch.setattr(build, "_run", run)
    monkeypatch.setattr(build, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "binding.so"))
    return seen


def test_library_first_then_the_binding(runs):
    assert build.build() == build.LIB
    assert [os.path.basename(c[0]) for c in runs] == ["nvcc", "g++"]


@pytest.mark.parametrize("missing", ["g++", "torch", "Python.h"])
def test_library_is_built_without_the_bindings_needs(runs, monkeypatch, capsys, tmp_path, missing):
    if missing == "g++":
        which = build.shutil.which
        monkeypatch.setattr(build.shutil, "which", lambda name, *a, **k: None if name == "g++" else which(name, *a, **k))
    elif missing == "torch":
        find = build.importlib.util.find_spec
        monkeypatch.setattr(build.importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))
    else:
        monkeypatch.setattr(build.sysconfig, "get_paths", lambda: {"include": str(tmp_path)})
    assert build.build() == build.LIB
    assert [os.path.basename(c[0]) for c in runs] == ["nvcc"]
    assert f"no {missing} here" in capsys.readouterr().err


def test_build_runs_as_a_script_without_torch(tmp_path):
    """The file by itself, in a Python that has no torch: nothing is left to do for a library that is up to date."""
    build.build()
    code = f"""
import sys
sys.modules["torch"] = None
import importlib.util
find = importlib.util.find_spec
importlib.util.find_spec = lambda name, *a: None if name == "torch" else find(name, *a)
spec = find("x") or importlib.util.spec_from_file_location("b", {build.__file__!r})
b = importlib.util.module_from_spec(spec)
spec.loader.exec_module(b)
print(b.build())
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=ROOT)
    assert r.returncode == 0 and r.stdout.strip() == build.LIB, r.stderr
    assert "no torch here" in r.stderr


def test_a_failing_binding_is_an_error(monkeypatch, tmp_path):
    build.build()
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "binding.so"))
    monkeypatch.setattr(build, "BINDING_FLAGS", ["--no-such-flag"])
    with pytest.raises(RuntimeError, match="no-such-flag"):
        build.build()


@pytest.mark.parametrize("changed", ["torch", "python", "flags"])
def test_a_binding_for_something_else_is_built_anew(runs, monkeypatch, changed):
    build.build_binding()
    with open(build.BINDING, "wb") as f:
        f.write(b"..." + build.binding_built_for().encode() + b"\0...")
    del runs[:]
    build.build_binding()
    assert runs == []  # kept
    if changed == "torch":
        monkeypatch.setattr(torch, "__version__", "2.0.0")
    elif changed == "python":
        var = sysconfig.get_config_var
        monkeypatch.setattr(build.sysconfig, "get_config_var", lambda n: ".cpython-39.so" if n == "EXT_SUFFIX" else var(n))
    else:
        monkeypatch.setattr(build, "BINDING_FLAGS", [*build.BINDING_FLAGS, "-g"])
    build.build_binding()
    assert len(runs) == 1
    assert f'-DAJVP_BUILT_FOR="{build.binding_built_for()}"' in runs[0]


def test_a_binding_for_another_torch_is_not_used(monkeypatch):
    build.build()
    monkeypatch.setattr(serving, "_bound", None)
    monkeypatch.setattr(torch, "__version__", "2.0.0")
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(RuntimeError, match=re.escape("built for 'torch ")):
        aj.prompt_attn(x, x, x, x)
    monkeypatch.undo()
    with pytest.raises(ValueError, match="CUDA"):
        aj.prompt_attn(x, x, x, x)
