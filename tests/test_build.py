"""global_attention_b200.build: the C library needs nvcc alone; the binding's module (csrc/torch_calls.cpp) is built where torch
is, again when torch or Python is another one, and its absence is told of without taking the library along."""
import os
import subprocess
import sys

import pytest

from global_attention_b200 import build as B


@pytest.fixture()
def module(monkeypatch, tmp_path):
    """The module's file and note elsewhere, the compiler a stand-in that writes the file and counts."""
    B.build()
    runs = tmp_path / "runs"
    cxx = tmp_path / "cxx"
    cxx.write_text(f"""#!/bin/sh
echo run >> {runs}
while [ "$1" != "-o" ]; do shift; done
echo module > "$2"
""")
    cxx.chmod(0o755)
    monkeypatch.setattr(B, "CALLS", str(tmp_path / "_calls.so"))
    monkeypatch.setattr(B, "CALLS_FOR", str(tmp_path / "_calls.for"), raising=False)
    monkeypatch.setattr(B, "CXX", str(cxx))
    return lambda: len(runs.read_text().splitlines()) if runs.exists() else 0


def test_module_follows_torch_and_python(module, monkeypatch):
    import torch
    B.build()
    B.build()
    assert module() == 1
    monkeypatch.setattr(torch, "__version__", "99.0+other")
    B.build()
    B.build()
    assert module() == 2
    monkeypatch.setattr(B.sysconfig, "get_config_var", lambda name: "another-python")
    B.build()
    assert module() == 3
    os.remove(B.CALLS_FOR)
    B.build()
    assert module() == 4


def test_library_without_torch(module, monkeypatch, capsys):
    monkeypatch.setitem(sys.modules, "torch", None)     # import torch raises ImportError
    assert B.build() == B.LIB and os.path.exists(B.LIB)
    assert module() == 0 and "torch" in capsys.readouterr().err


@pytest.mark.parametrize("compiler", ["/nonexistent/g++", "/bin/false"])
def test_library_without_a_compiler_for_the_module(module, monkeypatch, capsys, compiler):
    """No stale module is left in the place of one that could not be built."""
    B.build()
    os.remove(B.CALLS_FOR)
    monkeypatch.setattr(B, "CXX", compiler)
    assert B.build() == B.LIB
    assert compiler in capsys.readouterr().err and not os.path.exists(B.CALLS)
    with pytest.raises((OSError, RuntimeError)):
        B.build_calls()


def test_missing_module_is_told_of():
    """A call that needs the module says why it is not there and how to get it; the others work without."""
    code = """
import sys
sys.modules["global_attention_b200._calls"] = None
import torch, global_attention_b200 as ga
ga.load()
try:
    ga.zgcm_qk_norm_rope_fwd(*[torch.zeros(1)] * 5)
except RuntimeError as e:
    print(e)
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=B.ROOT)
    assert r.returncode == 0 and "python -m global_attention_b200.build" in r.stdout, r.stderr
