"""The build of the library and of its Python binding, on the host."""
import importlib.util
import os
import subprocess
import sys

import pytest
import torch

from bit_nf4_quantized_unpack_b200 import build, qlora


def test_library_builds_without_torch(tmp_path):
    """build.py run as a script in an interpreter that has no torch: the C library alone."""
    build.build()
    code = ("import runpy, sys, importlib.util as u\n"
            "find = u.find_spec\n"
            "u.find_spec = lambda name, *a: None if name == 'torch' else find(name, *a)\n"
            "sys.modules['torch'] = None\n"
            "sys.argv = ['build.py']\n"
            f"runpy.run_path({build.__file__!r}, run_name='__main__')\n")
    res = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=tmp_path)
    assert res.returncode == 0, res.stderr
    assert res.stdout.strip() == build.LIB and "left out" in res.stderr


def test_binding_is_left_out_without_headers(monkeypatch, tmp_path, capsys):
    spec = importlib.util.spec_from_file_location("torch", os.path.join(tmp_path, "torch", "__init__.py"))
    monkeypatch.setattr(build.importlib.util, "find_spec", lambda name: spec)
    assert build.build_binding(force=True) is None
    assert "pybind.h" in capsys.readouterr().err


def test_binding_is_compiled_again_for_another_torch(monkeypatch, tmp_path):
    """By what it was compiled for, not by the files' times alone."""
    calls = []

    def compiler(cmd, **_):
        calls.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")
    monkeypatch.setattr(build.subprocess, "run", compiler)
    monkeypatch.setattr(build, "OBJ", str(tmp_path / "obj"))
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "lib" / "qlora_binding.so"))
    build.build_binding()
    build.build_binding()
    assert len(calls) == 1
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    build.build_binding()
    build.build_binding()
    assert len(calls) == 2


def test_binding_of_another_torch_is_refused(monkeypatch):
    build.build()
    monkeypatch.setattr(qlora, "_binding", None)
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    with pytest.raises(RuntimeError, match="built for torch"):
        qlora.binding()
    assert qlora._binding is None
