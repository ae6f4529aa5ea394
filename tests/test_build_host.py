"""The build of the library and of its Python binding, on the host."""
import importlib.util
import os
import subprocess
import sys

from bit_nf4_quantized_unpack_b200 import build


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
