"""The module that the microscaled operators' Python calls go through needs
PyTorch's and Python's headers and a host compiler; the library and the calls
that were there without it do not."""
import importlib.util
import os
import subprocess
import sys

import pytest

import mxfp4_routed_expert_k3mx_gb300 as k3mx
from mxfp4_routed_expert_k3mx_gb300 import _build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_library_builds_without_the_binding(monkeypatch, tmp_path):
    """A compiler that fails: a warning with the reason, the library's path, and
    no older module in the place of the one that was not built."""
    out = tmp_path / "binding.so"
    monkeypatch.setattr(_build, "binding_path", lambda: str(out))
    monkeypatch.setenv("CXX", "false")
    out.write_bytes(b"an older one")
    os.utime(out, (1, 1))
    with pytest.warns(UserWarning, match="k3mx_mx.h are not available"):
        assert _build.build() == _build.LIB
    assert os.path.exists(_build.LIB) and not out.exists()
    # and where the library itself is compiled and linked
    (tmp_path / "one.cu").write_text("__global__ void k() {}\n")
    monkeypatch.setattr(_build, "sources", lambda: [str(tmp_path / "one.cu")])
    monkeypatch.setattr(_build, "BUILD", str(tmp_path))
    monkeypatch.setattr(_build, "LIB", str(tmp_path / "libk3mx.so"))
    with pytest.warns(UserWarning, match="binding.cpp"):
        assert os.path.exists(_build.build())
    with pytest.raises(RuntimeError, match="is missing"):
        k3mx._load_binding()


def test_library_builds_without_pytorch():
    """_build.py by itself, in a Python where PyTorch cannot be imported."""
    code = ("import importlib.util, sys, warnings; sys.modules['torch'] = None; warnings.simplefilter('ignore')\n"
            f"s = importlib.util.spec_from_file_location('b', {_build.__file__!r})\n"
            "m = importlib.util.module_from_spec(s); s.loader.exec_module(m); assert m.build() == m.LIB; print('built')")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=ROOT)
    assert r.returncode == 0 and "built" in r.stdout, r.stderr
    assert importlib.util.find_spec("torch") is not None


def test_binding_is_rebuilt_after_any_header(monkeypatch, tmp_path):
    """binding.cpp includes k3mx_mx.h, which includes k3mx.h."""
    out = tmp_path / "binding.so"
    monkeypatch.setattr(_build, "binding_path", lambda: str(out))
    monkeypatch.setenv("CXX", "false")
    include = tmp_path / "include"
    include.mkdir()
    for name in ("k3mx.h", "k3mx_mx.h"):
        (include / name).write_text("")
        os.utime(include / name, (5, 5))
    (tmp_path / "binding.cpp").write_text("")
    os.utime(tmp_path / "binding.cpp", (5, 5))
    out.write_bytes(b"x")
    os.utime(out, (6, 6))
    monkeypatch.setattr(_build, "INCLUDE", str(include))
    monkeypatch.setattr(_build, "CSRC", str(tmp_path))
    assert _build.build_binding() == str(out)
    os.utime(include / "k3mx.h", (7, 7))
    with pytest.raises(RuntimeError):
        _build.build_binding()
