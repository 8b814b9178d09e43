"""The native argument marshalling belongs to one interpreter, and the package is whole without it."""
import importlib.machinery
import os
import shutil
import subprocess
import sys

import __graft_entry__
import mixed_precision_numerics_gb300 as M
from tests.conftest import ROOT

PKG = os.path.join(ROOT, "mixed_precision_numerics_gb300")
TAGGED = "_mpcall" + importlib.machinery.EXTENSION_SUFFIXES[0]


def copy_of_package(tmp_path, *files):
    to = tmp_path / "mixed_precision_numerics_gb300"
    to.mkdir()
    for f in ("__init__.py", "build.py", "libmpnum.so", *files):
        shutil.copy2(os.path.join(PKG, f), to / f)
    return to


def run(tmp_path, code):
    env = dict(os.environ, PYTHONPATH=str(tmp_path))
    p = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, env=env, cwd=tmp_path, timeout=300)
    assert p.returncode == 0, p.stderr
    return p.stdout


CALLS = """
import torch
import mixed_precision_numerics_gb300 as M
assert {native}
x, s, y = torch.zeros(4, 256), torch.zeros(4, 2), torch.zeros(4, 256, dtype=torch.uint8)
for call in (lambda: M.rmsnorm_residual_fp8(x, x[0], y, s), lambda: M.swiglu_fp8(x, x, y, s),
             lambda: M.rmsnorm_residual_backward(x, x[0], s[0], x, x[0], y, h=x),
             lambda: M.swiglu_backward(x, x, x, gate=x, up=x)):
    try:
        call()
    except ValueError as e:
        assert "CUDA" in str(e)
    else:
        raise AssertionError("a host tensor was taken")
"""


def test_the_file_carries_the_interpreters_tag():
    build = __graft_entry__._package_builder()
    assert os.path.basename(build.CALL) == TAGGED != "_mpcall.so"
    if os.path.exists(build.PYTHON_H):
        assert os.path.exists(build.CALL) and M._mpcall is not None
    assert not os.path.exists(os.path.join(PKG, "_mpcall.so"))


def test_the_package_imports_without_the_extension(tmp_path):
    copy_of_package(tmp_path)
    run(tmp_path, CALLS.format(native="M._mpcall is None"))


def test_an_extension_of_another_interpreter_is_not_loaded(tmp_path):
    to = copy_of_package(tmp_path)
    for name in ("_mpcall.so", "_mpcall.cpython-311-" + TAGGED.split("-", 2)[-1]):
        (to / name).write_bytes(b"not of this interpreter")
    run(tmp_path, CALLS.format(native="M._mpcall is None"))


def test_it_is_up_to_date_for_its_own_interpreter_only(tmp_path, monkeypatch):
    build = __graft_entry__._package_builder()
    monkeypatch.setattr(build, "CALL", str(tmp_path / TAGGED))
    monkeypatch.setattr(build, "UNTAGGED", str(tmp_path / "_mpcall.so"))
    monkeypatch.setattr(build, "PYTHON_H", build.__file__)  # a file that is there
    assert build._call_stale()
    (tmp_path / TAGGED).write_bytes(b"")
    assert not build._call_stale()
    (tmp_path / "_mpcall.so").write_bytes(b"")
    assert build._call_stale()


def test_without_the_headers_nothing_old_stays(tmp_path, monkeypatch, capsys):
    build = __graft_entry__._package_builder()
    monkeypatch.setattr(build, "CALL", str(tmp_path / TAGGED))
    monkeypatch.setattr(build, "UNTAGGED", str(tmp_path / "_mpcall.so"))
    monkeypatch.setattr(build, "PYTHON_H", str(tmp_path / "Python.h"))
    assert not build._call_stale()  # nothing to build and nothing to remove
    for f in (build.CALL, build.UNTAGGED):
        open(f, "wb").close()
    build._compile_call()
    assert os.listdir(tmp_path) == [] and "not built" in capsys.readouterr().err
