"""The build: libqmm.so needs hipcc only, whatever becomes of the binding's native calls (CPU only, on a source of one line)."""

import ctypes
import importlib.util
import os
import shutil
import subprocess
import sys

import pytest

from tests.conftest import ROOT

PACKAGE = os.path.join(ROOT, "block_quantized_weight_matmul_amd")


@pytest.fixture
def small(tmp_path, monkeypatch):
    """The build script with one small source, into a folder of its own."""
    spec = importlib.util.spec_from_file_location("_small_build", os.path.join(PACKAGE, "build.py"))
    b = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(b)
    (tmp_path / "one.hip").write_text('extern "C" int one() { return 1; }\n')
    for name, value in (("BUILD", tmp_path / "objects"), ("LIB", tmp_path / "libqmm.so"), ("CALLS", tmp_path / "_calls.so")):
        monkeypatch.setattr(b, name, str(value))
    monkeypatch.setattr(b, "sources", lambda: [str(tmp_path / "one.hip")])
    return b


@pytest.mark.parametrize("error", [ImportError("no torch"), FileNotFoundError("g++"), RuntimeError("g++ on calls.cpp failed")])
def test_library_without_the_native_calls(small, error, monkeypatch, capsys):
    def fails(verbose):
        raise error
    monkeypatch.setattr(small, "_compile_calls", fails)
    with open(small.CALLS, "w") as f:
        f.write("of an earlier build")
    assert small.build() == small.LIB
    assert ctypes.CDLL(small.LIB).one() == 1
    assert not os.path.exists(small.CALLS)  # it would have taken the earlier library's arguments
    assert "_calls.so is not built" in capsys.readouterr().err


def test_a_library_that_does_not_compile_raises(small, monkeypatch):
    monkeypatch.setattr(small, "_compile_calls", lambda verbose: ["never linked"])
    with open(small.sources()[0], "w") as f:
        f.write("this is no source\n")
    with pytest.raises(RuntimeError, match="hipcc failed"):
        small.build()


def test_both_where_both_can_be_built(small, tmp_path, monkeypatch):
    obj = str(tmp_path / "calls.o")
    subprocess.run(["g++", "-x", "c++", "-fPIC", "-c", "-", "-o", obj], input='extern "C" int two() { return 2; }', text=True, check=True)
    monkeypatch.setattr(small, "_compile_calls", lambda verbose: [obj])
    small.build()
    assert ctypes.CDLL(small.LIB).one() == 1 and ctypes.CDLL(small.CALLS).two() == 2


@pytest.mark.skipif(not os.path.exists(os.path.join(PACKAGE, "_calls.so")), reason="_calls.so is not built")
def test_native_calls_of_another_torch_are_refused(tmp_path):
    """The module compares the torch it was built for with the one that is there, before anything of either is used."""
    shutil.copy(os.path.join(PACKAGE, "_calls.so"), tmp_path)
    os.symlink(os.path.join(PACKAGE, "libqmm.so"), tmp_path / "libqmm.so")
    code = "import torch, sys; sys.path.insert(0, '.'); torch.__version__ = sys.argv[1] or torch.__version__; import _calls; print('loaded')"

    def load(version):
        return subprocess.run([sys.executable, "-c", code, version], cwd=tmp_path, capture_output=True, text=True)

    assert load("").stdout == "loaded\n"
    other = load("1.13.0")
    assert other.returncode == 1 and "ImportError: built for torch and Python" in other.stderr
