"""The build: libqmm.so needs hipcc only, whatever becomes of the binding's native calls (CPU only, on a source of one line)."""

import ctypes
import importlib.util
import os
import subprocess

import pytest

from tests.conftest import ROOT


@pytest.fixture
def small(tmp_path, monkeypatch):
    """The build script with one small source, into a folder of its own."""
    spec = importlib.util.spec_from_file_location("_small_build", os.path.join(ROOT, "block_quantized_weight_matmul_amd", "build.py"))
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
