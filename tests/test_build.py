"""The build: the library without the binding's needs, and a binding that does
not outlive the PyTorch it was built against."""

import os
import sys

import pytest
import torch

from paged_kv_cache_222_gb300 import build as B


@pytest.fixture
def elsewhere(tmp_path, monkeypatch):
    """A build of one quick source into a folder of its own."""
    monkeypatch.setattr(B, "BUILD_DIR", str(tmp_path / "_build"))
    monkeypatch.setattr(B, "LIB_PATH", str(tmp_path / "libpkv.so"))
    monkeypatch.setattr(B, "BINDING_PATH", str(tmp_path / "_binding.so"))
    monkeypatch.setattr(B, "SOURCES", ["block_manager.cpp"])
    return tmp_path


def _no_headers(out):
    return [sys.executable, "-c", "import sys; print('Python.h: No such file or directory'); sys.exit(1)"]


def _no_torch(out):
    raise ImportError("No module named 'torch'")


def _no_compiler(out):
    return ["/nonexistent/g++"]


@pytest.mark.parametrize("command,why", [(_no_headers, "Python.h"), (_no_torch, "torch"), (_no_compiler, "g++")])
def test_the_library_does_not_need_the_binding(elsewhere, monkeypatch, capfd, command, why):
    monkeypatch.setattr(B, "_binding_command", command)
    (elsewhere / "_binding.so").write_bytes(b"of older sources")
    assert B.build(force=True) == str(elsewhere / "libpkv.so")
    assert os.path.getsize(elsewhere / "libpkv.so") > 0
    assert not (elsewhere / "_binding.so").exists()          # a stale one is not left to be loaded
    assert why in capfd.readouterr().err
    assert not B.up_to_date()                                # tried again next time


def test_sources_that_do_not_compile_still_fail_the_build(elsewhere, monkeypatch):
    monkeypatch.setattr(B, "_binding_command", _no_headers)
    monkeypatch.setattr(B, "SOURCES", ["no_such_source.cpp"])
    with pytest.raises(RuntimeError):
        B.build(force=True)


def test_a_binding_of_another_pytorch_is_out_of_date(elsewhere, monkeypatch):
    def touch(out):
        return [sys.executable, "-c", f"open({out!r}, 'w').write('binding')"]
    monkeypatch.setattr(B, "_binding_command", touch)
    B.build(force=True)
    assert B.up_to_date()
    monkeypatch.setattr(torch, "__version__", torch.__version__ + ".another")
    assert not B.up_to_date()
    before = os.stat(elsewhere / "libpkv.so").st_mtime_ns
    B.build()                                                # the binding alone
    assert B.up_to_date()
    assert os.stat(elsewhere / "libpkv.so").st_mtime_ns == before
