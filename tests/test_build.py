"""CPU checks of the in-tree build: the library does not need the binding's native module."""

import subprocess

import pytest

from linear_attention_recurrent_selective_b200 import build


def test_the_library_builds_without_the_native_module(monkeypatch):
    """Neither a missing compiler or header of the module nor a torch without CUDA keeps the
    library from being built; the module's failure is reported."""
    build.build()

    def fail(force=False):
        raise RuntimeError("g++ failed on marshal.cpp: no c10_cuda")
    monkeypatch.setattr(build, "build_marshal", fail)
    with pytest.warns(UserWarning, match="c10_cuda"):
        assert build.build() == build.LIB


def test_the_native_module_reports_a_failed_build(monkeypatch):
    build.build()
    bad = subprocess.CompletedProcess([], 1, "", "cannot find -lc10_cuda")
    monkeypatch.setattr(build.subprocess, "run", lambda *a, **k: bad)
    with pytest.raises(RuntimeError, match="c10_cuda"):
        build.build_marshal(force=True)
