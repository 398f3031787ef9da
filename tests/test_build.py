"""CPU checks of the in-tree build: the library does not need the binding's native module."""

import subprocess
import sysconfig

import pytest
import torch

from linear_attention_recurrent_selective_b200 import build, ssu


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


def test_the_native_module_belongs_to_one_torch_and_one_python(monkeypatch):
    """A module built against another torch is not taken for this one's: neither by the build
    nor by the binding, which asks for a build instead of loading it."""
    build.build()
    here = build.marshal_path()
    assert ssu._load_marshal().scan_decode
    assert torch.__version__ in here and here.endswith(sysconfig.get_config_var("EXT_SUFFIX"))
    monkeypatch.setattr(torch, "__version__", "0.0.0+other")
    assert build.marshal_path() != here
    with pytest.raises(ssu.SSULibraryMissing, match="build"):
        ssu._load_marshal()
    ran = []
    monkeypatch.setattr(build.subprocess, "run", lambda cmd, **k: (
        ran.append(cmd), subprocess.CompletedProcess(cmd, 1, "", "stop"))[1])
    with pytest.raises(RuntimeError, match="stop"):
        build.build_marshal()
    assert len(ran) == 1
