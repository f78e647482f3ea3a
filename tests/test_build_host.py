"""The extension of the paged cache calls is a choice: the build goes on
without it, and it never serves a torch that it was not built for."""
import os
import subprocess
import sys
import types

import pytest
import torch

import kv_cache_compression_sfa_b200 as sfa
from kv_cache_compression_sfa_b200 import build as sfa_build


@pytest.fixture
def place(tmp_path, monkeypatch):
    monkeypatch.setattr(sfa_build, "FAST_LIB", str(tmp_path / "_fast.so"))
    monkeypatch.setattr(sfa_build, "FAST_STAMP", str(tmp_path / "stamp" / "built_for"))
    monkeypatch.setattr(sfa_build, "BUILD_DIR", str(tmp_path / "stamp"))
    return tmp_path


def _compiler(runs, error=None):
    def run(cmd, check):
        runs.append(cmd)
        if error:
            raise error
        open(cmd[cmd.index("-o") + 1], "wb").close()
    return run


@pytest.mark.parametrize("error", [FileNotFoundError("g++"), subprocess.CalledProcessError(1, "g++")])
def test_a_build_without_compiler_or_headers_goes_on(place, monkeypatch, error):
    (place / "_fast.so").write_bytes(b"of other sources")
    monkeypatch.setattr(subprocess, "run", _compiler([], error))
    with pytest.warns(UserWarning, match="ctypes"):
        assert sfa_build.build_fast() is None
    assert not os.path.exists(sfa_build.FAST_LIB)


def test_another_torch_builds_it_again(place, monkeypatch):
    runs = []
    monkeypatch.setattr(subprocess, "run", _compiler(runs))
    assert sfa_build.build_fast() == sfa_build.FAST_LIB and len(runs) == 1
    assert sfa_build.build_fast() == sfa_build.FAST_LIB and len(runs) == 1
    monkeypatch.setattr(torch, "__version__", "9.9.9")
    assert sfa_build.build_fast() == sfa_build.FAST_LIB and len(runs) == 2
    assert any("9.9.9" in a for a in runs[-1])


@pytest.mark.parametrize("built_for,served", [("this", True), ("torch 0.0.0, Python 3.0", False), (None, False)])
def test_a_module_of_another_torch_is_left_alone(monkeypatch, built_for, served):
    fake = types.ModuleType("fake")
    if built_for:
        fake.built_for = sfa_build.fast_stamp() if built_for == "this" else built_for
    monkeypatch.setattr(sfa, "_fast", fake)
    monkeypatch.setitem(sys.modules, sfa.__name__ + "._fast", fake)
    assert (sfa._load_fast() is fake) == served


def test_it_is_built_here():
    sfa_build.build()
    assert sfa_build.build_fast() is not None
    code = "import kv_cache_compression_sfa_b200 as s; assert s._fast is not None and s._fast.built_for"
    subprocess.run([sys.executable, "-c", code], check=True, cwd=sfa_build.ROOT)
