"""What the build makes, and what it leaves where a part of it fails."""

import ctypes as C
import os
import sys
import sysconfig

import pytest
import torch

import mla_chunked_context_gb300 as M
from mla_chunked_context_gb300 import _lib, build


@pytest.fixture
def small(tmp_path, monkeypatch):
    """The build's outputs in a folder of their own, of one short source."""
    src = tmp_path / "one.cpp"
    src.write_text('extern "C" __attribute__((visibility("default"))) int one() { return 1; }\n')
    monkeypatch.setattr(build, "_sources", lambda: [str(src)])
    monkeypatch.setattr(build, "BUILD", str(tmp_path / "obj"))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libone.so"))
    monkeypatch.setattr(build, "MODULE", str(tmp_path / os.path.basename(build.MODULE)))
    monkeypatch.setattr(build, "HERE", str(tmp_path))
    return tmp_path


def test_library_stays_built_where_the_module_fails(small, monkeypatch):
    def fails():
        raise RuntimeError("no headers")
    monkeypatch.setattr(build, "_compile_module", fails)
    with pytest.raises(RuntimeError, match="no headers"):
        build.build()
    assert C.CDLL(build.LIB).one() == 1
    assert not os.path.exists(build.MODULE)


def test_library_alone_needs_no_torch(small, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)
    assert C.CDLL(build.build_library()).one() == 1


def test_stale_without_either_output_or_older_than_a_source(small):
    outputs = [build.LIB, build.MODULE]
    assert build.stale()
    for path in outputs:
        open(path, "w").close()
    assert not build.stale()
    for path in outputs:
        os.utime(path, (1, 1))
        assert build.stale()
        os.remove(path)
        assert build.stale()
        open(path, "w").close()
        assert not build.stale()


def test_module_says_what_it_is_built_for(monkeypatch):
    module = _lib._native()
    assert module.__file__.endswith(sysconfig.get_config_var("EXT_SUFFIX"))
    assert module.built_for == torch.__version__
    monkeypatch.setattr(_lib, "_decode", None)
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    z, d = torch.zeros, M.Dims(2, 64, 16, 32, 32, 16, 0.1, torch.float32)
    with pytest.raises(ImportError, match="built for PyTorch"):
        M.mla_absorb_query(d, z(1, 2, 48), z(128, 64), z(1, 2, 80))
