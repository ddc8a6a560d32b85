"""The library is built and loaded without the marshalling module where that
cannot be had, and a module of another Python is not picked up (no GPU)."""
import os
import sys
import sysconfig

import pytest
import torch

import gemm_epilogue_fusion_gb300 as g
from gemm_epilogue_fusion_gb300 import _build


@pytest.fixture()
def no_module(tmp_path, monkeypatch):
    """A place for the module with none in it, the library as it is."""
    g.load_library()
    monkeypatch.setattr(_build, "MARSHAL", str(tmp_path / os.path.basename(_build.MARSHAL)))
    return tmp_path


@pytest.mark.parametrize("cc", ["false", "/no/such/compiler"])
def test_the_library_is_built_without_a_compiler_for_the_module(no_module, monkeypatch, cc):
    monkeypatch.setenv("CC", cc)
    open(_build.MARSHAL, "w").close()
    os.utime(_build.MARSHAL, (0, 0))  # of older sources
    with pytest.warns(RuntimeWarning, match="coda_marshal.c could not be compiled"):
        assert _build.build() == _build.LIB
    assert os.listdir(no_module) == []


def test_the_library_is_built_without_the_headers_of_python(no_module, monkeypatch):
    monkeypatch.setattr(sysconfig, "get_paths", lambda *a, **k: {"include": "/no/such/folder"})
    with pytest.warns(RuntimeWarning, match="Python.h"):
        assert _build.build() == _build.LIB


def test_a_library_that_is_up_to_date_needs_no_nvcc(no_module, monkeypatch):
    monkeypatch.setenv("NVCC", "/no/such/nvcc")
    with pytest.warns(RuntimeWarning, match="nvcc"):
        assert _build.build() == _build.LIB


def test_the_module_is_built_beside_the_library(no_module):
    assert _build.build() == _build.LIB and _build.marshal_up_to_date()
    assert os.path.basename(_build.MARSHAL).endswith(sysconfig.get_config_var("EXT_SUFFIX"))
    assert os.listdir(no_module) == [os.path.basename(_build.MARSHAL)]


def test_cuda_headers_are_found_behind_a_link_to_nvcc(no_module, monkeypatch):
    (no_module / "bin").mkdir()
    link = no_module / "bin" / "nvcc"
    link.symlink_to(os.path.realpath(_build.nvcc()))
    monkeypatch.setenv("NVCC", str(link))
    assert _build.build() == _build.LIB and _build.marshal_up_to_date()


def test_calls_are_checked_without_the_module(monkeypatch):
    lib = g.load_library()
    monkeypatch.setattr(g, "_fast", None)
    monkeypatch.delattr(g, "_coda_marshal", raising=False)
    monkeypatch.setitem(sys.modules, g.__name__ + "._coda_marshal", None)  # an import of it fails
    with pytest.warns(RuntimeWarning, match="cannot be loaded"):
        g._load_marshal(lib)
    assert g._fast is None
    with pytest.raises(ValueError, match="CUDA tensor"):
        g.coda_logprobs(torch.zeros(2, 16), torch.zeros(2, dtype=torch.int32))
