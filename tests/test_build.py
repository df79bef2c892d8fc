"""The in-tree build without a GPU: the library needs neither torch nor the operators'
module."""
import os
import sys

import pytest

import exact_top_token_gb300 as hk
from exact_top_token_gb300 import _build


@pytest.fixture
def small(tmp_path, monkeypatch):
    """A build of its own of one small source."""
    source = tmp_path / "one.cu"
    source.write_text("__global__ void k_one(int* p) { *p = 1; }\n"
                      "extern \"C\" void one(int* p) { k_one<<<1, 1>>>(p); }\n")
    monkeypatch.setattr(_build, "BUILD", str(tmp_path / "out"))
    monkeypatch.setattr(_build, "LIB", str(tmp_path / "out" / "libone.so"))
    monkeypatch.setattr(_build, "sources", lambda: [str(source)])
    return tmp_path / "out"


def test_the_library_builds_without_torch(small, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)
    assert hk.build() == _build.LIB and os.path.exists(_build.LIB)
    assert hk.build() == _build.LIB                      # up to date
    assert not [f for f in os.listdir(small) if f.startswith("_operators")]


def test_the_library_is_there_when_the_module_does_not_build(small, monkeypatch):
    monkeypatch.setenv("CXX", "false")
    with pytest.raises(RuntimeError, match="binding.cpp"):
        hk.build()
    assert os.path.exists(_build.LIB)
    with pytest.raises(RuntimeError, match="binding.cpp"):  # and says so again
        hk.build()


def test_the_module_is_named_for_what_it_was_built_against():
    import torch

    name = os.path.basename(_build.binding())
    assert torch.__version__ in name and sys.implementation.cache_tag in name
