"""CPU: the native marshalling module belongs to one torch and one interpreter; against another
it is built again, and never loaded."""

import sys

import pytest
import torch

from block_sparse_attention_tcgen05_b200 import _lib, build


def test_the_module_says_what_it_was_built_against():
    build.build()
    assert build.native_up_to_date()
    assert torch.__version__ in build.native_id() and sys.implementation.cache_tag in build.native_id()


def test_a_module_of_another_torch_is_stale(monkeypatch):
    build.build()
    monkeypatch.setattr(torch, "__version__", "1.0.0+other")
    assert not build.native_up_to_date()
    monkeypatch.setattr(_lib, "_native", None)
    with pytest.raises(RuntimeError, match="another torch or Python"):
        _lib.native()
    built = []
    monkeypatch.setattr(build, "_compile", lambda cmd, out, verbose: built.append(out))
    build.build_native()
    assert built == [build.NATIVE]


def test_a_missing_module_is_named(monkeypatch, tmp_path):
    monkeypatch.setattr(build, "NATIVE", str(tmp_path / "_native.so"))
    assert not build.native_up_to_date()
