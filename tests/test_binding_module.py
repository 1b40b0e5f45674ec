"""The extension module is refused where it was built for another torch, or does not load."""
import sys
import types

import pytest
import torch

import paged_kv_cache_87_gb300 as package
from paged_kv_cache_87_gb300 import binding, build


@pytest.fixture
def fresh(monkeypatch):
    build.build()
    monkeypatch.setattr(binding, "_calls", None)
    return monkeypatch


def test_the_module_of_this_torch_loads(fresh):
    assert binding._marshal().TORCH == torch.__version__


def test_a_module_built_for_another_torch_is_refused(fresh):
    name = package.__name__ + "._marshal"
    other = types.SimpleNamespace(TORCH="2.0.0+cu118", set_error=lambda e: None)
    fresh.setitem(sys.modules, name, other)
    fresh.setattr(package, "_marshal", other, raising=False)
    with pytest.raises(RuntimeError, match="built for torch 2.0.0"):
        binding._marshal()
    assert binding._calls is None


def test_a_module_that_does_not_load_names_the_build(fresh):
    fresh.setitem(sys.modules, package.__name__ + "._marshal", None)     # its import fails
    fresh.delattr(package, "_marshal", raising=False)
    with pytest.raises(RuntimeError, match="does not fit.*paged_kv_cache_87_gb300.build"):
        binding._marshal()


def test_another_torch_means_another_build(fresh):
    here = build._marshal_digest()
    fresh.setattr(torch, "__version__", "2.0.0")
    assert build._marshal_digest() != here
