"""The marshalling module belongs to the PyTorch and the Python that it was compiled with: with
others it is compiled again, and not used."""

import os
import sys
from types import SimpleNamespace

import pytest
import torch


@pytest.fixture(scope="module")
def built():
    from w8a16_linear_gb300 import build as B
    B.build()
    return B


def here():
    return f"{torch.__version__} {sys.implementation.cache_tag}"


def test_compiled_again_for_another_pytorch(built):
    if not os.path.exists(built.MARSHAL):
        pytest.skip("csrc/marshal.cpp does not compile here")
    assert not built._marshal_stale(here())
    assert built._marshal_stale("0.0 " + sys.implementation.cache_tag)
    assert built._marshal_stale(f"{torch.__version__} cpython-0")


@pytest.mark.parametrize("built_for,used", [(here(), True), ("0.0 cpython-312", False), (None, False)])
def test_used_with_its_own_pytorch_alone(built, monkeypatch, built_for, used):
    import w8a16_linear_gb300 as package
    from w8a16_linear_gb300 import binding
    if not os.path.exists(built.MARSHAL):
        pytest.skip("csrc/marshal.cpp does not compile here")
    bound = []
    module = SimpleNamespace(bind=lambda *a: bound.append(a))
    if built_for:
        module.built_for = built_for
    monkeypatch.setitem(sys.modules, "w8a16_linear_gb300._marshal", module)
    monkeypatch.setattr(package, "_marshal", module, raising=False)
    monkeypatch.setattr(binding, "_lib", None)
    monkeypatch.setattr(binding, "_marshal", None)
    binding.lib()
    assert (binding._marshal is module) == used and len(bound) == used
