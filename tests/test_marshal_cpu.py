"""The compiled marshalling is built for one PyTorch and interpreter, and is left out under any other."""
import os

import pytest
import torch

from partial_activation_sync_caat_b200 import build as B
from partial_activation_sync_caat_b200 import caat as C


@pytest.fixture(scope="module")
def L():
    B.build()
    return C.lib()


def test_another_pytorch_leaves_it_out(L, monkeypatch):
    monkeypatch.setattr(C, "_marshal", None)
    C._bind_marshal(L)
    assert C._marshal is not None
    monkeypatch.setattr(torch, "__version__", torch.__version__ + ".other")
    C._bind_marshal(L)
    assert C._marshal is None


def test_the_file_carries_what_it_was_built_for(monkeypatch):
    assert B.torch_version() == torch.__version__
    here = B.marshal_path()
    assert os.path.dirname(here) == B.PKG and here == B.marshal_path(torch.__version__)
    assert len({here, B.marshal_path("2.0.0"), B.marshal_path("2.0.0+cpu")}) == 3
    monkeypatch.setattr(B.sysconfig, "get_config_var", lambda name: "cpython-399-x86_64-linux-gnu")
    assert B.marshal_path() != here


def test_another_pytorch_is_built_for(L, monkeypatch):
    """What is there for one PyTorch does not count for another."""
    assert B.up_to_date()
    monkeypatch.setattr(B, "torch_version", lambda: "0.0.0")
    assert not B.marshal_up_to_date()
