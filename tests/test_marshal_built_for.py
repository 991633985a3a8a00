"""The binding loads the helper that was built for this Python and torch and no other, and another one does not keep it from being
built: a helper reads tensors at places that differ from one torch to the next."""
import struct
import sysconfig

import pytest
import torch

from collective_communication_primitives_b200 import build as B
from collective_communication_primitives_b200 import simcomm as SC


@pytest.fixture
def loaded():
    B.build()
    kept = SC._marshal
    yield
    SC._marshal = kept


def change_torch(monkeypatch):
    monkeypatch.setattr(torch, "__version__", "0.1.0")


def change_flag(monkeypatch):
    now = torch.compiled_with_cxx11_abi()
    monkeypatch.setattr(torch, "compiled_with_cxx11_abi", lambda: not now)


def change_python(monkeypatch):
    real = sysconfig.get_config_var
    monkeypatch.setattr(sysconfig, "get_config_var", lambda name: "cpython-30-none" if name == "SOABI" else real(name))


def test_the_helper_of_this_torch_is_loaded(loaded):
    assert SC._load_marshal()
    t = torch.zeros(3)
    assert SC._marshal.address(t, torch.float32, (3,), -1) == t.data_ptr()
    assert not B._stale()


@pytest.mark.parametrize("change", [change_torch, change_flag, change_python])
def test_another_one_is_not(loaded, monkeypatch, change):
    change(monkeypatch)
    assert SC._load_marshal() is False
    assert B._stale()
    c = object.__new__(SC.SimComm)  # the binding looks at tensors itself
    c.p, c.rank, c._device, c._h = 2, None, -1, None
    c._pack = struct.Struct("2P").pack
    t = torch.zeros(3)
    assert c._tensors("t", [t, t], torch.float32, (3,)) == struct.pack("2P", t.data_ptr(), t.data_ptr())


def test_without_torch_there_is_nothing_to_build(monkeypatch):
    import sys
    monkeypatch.setitem(sys.modules, "torch", None)
    assert not B._marshal_stale()
