"""Argument checks of the router, the products with sharded weights and the log probabilities that need no
GPU: NULL communicators, and the binding's checks of the tensors it is given."""
import struct
import types

import pytest
import torch

from collective_communication_primitives_b200 import build as B
from collective_communication_primitives_b200 import simcomm as SC


@pytest.fixture(scope="module")
def lib():
    B.build()
    return SC.load_library()


def test_null_communicators_are_refused(lib):
    assert lib.coll_moe_route(None, None, 4, 2, 8, 1, 1, None, None, None) == SC.INVALID_ARG
    assert lib.coll_moe_route_backward(None, None, None, None, 4, 2, 8, 1, 1, None, None) == SC.INVALID_ARG
    assert lib.coll_linear_w4(None, None, None, None, 4, 8, 64, 32, 1, 1, None, None) == SC.INVALID_ARG
    assert lib.coll_moe_layer(None, None, None, None, None, 4, 2, 8, 8, 8, 0, 0, None, None, None, None, 2, None,
                              None) == SC.INVALID_ARG
    assert lib.coll_logprobs(None, None, 8, None, 4, 8, 1, None, None, None, 0, None, None, None) == SC.INVALID_ARG
    assert lib.coll_logprobs_backward(None, None, 8, None, 4, 8, 1, None, None, None, None, None, 8,
                                      None) == SC.INVALID_ARG


def fake(p=2, rank=None):
    """A handle's tensor checks without a communicator (they look at p, rank and the device alone)."""
    c = object.__new__(SC.SimComm)
    c.p, c.rank, c._device, c._h = p, rank, -1, None  # a CPU tensor's device number is -1
    c._pack, c._torch = struct.Struct(f"{p}P").pack, torch
    return c


def pointers(b):
    return list(struct.unpack(f"{len(b) // 8}P", b))


def test_tensors_are_checked_before_their_addresses_are_taken():
    c, f = fake(), torch.float32
    good = [torch.zeros(4, 3), torch.zeros(4, 3)]
    got = c._tensors("t", good, f, 12)
    assert pointers(got) == [t.data_ptr() for t in good]
    assert c._tensors("t", None, f, 12) is None
    assert c._tensors("t", good[0], f, 12, one=True) == good[0].data_ptr()
    with pytest.raises(TypeError):
        c._tensors("t", [good[0], good[1].int()], f, 12)
    with pytest.raises(ValueError):
        c._tensors("t", [good[0], torch.zeros(4, 4)], f, 12)
    with pytest.raises(ValueError):
        c._tensors("t", [good[0], torch.zeros(3, 4).t()], f, 12)
    with pytest.raises(ValueError):
        c._tensors("t", good[:1], f, 12)
    with pytest.raises(TypeError):
        c._tensors("t", [good[0], None], f, 12)
    c._device = 0
    with pytest.raises(ValueError):
        c._tensors("t", good, f, 12)


def test_rows_at_a_distance():
    c, f = fake(), torch.float32
    wide = [torch.zeros(4, 10)[:, :3] for _ in range(2)]
    assert pointers(c._tensors("t", wide, f, 12, row=(10, 3))) == [t.data_ptr() for t in wide]
    with pytest.raises(ValueError):
        c._tensors("t", [wide[0], torch.zeros(4, 9)[:, :3]], f, 12, row=(10, 3))
    with pytest.raises(ValueError):
        c._tensors("t", [wide[0], torch.zeros(3, 4).t()], f, 12, row=(10, 3))
    with pytest.raises(ValueError):
        c._tensors("t", wide, f, 12)  # not contiguous


def test_a_view_needs_its_own_entries_only():
    c = fake(3, rank=1)
    t = torch.zeros(5)
    assert pointers(c._tensors("t", [None, t, 4096], torch.float32, 5)) == [0, t.data_ptr(), 4096]


def test_shapes_that_do_not_fit_are_refused_in_the_binding():
    c, bf = fake(), torch.bfloat16
    c._L = types.SimpleNamespace()
    x = [torch.zeros(4, 64, dtype=bf)] * 2
    w = [torch.zeros(8, 32, dtype=torch.uint8)] * 2
    with pytest.raises(ValueError, match="parallel"):
        c.linear_w4(x, w, [torch.zeros(8, 2, dtype=bf)] * 2, x, parallel="both")
    with pytest.raises(ValueError, match="groups"):
        c.linear_w4(x, w, [torch.zeros(8, 3, dtype=bf)] * 2, x)
    idx = [torch.zeros(4, 2, dtype=torch.int32)] * 2
    up = [torch.zeros(4, 64, 64, dtype=bf)] * 2
    with pytest.raises(ValueError, match="w_up"):
        c.moe_layer(x, idx, idx, 4, up, up, x)  # 4 experts on each of 2 ranks are 8
    with pytest.raises(ValueError, match="w_up"):
        c.moe_layer(x, idx, idx, 8, up, up, x, down_scale=up)
    with pytest.raises(ValueError, match="columns per rank"):
        c.logprobs(x, idx[0], 200, x)
    with pytest.raises(ValueError, match="grad_entropy"):
        c.logprobs_backward(x, idx[0], 128, x, x[0], x, grad_entropy=x[0])
