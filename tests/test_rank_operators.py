"""Host side of the operators of a model's step on rank views, without a GPU: a call that reads the peers' memory
stands between two meetings of all ranks, also when the library refuses it; the others meet nobody."""
import inspect
import struct

import pytest
import torch

from collective_communication_primitives_b200 import ranks
from collective_communication_primitives_b200 import simcomm as SC

BF = torch.bfloat16


def fake(p=2, rank=1, status=SC.OK):
    """A rank view whose library and ranks are a list of what happens."""
    c = object.__new__(ranks.RankComm)
    c.p, c.rank, c._device, c._h = p, rank, -1, None  # a CPU tensor's device number is -1
    c._pack, c._torch = struct.Struct(f"{p}P").pack, torch
    c.log = []

    class Lib:
        def __getattr__(self, name):
            def call(*args):
                c.log.append(name)
                return status
            return call
    c._L = Lib()
    c._check = lambda rc: (_ for _ in ()).throw(SC.SimCommError(rc, "refused")) if rc else None
    c.sync = lambda stream=None: c.log.append(("sync", stream))
    c._launch_stream = lambda stream: 0
    return c


def own(t, p=2, rank=1, other=None):
    return [t if r == rank else other for r in range(p)]


def calls(c):
    x, idx = torch.zeros(4, 64, dtype=BF), torch.zeros(4, 2, dtype=torch.int32)
    w, s, f = torch.zeros(8, 32, dtype=torch.uint8), torch.zeros(8, 2, dtype=BF), torch.zeros(4)
    lin = (own(x, other=64), own(w, other=64), own(s, other=64), own(torch.zeros(4, 8)))
    up, down = torch.zeros(2, 32, 64, dtype=BF), torch.zeros(2, 64, 16, dtype=BF)
    scores = own(torch.zeros(4, 10), other=64)
    return {
        "coll_linear_w4": lambda **k: c.linear_w4(*lin, parallel="row", **k),
        "coll_moe_layer": lambda **k: c.moe_layer(own(x), own(idx), own(torch.zeros(4, 2)), 4, own(up, other=64),
                                                  own(down, other=64), own(x), **k),
        "coll_logprobs": lambda **k: c.logprobs(scores, idx[:, 0].contiguous(), 20, own(f), **k),
        "coll_logprobs_backward": lambda **k: c.logprobs_backward(scores, idx[:, 0].contiguous(), 20, own(f), f,
                                                                  own(torch.zeros(4, 10)), **k)}


NAMES = ["coll_linear_w4", "coll_moe_layer", "coll_logprobs", "coll_logprobs_backward"]


@pytest.mark.parametrize("name", NAMES)
def test_calls_that_read_peers_meet_the_ranks_before_and_after(name):
    c = fake()
    calls(c)[name]()
    assert c.log == [("sync", None), name, ("sync", None)]
    c.log.clear()
    calls(c)[name](stream=5)
    assert c.log == [("sync", 5), name, ("sync", 5)]


@pytest.mark.parametrize("name", NAMES)
def test_a_refused_call_still_meets_both(name):
    c = fake(status=SC.INVALID_ARG)
    with pytest.raises(SC.SimCommError):
        calls(c)[name]()
    assert c.log == [("sync", None), name, ("sync", None)]


def test_arguments_that_the_binding_refuses_still_meet_both():
    c = fake()
    with pytest.raises(ValueError):
        c.linear_w4(own(torch.zeros(4, 64, dtype=BF)), own(torch.zeros(8, 32, dtype=torch.uint8)),
                    own(torch.zeros(8, 3, dtype=BF)), own(torch.zeros(4, 8)), parallel="row")
    assert c.log == [("sync", None)] * 2


@pytest.mark.parametrize("name", ["linear_w4", "moe_layer", "logprobs", "logprobs_backward"])
def test_arguments_are_those_of_the_whole_communicator(name):
    assert inspect.signature(getattr(ranks.RankComm, name)) == inspect.signature(getattr(SC.SimComm, name))


def test_calls_on_own_memory_meet_nobody():
    c = fake()
    x, w, s = torch.zeros(4, 64, dtype=BF), torch.zeros(8, 32, dtype=torch.uint8), torch.zeros(8, 2, dtype=BF)
    c.linear_w4(own(x), own(w), own(s), own(torch.zeros(4, 8)), parallel="column")
    idx, f = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    c.moe_route(own(torch.zeros(4, 8)), own(idx), own(f))
    c.moe_route_backward(own(torch.zeros(4, 8)), own(idx), own(f), own(torch.zeros(4, 8)))
    assert c.log == ["coll_linear_w4", "coll_moe_route", "coll_moe_route_backward"]
