"""Without the helper the binding looks at the usual call's tensors in one sweep of its own: right ones are asked for no more than the
sweep asks, and what is wrong is refused as ever."""
import struct

import pytest
import torch

from collective_communication_primitives_b200 import simcomm as SC


class Watched:
    """A tensor that notes what it is asked for."""

    def __init__(self, t, log):
        self.t, self.log = t, log

    def __getattr__(self, name):
        self.log.append(name)
        return getattr(self.t, name)


@pytest.fixture
def comm(monkeypatch):
    monkeypatch.setattr(SC, "_marshal", False)
    c = object.__new__(SC.SimComm)
    c.p, c.rank, c._device, c._h = 2, None, -1, None  # a CPU tensor's device number is -1
    c._pack = struct.Struct("2P").pack
    return c


@pytest.mark.parametrize("shape,row", [((4, 6), None), ((4, 6), (6, 6)), (24, None), ((24,), None), ((0, 6), None), ((1, 6), (6, 6))])
def test_right_tensors_take_one_sweep(comm, shape, row):
    log = []
    ts = [Watched(torch.zeros(shape), log) for _ in range(2)]
    got = comm._tensors("t", ts, torch.float32, shape, row=row)
    assert got == struct.pack("2P", *[v.t.data_ptr() for v in ts])
    assert len(log) == 10 and set(log) <= {"dtype", "get_device", "numel", "shape", "is_contiguous", "data_ptr"}


def test_the_rest_takes_the_slow_way(comm):
    wide = [torch.zeros(4, 9)[:, :6] for _ in range(2)]
    assert comm._tensors("t", wide, torch.float32, (4, 6), row=(9, 6)) == struct.pack("2P", *[v.data_ptr() for v in wide])
    good = [torch.zeros(4, 6) for _ in range(2)]
    for ts, row, error in ((good[:1], None, ValueError), (good + good[:1], None, ValueError), ([good[0], None], None, TypeError),
                           ([good[0], torch.zeros(4, 6, dtype=torch.int32)], None, TypeError), (wide, None, ValueError),
                           ([good[0], torch.zeros(6, 4)], None, ValueError), (wide, (6, 6), ValueError), (good, (9, 6), ValueError)):
        with pytest.raises(error):
            comm._tensors("t", ts, torch.float32, (4, 6), row=row)
    comm._device = 0
    with pytest.raises(ValueError, match="device"):
        comm._tensors("t", good, torch.float32, (4, 6))
