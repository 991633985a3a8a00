"""The helper that looks at a call's tensors takes exactly what the binding's own checks take, and gives the same addresses."""
import itertools
import struct

import pytest
import torch

from collective_communication_primitives_b200 import build as B
from collective_communication_primitives_b200 import simcomm as SC

F, BF, I32, U8, E4 = torch.float32, torch.bfloat16, torch.int32, torch.uint8, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def helper():
    B.build()
    SC._marshal = None
    assert SC._load_marshal(), "the helper is built with the library"
    return SC._marshal


def fake(p, device=-1):
    c = object.__new__(SC.SimComm)
    c.p, c.rank, c._device, c._h = p, None, device, None  # a CPU tensor's device number is -1
    c._pack, c._torch = struct.Struct(f"{p}P").pack, torch
    return c


def by_python(c, *args, **kw):
    kept, SC._marshal = SC._marshal, False
    try:
        return c._tensors("t", *args, **kw)
    except (TypeError, ValueError, AttributeError):
        return None
    finally:
        SC._marshal = kept


TENSORS = [torch.zeros(4, 6), torch.zeros(4, 6, dtype=BF), torch.zeros(6, 4).t(), torch.zeros(4, 9)[:, :6], torch.zeros(24), torch.zeros(1, 6),
           torch.zeros(1, 9)[:, :6], torch.zeros(4, 6, 1), torch.zeros(0, 6), torch.zeros(4, 6, dtype=E4), torch.zeros(2, 3, 4), torch.zeros(4, 1),
           torch.zeros(4, 5)[:, 2:3], torch.zeros(6)[::2], torch.zeros(()), torch.nn.Parameter(torch.zeros(4, 6)), torch.zeros(8, 6)[::2]]
SHAPES = [(4, 6), 24, (24,), (1, 6), (0, 6), 0, (4, 6, 1), (2, 3, 4), (4, 1), (3,), 1, (), (6, 4), torch.Size([4, 6])]


@pytest.mark.parametrize("dtype", [F, BF, I32, E4])
def test_the_same_is_taken_and_the_same_given(helper, dtype):
    c, taken = fake(2), 0
    for t, shape, row in itertools.product(TENSORS, SHAPES, (None, (6, 6), (9, 6), (5, 1), (12, 6))):
        if row is not None and (isinstance(shape, int) or len(shape) != 2):
            continue  # rows at a distance are asked for with their shape
        want = by_python(c, [t, t], dtype, shape, row=row)
        got = helper.addresses([t, t], dtype, shape, -1, 2, -1 if row is None else row[0])
        # the slow way also takes a flat tensor in place of a shaped one
        flat = not isinstance(shape, int) and t.dim() == 1 and len(shape) != 1
        assert got == want or (flat and got is None), (t.shape, t.stride(), shape, row)
        taken += got is not None
        if row is None:
            assert helper.address(t, dtype, shape, -1) == (None if got is None else t.data_ptr())
    assert taken > 0 or dtype is I32


def test_what_is_no_list_of_tensors_is_left_to_the_binding(helper):
    t = torch.zeros(4, 6)
    assert helper.addresses((t, t), F, (4, 6), -1, 2, -1) == struct.pack("2P", t.data_ptr(), t.data_ptr())
    for wrong in ([t], [t, None], [t, 4096], [t, t, t], None, t, "ab", [], [t, t.numpy()]):
        assert helper.addresses(wrong, F, (4, 6), -1, 2, -1) is None
    assert helper.addresses([t, t], "fp32", (4, 6), -1, 2, -1) is None
    assert helper.addresses([t, t], F, [4, 6], -1, 2, -1) is None
    assert helper.addresses([t, t], F, (4, 6.0), -1, 2, -1) is None
    assert helper.addresses([t, t], F, (4, 6), 0, 2, -1) is None  # another device
    assert helper.addresses([t] * 65, F, (4, 6), -1, 65, -1) is None
    assert helper.addresses([t, t], F, (4, 6)) is None
    assert helper.address(None, F, (4, 6), -1) is None and helper.address(7, F, (4, 6), -1) is None
    assert helper.addresses([torch.zeros(4, 6, device="meta")] * 2, F, (4, 6), -1, 2, -1) is None
    assert helper.addresses([torch.eye(4).to_sparse()] * 2, F, (4, 4), -1, 2, -1) is None


def test_the_binding_works_without_it(helper):
    c, t = fake(3), torch.zeros(5)
    want = struct.pack("3P", *[t.data_ptr()] * 3)
    assert c._tensors("t", [t] * 3, F, 5) == want == by_python(c, [t] * 3, F, 5)
