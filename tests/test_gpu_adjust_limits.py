"""Limits of the score adjustment's arguments that no tensor of a test can have: refused before any array is looked at."""
import ctypes

import pytest
import torch

from collective_communication_primitives_b200 import simcomm as SC

pytestmark = pytest.mark.gpu


def test_histories_that_a_count_cannot_hold():
    x = torch.zeros(1, 64, device="cuda")
    y = torch.zeros(1, 64, device="cuda")
    n = torch.zeros(1, dtype=torch.int32, device="cuda")
    u = SC.LogitRules()
    u.history, u.history_len = n.data_ptr(), n.data_ptr()  # of length 0
    with SC.SimComm(1) as c:
        def call():
            one = lambda t: (ctypes.c_void_p * 1)(t.data_ptr())  # noqa: E731
            return c._L.coll_adjust_logits(c._h, ctypes.cast(one(x), ctypes.c_char_p), 64, 1, 64, 1, ctypes.byref(u),
                                           ctypes.cast(one(y), ctypes.c_char_p), 64, None)
        for length, status in ((1 << 30, SC.INVALID_ARG), ((1 << 31) + 5, SC.INVALID_ARG), (1, SC.OK)):
            u.ld_history = length
            assert call() == status
        torch.cuda.synchronize()
        assert c.async_error() == 0
