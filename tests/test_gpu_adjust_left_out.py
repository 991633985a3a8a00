"""Arrays of a rule that is left out (a NULL history_len, bias_start or mask) are not looked at: whatever they hold, and
whatever else lies there, the scores come out as they went in."""
import ctypes

import pytest
import torch

from collective_communication_primitives_b200 import simcomm as SC

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("R,V", [(1, 64), (5, 3001)])
def test_scores_are_copied(R, V, dtype):
    x = torch.randn(R, V, device="cuda").to(dtype)
    y = torch.zeros_like(x)
    nan = torch.full((max(R, 8),), float("nan"), device="cuda")
    n = torch.full((R + 1,), 3, dtype=torch.int32, device="cuda")
    u = SC.LogitRules()
    u.ld_history, u.bias_count, u.ld_mask, u.mask_rows = 5, 1 << 40, 0, 0
    for name in ("history", "prompt_len", "bias_token", "mask_row"):
        setattr(u, name, n.data_ptr())
    for name in ("frequency", "presence", "bias_value"):
        setattr(u, name, nan.data_ptr())
    u.repetition = y.data_ptr()  # what is written
    one = lambda t: ctypes.cast((ctypes.c_void_p * 1)(t.data_ptr()), ctypes.c_char_p)  # noqa: E731
    with SC.SimComm(1) as c:
        status = c._L.coll_adjust_logits(c._h, one(x), V, R, V, SC.DTYPES[SC._dtype_of(x)], ctypes.byref(u), one(y), V, None)
        torch.cuda.synchronize()
        assert status == SC.OK and c.async_error() == SC.OK
    assert torch.equal(x, y)
