"""GPU test of the router's gradient in rows with a NaN score: the forward pass makes every weight of such a row NaN, and
the gradient of the scores that the weights depend on is NaN with them, wherever the NaN stands and whatever was
picked. Other rows are as ever."""
import math

import pytest
import torch

from collective_communication_primitives_b200 import simcomm as SC

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E", [4, 8, 13, 64, 250, 256, 500, 1024, 1030, 4096])
@pytest.mark.parametrize("normalise", [True, False])
def test_nan_in_an_expert_that_was_not_picked(normalise, E, dtype):
    T, k = 9, 3
    g = torch.Generator("cuda").manual_seed(E)
    x = torch.randn(T, E, generator=g, device="cuda").to(dtype)
    gw = torch.randn(T, k, generator=g, device="cuda")
    idx, w = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    plain, gx = torch.empty_like(x), torch.full_like(x, 9.0)
    rows = {1: 0, 4: E - 1, 8: E // 2}  # row: column of its NaN
    with SC.SimComm(1) as c:
        c.moe_route([x], [idx], [w], normalise=normalise)
        c.moe_route_backward([x], [idx], [gw], [plain], normalise=normalise)
        for t, e in rows.items():
            x[t, e] = math.nan
        c.moe_route([x], [idx], [w], normalise=normalise)
        c.moe_route_backward([x], [idx], [gw], [gx], normalise=normalise)
        torch.cuda.synchronize()
        assert c.async_error() == SC.OK
    for t in range(T):
        if t not in rows:
            assert torch.equal(gx[t], plain[t])
            continue
        assert bool(w[t].isnan().all()) and rows[t] not in idx[t].tolist()[:min(k, E - 1)]
        picked = torch.zeros(E, dtype=torch.bool, device="cuda").scatter_(0, idx[t].long(), True)
        assert bool(gx[t][picked].isnan().all())
        if normalise:
            assert bool((gx[t][~picked] == 0).all())
        else:
            assert bool(gx[t].isnan().all())
