"""The norm and its gradient with many rows, which go through a ring in shared memory: against float64, and what happens
when the warp that fills the ring falls silent (host-side fault injection, no GPU fault)."""
import time

import pytest
import torch

from collective_communication_primitives_b200 import simcomm as SC
from test_gpu_rmsnorm import Back, Norm

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("p,T,H,group", [(8, 700, 4096, 128), (1, 1301, 1024, 0), (3, 1400, 264, 0), (2, 1250, 64, 32),
                                         (64, 1200, 128, 128), (2, 601, 8192, 1024), (4, 333, 5120, 0), (1, 299, 16384, 16384),
                                         (2, 1190, 8, 0), (5, 620, 2048, 2048)])
def test_many_rows(p, T, H, group, dtype):
    with SC.SimComm(p) as c:
        for residual in (True, False):
            a = Norm(p, T, H, dtype, residual, group, seed=T)
            a.run(c)
            b = Back(p, T, H, dtype, residual, seed=H)
            b.run(c)
            torch.cuda.synchronize()
            assert c.async_error() == SC.OK
            a.check()
            b.check()
        first = [v.clone() for v in b.gx + b.gw]
        b.run(c)
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(first, b.gx + b.gw))


def test_residual_in_place_of_many_rows():
    with SC.SimComm(2) as c:
        a = Norm(2, 900, 2048, "bf16", seed=2)
        res = a.res.clone()
        a.total[1].copy_(a.res)
        c.rmsnorm(a.x, a.w, 1e-5, out=a.y, residual=a.total[1], total=a.total)
        torch.cuda.synchronize()
        a.check(res)


@pytest.mark.parametrize("H", [512, 4096])
def test_huge_rows_among_others(H):
    """Rows whose squares pass fp32 between rows that are sums as usual."""
    with SC.SimComm(1) as c:
        a = Norm(1, 1200, H, "fp32", False, seed=4)
        scale = torch.where(torch.arange(1200, device="cuda") % 3 == 1, 2.0 ** 70, 1.0)[:, None]
        b = Norm(1, 1200, H, "fp32", False, seed=4)
        a.run(c)
        b.x[0] *= scale
        b.run(c)
        torch.cuda.synchronize()
        # the same numbers but for eps, which the large rows lose: 1e-5 / (2 mean h^2) of them, and a rounding
        off = 1e-5 / a.x[0].square().mean(1, keepdim=True) + 2.0 ** -20
        assert bool(((a.y[0] - b.y[0]).abs() <= off * a.y[0].abs()).all())


@pytest.mark.parametrize("cta", [0, 1])
@pytest.mark.parametrize("back", [False, True])
def test_a_silent_copying_warp_runs_the_waits_out(cta, back):
    a = (Back if back else Norm)(2, 1000, 4096, "bf16", seed=1)
    with SC.SimComm(2) as c:
        c.set_option("timeout_ns", 50_000_000)
        c.set_option("fault_skip_rank", cta)
        t0 = time.time()
        a.run(c)
        torch.cuda.synchronize()
        assert time.time() - t0 < 5.0
        assert c.async_error() == SC.TIMEOUT
        with pytest.raises(SC.SimCommError) as e:  # refused until reset
            a.run(c)
        assert e.value.status == SC.TIMEOUT
        c.set_option("fault_skip_rank", -1)
        c.reset()
        a.run(c)
        torch.cuda.synchronize()
        assert c.async_error() == SC.OK
        a.check()
