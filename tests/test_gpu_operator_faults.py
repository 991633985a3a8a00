"""Failure detection of the 4-bit linear and the expert layer, tested without a GPU fault: host-side fault injection
(option fault_skip_rank: one warp of a CTA falls silent) leaves the CTA's other warps without tokens, free buffers or
finished sums. Each of their waits runs out, the kernel returns, the call reports COLL_ERR_TIMEOUT, and sim_comm_reset
makes the communicator usable again."""
import time

import pytest
import torch

from collective_communication_primitives_b200 import simcomm as SC
from test_gpu_linear_w4 import make
from test_gpu_moe_layer import Layer

pytestmark = pytest.mark.gpu


def _fails_and_recovers(c, run, cta):
    c.set_option("timeout_ns", 50_000_000)
    c.set_option("fault_skip_rank", cta)
    t0 = time.time()
    run()
    torch.cuda.synchronize()
    assert time.time() - t0 < 5.0
    assert c.async_error() == SC.TIMEOUT
    with pytest.raises(SC.SimCommError) as e:  # refused until reset
        run()
    assert e.value.status == SC.TIMEOUT
    c.set_option("fault_skip_rank", -1)
    c.reset()
    run()
    torch.cuda.synchronize()
    assert c.async_error() == SC.OK


# warps that share a row tile (few rows) and warps that do not, one unit to a CTA and several
@pytest.mark.parametrize("T,N,K,group,parallel", [(1, 512, 4096, 128, "row"), (16, 2048, 2048, 64, "row"),
                                                  (33, 16384, 1024, 32, "column"), (5, 65536, 512, 128, "column")])
@pytest.mark.parametrize("cta", [0, 1])
def test_linear(T, N, K, group, parallel, cta):
    xs, w, s, wd, out = make(2, T, N, K, group, parallel, "fp32")
    with SC.SimComm(2) as c:
        c.linear_w4(xs, w, s, out, parallel=parallel)
        torch.cuda.synchronize()
        want = [o.clone() for o in out]
        _fails_and_recovers(c, lambda: c.linear_w4(xs, w, s, out, parallel=parallel), cta)
        assert all(torch.equal(a, b) for a, b in zip(want, out))


@pytest.mark.parametrize("group,tensor", [(0, 0), (0, 1), (32, -1), (64, -1), (128, -1)])
@pytest.mark.parametrize("T,E,H,F", [(1, 8, 1024, 512), (40, 8, 640, 1024), (96, 32, 512, 1536)])
def test_expert_layer(T, E, H, F, group, tensor):
    a = Layer(2, T, E, 4, H, F, group, seed=T)
    with SC.SimComm(2) as c:
        c.set_option("moe_layer_tensor", tensor)
        _fails_and_recovers(c, lambda: a.run(c), 1)
    a.check()
