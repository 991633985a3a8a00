"""Shapes that take other ways through the adapters, the score adjustment and the distillation: more ranks than a warp has turns,
many tiles to a warp, many adapters in one group of tokens, the largest ranks, hash tables of many rows, columns listed twice
among the most places."""
import math

import pytest
import torch

from collective_communication_primitives_b200 import simcomm as SC
from test_gpu_adapters import Adapted
from test_gpu_adjust_logits import Adjust
from test_gpu_distill import Distill, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("p,T,N,K,S,R,parallel,runs", [
    (16, 5, 64, 256, 4, 16, "row", 1), (16, 40, 128, 128, 2, 32, "row", 1), (12, 3, 96, 96, 3, 64, "row", 1),   # ranks in turns
    (1, 40, 4096, 64, 9, 32, "column", 1), (2, 100, 4096, 64, 5, 64, "column", 30), (2, 20, 2056, 64, 3, 16, "row", 1),
    (1, 130, 72, 64, 3, 256, "column", 50), (2, 100, 64, 512, 2, 192, "row", 100), (1, 2, 8, 16, 1, 256, "column", 2),
    (2, 700, 64, 128, 40, 16, "row", 1), (1, 1500, 40, 64, 24, 48, "column", 1), (4, 513, 64, 640, 2, 33, "row", 513),
    (8, 64, 64, 64, 64, 8, "column", 1), (8, 65, 64, 64, 1, 8, "row", 65), (64, 3, 64, 128, 2, 4, "row", 1)])
def test_adapters(p, T, N, K, S, R, parallel, runs):
    with SC.SimComm(p) as c:
        for base, out in (("fp32", "bf16"), ("bf16", "fp32"), (None, "bf16")):
            a = Adapted(p, T, N, K, S, R, parallel, base, out, seed=T + R, runs=runs)
            a.run(c)
            torch.cuda.synchronize()
            assert c.async_error() == SC.OK
            a.check(exact=True)


def test_adapters_that_differ_in_rank_beside_tokens_in_runs():
    with SC.SimComm(2) as c:
        a = Adapted(2, 600, 64, 256, 5, 64, "row", "bf16", "bf16", seed=3, runs=90, ranks=[64, 0, 7, 33, 16])
        for r in range(2):
            for e, k in enumerate(a.rk.tolist()):
                a.a[r][e, k:] = math.nan
                a.b[r][e, :, k:] = math.inf
        a.run(c)
        torch.cuda.synchronize()
        a.check(exact=True)


@pytest.mark.parametrize("p,R,V,L,bias,dtype", [(3, 320, 12007, 300, 0, "fp32"), (8, 600, 8192, 1000, 0, "bf16"), (1, 200, 20000, 40, 3, "bf16"),
                                                (4, 700, 2050, 100, 0, "fp32"), (5, 64, 131, 4000, 0, "bf16")])
def test_score_adjustment_of_many_rows(p, R, V, L, bias, dtype):
    with SC.SimComm(p) as c:
        a = Adjust(p, R, V, dtype, L, bias, True, seed=R)
        a.run(c)
        torch.cuda.synchronize()
        assert c.async_error() == SC.OK
        a.check()
        a.run(c, in_place=True)
        torch.cuda.synchronize()
        a.check(a.logits)


@pytest.mark.parametrize("R,V,p", [(3, 30011, 4), (700, 900, 3), (2, 300, 1)])
@pytest.mark.parametrize("tail", [False, True])
def test_columns_listed_twice_and_more_among_the_most_places(R, V, p, tail):
    n = 256
    x, idx, val = make(R, V, n, "bf16", 6, tail)
    idx[0, 1::2] = idx[0, 0::2]
    idx[1, ::3] = idx[1, 3]
    idx[-1, 100:] = idx[-1, 5]
    val = val - math.log(400) if tail else val  # so that the places' q stay below 1 in all
    gl = torch.rand(R, device="cuda") + 0.5
    with SC.SimComm(p) as c:
        a = Distill(x, idx, val, p, 1.0, tail)
        a.run(c)
        a.grad(c, gl)
        torch.cuda.synchronize()
        assert c.async_error() == SC.OK
        a.check()
        a.check_grad(gl)
        first = [v.clone() for v in a.loss + a.gx]
        a.run(c)
        a.grad(c, gl)
        torch.cuda.synchronize()
        assert all(torch.equal(u.contiguous(), v.contiguous()) for u, v in zip(first, a.loss + a.gx))
