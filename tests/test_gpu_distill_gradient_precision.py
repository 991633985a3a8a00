"""The distillation's gradient where its exponentials are exact: in a row of equal scores every P is 1 / V, the sum of V ones is
exact in fp32 (V below 2^24) and 2^0 is 1, so that only the row's constants and the last products round.

Tolerance: without the class of the rest a score off the list has g / (T V), one listed with q = 0 the same: the constant is
rounded once (2^-24), 1 / T once, its product with g and the result once each, two more for what a listed column's product takes:
6 2^-24, and half a step of the result's type. With the rest the gradient off the list is g P (A - Q / P_rest) = g (A P_rest - Q) / (V - n), A = 1, whose
A P_rest - Q is formed in 64 bits from the fp32 values' exponentials. The logarithm of a sum of V held in fp32 would be off by up to
2^-21 for V from 2^11 to 2^16 and by 2^-20 up to 2^32, times ln 2: 5 to 11 of those 2^-24."""
import math

import pytest
import torch

from collective_communication_primitives_b200 import simcomm as SC
from test_gpu_logprobs import shards

pytestmark = pytest.mark.gpu


def gradient(p, x, V, idx, value, g, **kw):
    R = x.shape[0]
    logits = shards(x, p, 0, 0)
    stats = [torch.empty(R, 8, device="cuda") for _ in range(p)]
    loss = [torch.empty(R, device="cuda") for _ in range(p)]
    out = [torch.empty_like(v) for v in logits]
    with SC.SimComm(p) as c:
        c.distill(logits, V, idx, value, loss, stats=stats, **kw)
        c.distill_backward(logits, V, idx, value, stats, g, out, **kw)
        torch.cuda.synchronize()
        assert c.async_error() == 0
    return torch.cat(out, 1)[:, :V].double()


@pytest.mark.parametrize("V", [3001, 5003, 20011, 50257, 100003, 131071])
@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("p,R,dtype", [(1, 3, torch.float32), (4, 3, torch.float32), (2, 300, torch.float32), (2, 3, torch.bfloat16)])
def test_rows_of_equal_scores(p, R, dtype, tail, V):
    gen = torch.Generator("cuda").manual_seed(V)
    x = torch.full((R, V), 1.5, device="cuda").to(dtype)
    g = torch.rand(R, generator=gen, device="cuda") + 0.5
    idx = torch.tensor([5, V // 2, V - 1], dtype=torch.int32, device="cuda").repeat(R, 1)
    half = 0.5 * torch.finfo(dtype).eps if dtype is torch.bfloat16 else 0.0
    G = g.double()[:, None]
    off = torch.ones(V, dtype=torch.bool, device="cuda")
    off[idx[0].long()] = False
    if tail:
        value = torch.tensor([math.log(0.25), math.log(0.125), -math.inf], device="cuda").repeat(R, 1)
        got = gradient(p, x, V, idx, value, g, tail=True)
        q = value[0].double().exp()
        Q = 1 - q.sum()
        rest = G * ((V - 3) / V - Q) / (V - 3)
    else:
        value = torch.tensor([0.3, -0.7, -math.inf], device="cuda").repeat(R, 1)
        got = gradient(p, x, V, idx, value, g, temperature=2.0)
        rest = G / 2 / V
    bound = 6 * 2 ** -24 + half
    far = ((got[:, off] - rest).abs() / rest.abs()).max().item()
    assert far <= bound, far * 2 ** 24
    listed = G / V if tail else G / 2 / V  # q = 0
    far = ((got[:, V - 1:] - listed).abs() / listed).max().item()
    assert far <= bound, far * 2 ** 24
