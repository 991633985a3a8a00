"""GPU tests of the MoE router and its gradient against float64.

Picks are whole numbers and must be equal (the lower id among equal scores). Weights and gradients are
fp32: an exponential's argument is rounded once (|x - max| 2^-24, times ln 2 log2 e) and the instruction is
good to 2^-22; sums of E terms add E 2^-24 relative to themselves, the division and the product one half
step each.
"""
import math

import pytest
import torch

from collective_communication_primitives_b200 import simcomm as SC

pytestmark = pytest.mark.gpu
DT = {"fp32": torch.float32, "bf16": torch.bfloat16}


def reference(x, k, normalise):
    """ids and weights in float64, by a stable sort."""
    x = x.double()
    idx = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :k]
    prob = torch.softmax(x, 1)
    w = prob.gather(1, idx)
    return idx, prob, (w / w.sum(1, keepdim=True) if normalise else w)


def rel_bound(x, E):
    """Relative error of a weight, from the derivation above."""
    xd = x.double()
    span = float((xd.amax(1, keepdim=True) - xd).amax()) if E > 1 else 0.0
    return 2 * (2.0 ** -22 + 2 * span * 2.0 ** -24) + (E + 4) * 2.0 ** -24


def route(x, k, normalise, p=1, rank=None):
    T, E = x[0].shape
    idx = [torch.full((T, k), -9, dtype=torch.int32, device="cuda") for _ in range(p)]
    w = [torch.full((T, k), -9.0, device="cuda") for _ in range(p)]
    with SC.SimComm(p) as c:
        c.moe_route(x, idx, w, normalise=normalise)
        torch.cuda.synchronize()
        assert c.async_error() == SC.OK
    return idx, w


CASES = [
    # p, T, E, k
    (1, 1, 1, 1), (1, 1, 8, 8), (2, 3, 10, 3), (3, 5, 12, 12), (4, 33, 16, 2), (8, 1, 64, 2), (2, 129, 64, 8),
    (1, 70, 100, 4), (5, 7, 130, 32), (2, 31, 256, 8), (1, 17, 384, 6), (2, 9, 512, 1), (1, 5, 1000, 8),
    (2, 3, 1024, 32), (1, 4, 1025, 8), (2, 3, 4096, 16),
]


@pytest.mark.parametrize("p,T,E,k", CASES)
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("normalise", [True, False])
def test_route_and_gradient(p, T, E, k, dtype, normalise):
    g = torch.Generator("cuda").manual_seed(p * 1000 + T * 10 + E)
    x = [(2 * torch.randn(T, E, generator=g, device="cuda")).to(DT[dtype]) for _ in range(p)]
    gw = [torch.randn(T, k, generator=g, device="cuda") for _ in range(p)]
    idx, w = route(x, k, normalise, p)
    gx = [torch.full((T, E), 7.0, dtype=DT[dtype], device="cuda") for _ in range(p)]
    with SC.SimComm(p) as c:
        c.moe_route_backward(x, idx, gw, gx, normalise=normalise)
        torch.cuda.synchronize()
        assert c.async_error() == SC.OK
    for r in range(p):
        ri, prob, rw = reference(x[r], k, normalise)
        assert torch.equal(idx[r].long(), ri)
        eps = rel_bound(x[r], E)
        assert bool(((w[r].double() - rw).abs() <= eps * rw + 1e-37).all())
        G = torch.zeros_like(prob).scatter_add_(1, ri, gw[r].double())
        base = torch.zeros_like(prob).scatter_(1, ri, rw) if normalise else prob
        mean = (gw[r].double() * rw).sum(1, keepdim=True)
        want = base * (G - mean)
        # the factor in brackets is a difference: its error is relative to its parts
        slack = base * (G.abs() + (gw[r].double().abs() * rw).sum(1, keepdim=True)) * (2 * eps + (k + 4) * 2.0 ** -24)
        half = torch.finfo(DT[dtype]).eps / 2
        assert bool(((gx[r].double() - want).abs() <= half * want.abs() * 1.01 + slack + 1e-37).all())


@pytest.mark.parametrize("normalise", [True, False])
@pytest.mark.parametrize("E,k", [(16, 4), (300, 3), (2000, 4)])
def test_gradient_against_differences(normalise, E, k):
    """d/dx of sum g w, by central differences of the float64 formula at fixed picks."""
    g = torch.Generator("cuda").manual_seed(E)
    x = torch.randn(1, E, generator=g, device="cuda")
    gw = torch.randn(1, k, generator=g, device="cuda")
    idx, _ = route([x], k, normalise)
    gx = [torch.empty_like(x)]
    with SC.SimComm(1) as c:
        c.moe_route_backward([x], idx, [gw], gx, normalise=normalise)
    torch.cuda.synchronize()

    def loss(v):
        q = torch.softmax(v, 1).gather(1, idx[0].long())
        return float(((q / q.sum() if normalise else q) * gw.double()).sum())

    h = 1e-5  # the formula's third derivative is below |g| k: the truncation is below 1e-9, the rounding 1e-10
    for e in sorted({0, E - 1, *idx[0][0].tolist()}):
        lo, hi = x.double().clone(), x.double().clone()
        lo[0, e] -= h
        hi[0, e] += h
        assert abs((loss(hi) - loss(lo)) / (2 * h) - float(gx[0][0, e])) < 1e-6


def test_ties_take_the_lower_id():
    for E, k in ((8, 8), (64, 5), (300, 32), (1500, 9)):
        x = torch.zeros(2, E, device="cuda")
        x[1, ::2] = -0.0  # equal to +0
        idx, w = route([x], k, True)
        assert idx[0].tolist() == [list(range(k))] * 2
        assert torch.allclose(w[0], torch.full_like(w[0], 1 / k), rtol=1e-6)


@pytest.mark.parametrize("E", [16, 64, 700, 1200])
def test_masked_and_special_rows(E):
    inf, k = math.inf, 4
    x = torch.full((6, E), -inf, device="cuda")
    x[1, E - 1] = 2.0                      # one expert is left
    x[2] = torch.finfo(torch.float32).min  # masked throughout by the type's lowest value: equal scores
    x[3] = 0.5
    x[3, 3] = math.nan
    x[4] = 0.5
    x[4, 1] = inf
    x[5, 2:6] = torch.tensor([1.0, 2.0, 3.0, 4.0])
    for normalise in (True, False):
        idx, w = route([x], k, normalise)
        i, v = idx[0].tolist(), w[0]
        assert i[0] == [0, 1, 2, 3] and v[0].tolist() == [0.0] * k
        assert i[1] == [E - 1, 0, 1, 2] and v[1].tolist() == [1.0, 0.0, 0.0, 0.0]
        assert i[2] == [0, 1, 2, 3]
        assert torch.allclose(v[2], torch.full((k,), 1 / k if normalise else 1 / E, device="cuda"), rtol=1e-5)
        assert i[3] == [0, 1, 2, 4] and bool(v[3].isnan().all())
        assert i[4][0] == 1 and bool(v[4].isnan().all())
        assert i[5] == [5, 4, 3, 2] and abs(float(v[5].sum()) - 1) < 1e-6
    gx = [torch.full_like(x, 9.0)]
    with SC.SimComm(1) as c:
        c.moe_route_backward([x], idx, [torch.ones(6, k, device="cuda")], gx, normalise=False)
        torch.cuda.synchronize()
    assert gx[0][0].abs().max() == 0  # no distribution, no gradient
    assert bool(gx[0][1].abs().max() < 1e-6) and bool(gx[0][3].isnan().all())


@pytest.mark.parametrize("E", [24, 1500])
def test_an_id_twice_counts_twice_and_a_bad_id_is_reported(E):
    x = torch.randn(1, E, device="cuda")
    gw = torch.tensor([[1.0, 2.0, -1.0]], device="cuda")
    idx = torch.tensor([[3, 3, 5]], dtype=torch.int32, device="cuda")
    prob = torch.softmax(x.double(), 1)
    G = torch.zeros_like(prob)
    G[0, 3], G[0, 5] = 3.0, -1.0
    with SC.SimComm(1) as c:
        for normalise in (False, True):
            gx = [torch.empty_like(x)]
            c.moe_route_backward([x], [idx], [gw], gx, normalise=normalise)
            torch.cuda.synchronize()
            if normalise:
                t = prob[0, [3, 3, 5]]
                q = t / t.sum()
                mean = float((q * gw[0].double()).sum())
                want = torch.zeros_like(prob)
                want[0, 3], want[0, 5] = q[0] * (3 - 2 * mean), q[2] * (-1 - mean)
            else:
                want = prob * (G - (prob[0, [3, 3, 5]] * gw[0].double()).sum())
            assert torch.allclose(gx[0].double(), want, rtol=1e-5, atol=1e-7)
        idx[0, 1] = E
        c.moe_route_backward([x], [idx], [gw], gx)
        torch.cuda.synchronize()
        assert c.async_error() == SC.INVALID_ARG
        with pytest.raises(SC.SimCommError):
            c.moe_route([x], [idx], [gw])
        c.reset()
        idx[0, 1] = 0
        c.moe_route_backward([x], [idx], [gw], gx)
        torch.cuda.synchronize()
        assert c.async_error() == SC.OK


def test_odd_addresses_and_a_graph_and_a_view():
    T, E, k = 37, 64, 2
    flat = torch.randn(T * E + 3, device="cuda")
    x = flat[3:].view(T, E)  # 12 bytes past an aligned address
    idx, w = route([x], k, True)
    ri, _, rw = reference(x, k, True)
    assert torch.equal(idx[0].long(), ri) and torch.allclose(w[0].double(), rw, rtol=1e-5)
    with SC.SimComm(1) as c:
        s = torch.cuda.Stream()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            c.moe_route([x], idx, w)
        flat.copy_(torch.randn_like(flat))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        ri, _, rw = reference(x, k, True)
        assert torch.equal(idx[0].long(), ri) and torch.allclose(w[0].double(), rw, rtol=1e-5)
        del graph
    with SC.SimComm(4, rank=1) as v:
        i2, w2 = torch.empty_like(idx[0]), torch.empty_like(w[0])
        v.moe_route([None, x, None, None], [None, i2, None, None], [None, w2, None, None])
        torch.cuda.synchronize()
        assert torch.equal(i2, idx[0]) and torch.equal(w2, w[0])


def test_refusals():
    x = [torch.zeros(4, 8, device="cuda") for _ in range(2)]
    idx = [torch.zeros(4, 2, dtype=torch.int32, device="cuda") for _ in range(2)]
    w = [torch.zeros(4, 2, device="cuda") for _ in range(2)]
    with SC.SimComm(2) as c:
        with pytest.raises(SC.SimCommError, match="overlap"):
            c.moe_route(x, idx, [w[0], w[0]])
        with pytest.raises(SC.SimCommError, match="overlap"):
            c.moe_route(x, idx, [w[0], x[1].view(-1)[:8].view(4, 2)])
        with pytest.raises(SC.SimCommError, match="k exceeds"):
            c.moe_route(x, [torch.zeros(4, 9, dtype=torch.int32, device="cuda") for _ in range(2)],
                        [torch.zeros(4, 9, device="cuda") for _ in range(2)])
        with pytest.raises(SC.SimCommError) as e:
            c.moe_route([t.int() for t in x], idx, w)
        assert e.value.status == SC.UNSUPPORTED
        with pytest.raises(SC.SimCommError, match="multiple of p"):
            c.moe_route([torch.zeros(4, 9, device="cuda") for _ in range(2)], idx, w)
        with pytest.raises(TypeError):
            c.moe_route(x, [t.long() for t in idx], w)
        with pytest.raises(ValueError):
            c.moe_route(x, idx, [t.t().contiguous().t() for t in w])
        with pytest.raises(ValueError):
            c.moe_route(x, idx, [w[0], w[1].cpu()])
        with pytest.raises(ValueError):
            c.moe_route(x[:1], idx, w)
        n = c.launch_count()
        c.moe_route([t[:0] for t in x], [t[:0] for t in idx], [t[:0] for t in w])  # no tokens
        assert c.launch_count() == n
