"""GPU tests of the log probabilities, entropy, alternatives and their gradient against float64.

Columns are whole numbers and must be equal (the lower column among equal scores). With D the largest
|x - max| that matters (at most 104: below e^-104 a term vanishes in fp32): an exponential errs by 2^-22
plus D 2^-23 of itself, a sum of V positive terms by another (V / 256 + 32) 2^-24 (a thread's chain and the
joins), its logarithm by that absolutely plus 2^-23 of itself.
"""
import math

import pytest
import torch

from collective_communication_primitives_b200 import simcomm as SC

pytestmark = pytest.mark.gpu
DT = {"fp32": torch.float32, "bf16": torch.bfloat16}
inf = math.inf


def shards(x, p, ld_extra=0, offset=0, fill=77.0):
    """[R][V] cut into p tensors [R][ceil(V / p)], padding columns filled with a number that would show."""
    R, V = x.shape
    m = -(-V // p)
    out = []
    for r in range(p):
        ld = m + ld_extra
        buf = torch.full((R * ld + offset,), fill, dtype=x.dtype, device=x.device)
        v = buf[offset:].view(R, ld)[:, :m]
        part = x[:, r * m:(r + 1) * m]
        v[:, :part.shape[1]] = part
        out.append(v)
    return out


class Call:
    def __init__(self, x, ids, p=1, n=0, ld_extra=0, offset=0):
        self.x, self.ids, self.p, self.n, (self.R, self.V) = x, ids, p, n, x.shape
        self.logits = shards(x, p, ld_extra, offset)
        new = lambda *s, t=torch.float32: [torch.full(s, 9, dtype=t, device="cuda") for _ in range(p)]  # noqa: E731
        self.lp, self.en, self.lse = new(self.R), new(self.R), new(self.R)
        self.ti = new(self.R, n, t=torch.int32) if n else None
        self.tl = new(self.R, n) if n else None

    def run(self, c, **more):
        c.logprobs(self.logits, self.ids, self.V, self.lp, entropy=self.en, lse=self.lse, top_idx=self.ti,
                   top_logprob=self.tl, **more)

    def grad(self, c, gl, ge=None):
        m = self.logits[0].shape[1]
        gx = [torch.full((self.R, m), 5.0, dtype=self.x.dtype, device="cuda") for _ in range(self.p)]
        c.logprobs_backward(self.logits, self.ids, self.V, self.lse, gl, gx, entropy=self.en, grad_entropy=ge)
        return gx

    def check(self):
        x = self.x.double()
        logp = torch.log_softmax(x, 1)
        prob = logp.exp()
        h = -torch.special.xlogy(prob, prob).sum(1)
        exp_err = 2.0 ** -22 + 104 * 2.0 ** -23
        sum_err = exp_err + (self.V / 256 + 32) * 2.0 ** -24
        given = self.ids >= 0
        want = torch.where(given, logp.gather(1, self.ids.clamp(min=0).long()[:, None])[:, 0], 0)
        big = torch.where(x.isfinite(), x.abs(), 0).amax(1)
        for r in range(self.p):
            got = self.lp[r].double()
            fin = want.isfinite()
            assert torch.equal(got[~fin], want[~fin])
            assert bool(((got - want).abs()[fin] <= (2 * sum_err + 2.0 ** -22 * (want.abs() + 12))[fin]).all())
            assert bool(((self.lse[r].double() - torch.logsumexp(x, 1)).abs() <= 2 * sum_err + 2.0 ** -22 * (big + 12)).all())
            assert bool(((self.en[r].double() - h).abs() <= (4 * sum_err + 2.0 ** -22) * (h + 1)).all())
            if self.n:
                order = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :self.n]
                assert torch.equal(self.ti[r].long(), order)
                tw, tg = logp.gather(1, order), self.tl[r].double()
                fin = tw.isfinite()
                assert torch.equal(tg[~fin], tw[~fin])
                assert bool(((tg - tw).abs()[fin] <= (2 * sum_err + 2.0 ** -22 * (tw.abs() + 12))[fin]).all())
        return prob, logp, h, sum_err

    def check_grad(self, gx, gl, ge=None):
        prob, logp, h, sum_err = self.check()
        gl = torch.where(self.ids >= 0, gl.double(), 0)
        ge = torch.zeros_like(gl) if ge is None else ge.double()
        hit = torch.zeros_like(prob).scatter_(1, self.ids.clamp(min=0).long()[:, None], 1.0) * gl[:, None]
        held = torch.where(prob > 0, logp, 0) + h[:, None]
        want = hit - prob * (gl[:, None] + ge[:, None] * held)
        big = torch.where(self.x.isfinite(), self.x.abs(), 0).double().amax(1, keepdim=True)
        # The gradient is -P d with d = gl + ge (lp + H). lp and H carry the absolute errors that check() allows
        # them (a_lp: x - lse with |lse| <= big + 12; a_h), which pass to d as |ge| (a_lp + a_h) however small
        # lp + H itself is, and to P as its relative error a_lp plus the exponential's; the two additions and
        # the product in d round once each, relative to their parts.
        a_lp = 2 * sum_err + 2.0 ** -22 * (big + logp.abs().clamp(max=104) + 12)
        a_h = (4 * sum_err + 2.0 ** -22) * (h[:, None] + 1)
        part = gl[:, None].abs() + ge[:, None].abs() * (torch.where(prob > 0, logp, 0).abs() + h[:, None])
        d = (gl[:, None] + ge[:, None] * held).abs()
        slack = prob * ((a_lp + sum_err) * d + ge[:, None].abs() * (a_lp + a_h) + 2.0 ** -22 * part) + 1e-37
        half = torch.finfo(self.x.dtype).eps / 2
        slack = slack + (2.0 ** -23) * hit.abs()
        bound = slack + half * (want.abs() + slack)
        full = torch.cat([v.double() for v in gx], 1)
        assert bool(((full[:, :self.V] - want).abs() <= bound).all())
        assert bool((full[:, self.V:] == 0).all())


def scores(R, V, dtype, seed, scale=2.5):
    g = torch.Generator("cuda").manual_seed(seed)
    return (scale * torch.randn(R, V, generator=g, device="cuda")).to(DT[dtype])


def tokens(R, V, seed, none=False):
    g = torch.Generator("cuda").manual_seed(seed + 1)
    t = torch.randint(0, V, (R,), generator=g, device="cuda", dtype=torch.int32)
    if none:
        t[::3] = -1
    return t


CASES = [
    # p, R, V, n, extra columns between rows, element offset
    (1, 1, 1, 1, 0, 0), (1, 1, 7, 3, 0, 0), (2, 3, 9, 9, 0, 1), (3, 2, 100, 32, 5, 3), (4, 5, 1001, 4, 0, 0),
    (8, 1, 5000, 8, 0, 0), (8, 33, 50257, 5, 0, 0), (1, 2, 131072, 20, 0, 0), (2, 300, 4097, 2, 0, 0),
    (4, 1200, 777, 1, 3, 0), (64, 2, 70, 3, 0, 0), (16, 3, 20, 2, 0, 0), (1, 700, 2048, 0, 0, 0), (5, 4, 33001, 32, 7, 1),
]


@pytest.mark.parametrize("p,R,V,n,extra,offset", CASES)
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_logprobs_and_gradient(p, R, V, n, extra, offset, dtype):
    x, ids = scores(R, V, dtype, V + R), tokens(R, V, R, none=R > 2)
    a = Call(x, ids, p, n, extra, offset)
    g = torch.Generator("cuda").manual_seed(3)
    gl, ge = torch.randn(R, generator=g, device="cuda"), torch.randn(R, generator=g, device="cuda")
    with SC.SimComm(p) as c:
        a.run(c)
        gx, only = a.grad(c, gl, ge), a.grad(c, gl)
        torch.cuda.synchronize()
        assert c.async_error() == SC.OK
    a.check_grad(gx, gl, ge)
    a.check_grad(only, gl)
    assert all(torch.equal(v, a.lp[0]) for v in a.lp) and all(torch.equal(v, a.lse[0]) for v in a.lse)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("V", [600, 40000])
def test_masked_and_special_rows(dtype, V):
    low = torch.finfo(DT[dtype]).min
    x = scores(10, V, dtype, 5)
    x[0] = -inf                       # nothing left
    x[1] = -inf
    x[1, V - 2] = 1.5                 # one left
    x[2] = low                        # masked throughout by the lowest value: uniform
    x[3, 1::2] = -inf
    x[4, 1::2] = low
    x[5] = 0.0                        # constant: ties
    x[6, 3] = math.nan
    x[7, V - 1] = inf
    x[8] = -inf
    x[8, 5] = low                     # the lowest value next to nothing: certain
    x[9] = x[9] + (30000.0 if dtype == "fp32" else 300.0)
    ids = torch.tensor([0, V - 2, 4, 1, 1, 7, 0, 1, 5, 11], dtype=torch.int32, device="cuda")
    a = Call(x, ids, 4, 5)
    gl, ge = torch.ones(10, device="cuda"), torch.full((10,), 0.5, device="cuda")
    with SC.SimComm(4) as c:
        a.run(c)
        gx = a.grad(c, gl, ge)
        torch.cuda.synchronize()
        assert c.async_error() == SC.OK
    assert float(a.lp[0][0]) == -inf and float(a.lse[0][0]) == -inf and float(a.en[0][0]) == 0
    assert a.ti[0][0].tolist() == [0, 1, 2, 3, 4] and bool((a.tl[0][0] == -inf).all())
    for t in (6, 7):
        assert bool(a.lp[0][t].isnan()) and bool(a.lse[0][t].isnan()) and bool(a.en[0][t].isnan())
        assert bool(a.tl[0][t].isnan().all())
    assert int(a.ti[0][7][0]) == V - 1 and 3 not in a.ti[0][6].tolist()
    full = torch.cat(gx, 1)[:, :V]
    assert bool((full[0] == 0).all()) and bool(full[6].isnan().all())
    rows = [1, 2, 3, 4, 5, 8, 9]
    b = Call(x[rows], ids[rows], 4, 5)
    b.lp, b.en, b.lse = ([t[rows] for t in v] for v in (a.lp, a.en, a.lse))
    b.ti, b.tl = ([t[rows] for t in v] for v in (a.ti, a.tl))
    b.check_grad([g[rows] for g in gx], gl[rows], ge[rows])


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_masked_columns_get_zero_whatever_comes_in(dtype):
    """Gradients scaled by a power of two come out scaled by it, bit for bit, and masked columns stay at zero."""
    x, ids = scores(6, 5000, dtype, 8), tokens(6, 5000, 2)
    masked = torch.arange(5000, device="cuda") % 3 == 0
    x[::2, masked] = -inf
    x[1::2, masked] = torch.finfo(DT[dtype]).min
    ids = torch.where(ids % 3 == 0, ids - 2, ids).clamp(min=1)
    a = Call(x, ids, 2)
    one = torch.ones(6, device="cuda")
    with SC.SimComm(2) as c:
        a.run(c)
        plain, scaled = a.grad(c, one, one), a.grad(c, one * 2.0 ** 70, one * 2.0 ** 70)
        torch.cuda.synchronize()
    for u, v in zip(plain, scaled):
        assert torch.equal(u.double() * 2.0 ** 70, v.double())
    assert bool((torch.cat(scaled, 1)[:, masked] == 0).all())


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_far_scores_keep_their_differences(dtype):
    """Rows whose maximum is far from 0, in either direction, with neighbours one representable step below."""
    V = 3000
    x = torch.full((4, V), -inf, dtype=DT[dtype], device="cuda")
    for t, top in enumerate((2.0 ** 20, -2.0 ** 20, 2.0 ** 40, -2.0 ** 110)):
        x[t, 7::11] = top
    ids = torch.full((4,), 7, dtype=torch.int32, device="cuda")
    a = Call(x, ids, 2, 3)
    gl, ge = torch.ones(4, device="cuda"), torch.ones(4, device="cuda")
    with SC.SimComm(2) as c:
        a.run(c)
        gx = a.grad(c, gl, ge)
        torch.cuda.synchronize()
    n = len(range(7, V, 11))
    assert torch.allclose(a.lp[0], torch.full((4,), -math.log(n), device="cuda"), rtol=1e-5)
    assert torch.allclose(a.en[0], torch.full((4,), math.log(n), device="cuda"), rtol=1e-5)
    full = torch.cat(gx, 1)[:, :V].float()
    assert torch.allclose(full[:, 18], torch.full((4,), -1 / n, device="cuda"), rtol=2.0 ** -8)
    assert torch.allclose(full[:, 7], torch.full((4,), 1 - 1 / n, device="cuda"), rtol=2.0 ** -8)
    assert bool((full[:, 8] == 0).all())


@pytest.mark.parametrize("order", ["up", "down", "constant", "saw"])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_alternatives_in_hard_orders(order, dtype):
    V, n = 70001, 32
    at = torch.arange(V, device="cuda")
    v = {"up": at, "down": -at, "constant": 0 * at, "saw": at % 37}[order].float() * 1e-3
    x = v.to(DT[dtype]).expand(3, V).contiguous()
    for rows in (1, 3):
        a = Call(x[:rows], tokens(rows, V, 2), 3, n)
        with SC.SimComm(3) as c:
            a.run(c)
            torch.cuda.synchronize()
        a.check()
    many = Call(x[:1].expand(400, V)[:, :5000].contiguous(), tokens(400, 5000, 2), 2, n)  # one CTA per row
    with SC.SimComm(2) as c:
        many.run(c)
        torch.cuda.synchronize()
    many.check()


def test_gradient_against_differences():
    V = 11
    x = scores(1, V, "fp32", 4, 1.0)
    ids = torch.tensor([6], dtype=torch.int32, device="cuda")
    a = Call(x, ids, 2)
    gl, ge = torch.tensor([0.7], device="cuda"), torch.tensor([-1.3], device="cuda")
    with SC.SimComm(2) as c:
        a.run(c)
        gx = torch.cat(a.grad(c, gl, ge), 1)
        torch.cuda.synchronize()

    def loss(v):
        lp = torch.log_softmax(v, 1)
        return float(0.7 * lp[0, 6] + 1.3 * (lp.exp() * lp).sum())

    h = 1e-5  # truncation below 1e-9, rounding about 1e-10
    for v in range(V):
        lo, hi = x.double().clone(), x.double().clone()
        lo[0, v] -= h
        hi[0, v] += h
        assert abs((loss(hi) - loss(lo)) / (2 * h) - float(gx[0, v])) < 1e-6


def test_same_bits_views_graph_and_streams():
    R, V, p = 6, 30001, 4
    x, ids = scores(R, V, "bf16", 1), tokens(R, V, 1)
    a, b = Call(x, ids, p, 7), Call(x, ids, p, 7)
    with SC.SimComm(p) as c:
        a.run(c)
        torch.cuda.synchronize()
        for _ in range(5):
            b.run(c)
            torch.cuda.synchronize()
            for u, v in ((a.lp, b.lp), (a.en, b.en), (a.lse, b.lse), (a.ti, b.ti), (a.tl, b.tl)):
                assert all(torch.equal(s, t) for s, t in zip(u, v))
        graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        gl = torch.randn(R, device="cuda")
        gx = [torch.empty_like(t) for t in a.logits]
        with torch.cuda.graph(graph, stream=s):
            b.run(c)
            c.logprobs_backward(b.logits, ids, V, b.lse, gl, gx)
        n = Call(scores(R, V, "bf16", 9), tokens(R, V, 9), p, 7)
        for dst, src in zip(b.logits, n.logits):
            dst.copy_(src)
        ids.copy_(n.ids)
        big = Call(scores(40, 60000, "fp32", 2), tokens(40, 60000, 2), p, 32)
        big.run(c)  # needs more scratch: the graph keeps the old
        graph.replay()
        torch.cuda.synchronize()
        big.check()
        n.lp, n.en, n.lse, n.ti, n.tl = b.lp, b.en, b.lse, b.ti, b.tl
        n.check_grad(gx, gl)
        del graph
        s.wait_stream(torch.cuda.current_stream())
        m = Call(n.x, n.ids, p, 7)
        torch.cuda.synchronize()
        m.run(c, stream=s)
        s.synchronize()
        assert torch.equal(m.lp[0], n.lp[0])
    with SC.SimComm(p, rank=2) as v:
        only = lambda t: [None, None, t, None]  # noqa: E731
        lp, lse = torch.empty(R, device="cuda"), torch.empty(R, device="cuda")
        v.logprobs(n.logits, n.ids, V, only(lp), lse=only(lse))
        g2 = torch.empty_like(gx[2])
        v.logprobs_backward(n.logits, n.ids, V, only(lse), gl, only(g2))
        torch.cuda.synchronize()
        assert torch.equal(lp, n.lp[2]) and torch.equal(g2, gx[2])


def test_a_bad_token_is_reported_and_the_communicator_recovers():
    x = scores(4, 9000, "fp32", 3)
    with SC.SimComm(2) as c:
        for bad in (9000, -2, 2 ** 31 - 1):
            a = Call(x, torch.tensor([1, bad, 2, 3], dtype=torch.int32, device="cuda"), 2, 2)
            a.run(c)
            torch.cuda.synchronize()
            assert c.async_error() == SC.INVALID_ARG
            c.reset()
        a = Call(x, tokens(4, 9000, 1), 2, 2)
        a.run(c)
        torch.cuda.synchronize()
        assert c.async_error() == SC.OK
        a.check()
        a.ids[2] = 9000
        a.grad(c, torch.ones(4, device="cuda"))
        torch.cuda.synchronize()
        assert c.async_error() == SC.INVALID_ARG


def test_columns_between_the_rows_are_left_alone():
    R, V, p = 5, 30, 2
    a = Call(scores(R, V, "bf16", 6), tokens(R, V, 6), p)
    gl = torch.ones(R, device="cuda")
    wide = [torch.full((R, 20), 8.0, dtype=torch.bfloat16, device="cuda") for _ in range(p)]
    with SC.SimComm(p) as c:
        a.run(c)
        c.logprobs_backward(a.logits, a.ids, V, a.lse, gl, [w[:, :15] for w in wide])
        torch.cuda.synchronize()
    a.check_grad([w[:, :15].contiguous() for w in wide], gl)
    assert all(bool((w[:, 15:] == 8).all()) for w in wide)


def test_refusals():
    x, ids = scores(4, 10, "fp32", 3), tokens(4, 10, 3)
    a = Call(x, ids, 2, 2)
    with SC.SimComm(2) as c:
        with pytest.raises(SC.SimCommError, match="overlap"):
            c.logprobs(a.logits, ids, 10, a.lp, entropy=a.lp)
        with pytest.raises(SC.SimCommError, match="overlap"):
            c.logprobs_backward(a.logits, ids, 10, a.lse, a.lp[0], a.logits)  # never in place
        with pytest.raises(SC.SimCommError, match="top_n"):
            b = Call(x, ids, 2, 11)
            b.run(c)
        with pytest.raises(SC.SimCommError) as e:
            c.logprobs([t.int() for t in a.logits], ids, 10, a.lp)
        assert e.value.status == SC.UNSUPPORTED
        with pytest.raises(ValueError):
            c.logprobs(a.logits, ids, 11, a.lp)
        with pytest.raises(ValueError):
            c.logprobs(a.logits, ids, 10, a.lp, top_idx=a.ti)
        with pytest.raises(TypeError):
            c.logprobs(a.logits, ids.long(), 10, a.lp)
        with pytest.raises(ValueError):
            c.logprobs([t.t().contiguous().t() for t in a.logits], ids, 10, a.lp)
        with pytest.raises(ValueError):
            c.logprobs_backward(a.logits, ids, 10, a.lse, a.lp[0], a.logits, grad_entropy=a.lp[0])
        n = c.launch_count()
        c.logprobs([t[:0] for t in a.logits], ids[:0], 10, [t[:0] for t in a.lp])
        assert c.launch_count() == n
