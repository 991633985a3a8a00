"""GPU tests of the distillation loss and its gradient against float64.

As in the log probabilities an exponential errs by 2^-22 plus D 2^-23 of itself, D at most 104 (below e^-104 a term
vanishes), a sum of V of them by another (V / 256 + 32) 2^-24: sum_err. ln P and ln P_rest carry that twice, q nothing
beside its 64 bits, so the loss errs by 2 sum_err (sum q + Q) and its own rounding. In the gradient P carries
sum_err, the exponential and the rounding of the two logarithms that the forward call leaves (2^-22 of up to 40), off
the list k = A P_rest - Q errs by 2 sum_err A P_rest and a rounding.
"""
import math

import pytest
import torch

from collective_communication_primitives_b200 import simcomm as SC
from test_gpu_logprobs import shards

pytestmark = pytest.mark.gpu
DT = {"fp32": torch.float32, "bf16": torch.bfloat16}
inf = math.inf


class Distill:
    def __init__(self, x, idx, val, p=1, tau=1.0, tail=False, ld_extra=0, offset=0):
        self.x, self.idx, self.val, self.p, self.tau, self.tail = x, idx.int().contiguous(), val.float().contiguous(), p, tau, tail
        self.R, self.V = x.shape
        self.logits = shards(x, p, ld_extra, offset)
        new = lambda *s: [torch.full(s, 9.0, device="cuda") for _ in range(p)]  # noqa: E731
        self.loss, self.stats = new(self.R), new(self.R, 8)

    def run(self, c, **more):
        c.distill(self.logits, self.V, self.idx, self.val, self.loss, stats=self.stats, temperature=self.tau, tail=self.tail, **more)

    def grad(self, c, g, ld_extra=0, offset=0, **more):
        self.gx = shards(torch.full_like(self.x, 5), self.p, ld_extra, offset, fill=5.0)
        c.distill_backward(self.logits, self.V, self.idx, self.val, self.stats, g, self.gx, temperature=self.tau, tail=self.tail, **more)

    def exact(self):
        x = self.x.double() / self.tau
        logp = torch.log_softmax(x, 1)
        none = (x == -inf).all(1)
        logp[none] = -inf
        given = self.idx >= 0
        ids = torch.where(given, self.idx, self.V).long()
        v = self.val.double().masked_fill(~given, -inf) / self.tau
        if self.tail:
            q, lq = v.exp(), v
        else:
            teacher = (v > -inf).any(1, keepdim=True)
            lq = torch.where(teacher, torch.log_softmax(v, 1), -inf)
            q = lq.exp()
        lp = torch.cat((logp, torch.zeros(self.R, 1, device="cuda")), 1).gather(1, ids)
        loss = torch.where(q > 0, q * (lq - lp), 0).sum(1)
        on = torch.zeros(self.R, self.V + 1, dtype=torch.bool, device="cuda").scatter_(1, ids, True)[:, :self.V]
        A = q.sum(1)
        rest = torch.ones_like(A)
        Q = torch.zeros_like(A)
        if self.tail:
            ln_rest = torch.logsumexp(logp.masked_fill(on, -inf), 1)
            rest = ln_rest.exp()
            Q = 1 - A
            Q = torch.where(Q < 2.0 ** -20, 0, Q)
            loss = loss + torch.where(Q > 0, Q * (Q.log() - ln_rest), 0)
            A = A + Q
        full_q = torch.zeros(self.R, self.V + 1, dtype=torch.float64, device="cuda").scatter_add_(1, ids, q)[:, :self.V]
        return logp, on, full_q, A, Q, rest, none, loss

    def sum_err(self):
        exp_err = 2.0 ** -22 + 104 * 2.0 ** -23
        return exp_err, exp_err + (self.V / 256 + 32) * 2.0 ** -24

    def check(self):
        logp, on, q, A, Q, rest, none, loss = self.exact()
        _, e = self.sum_err()
        for r in range(self.p):
            got = self.loss[r].double()
            fin = loss.isfinite()
            assert torch.equal(got[~fin], loss[~fin])
            assert bool(((got - loss).abs()[fin] <= (2 * e * A + 2.0 ** -24 * loss.abs() + 1e-12)[fin]).all())

    def check_grad(self, g):
        logp, on, q, A, Q, rest, none, loss = self.exact()
        exp_err, e = self.sum_err()
        e_p = e + exp_err + 40 * 2.0 ** -22
        P = logp.exp()
        s = (g.double() / self.tau)[:, None]
        A, Q, rest = A[:, None], Q[:, None], rest[:, None]
        # P / P_rest of the columns off the list, also where both vanish
        cond = torch.nan_to_num(torch.softmax((self.x.double() / self.tau).masked_fill(on, -inf), 1), nan=0.0)
        off = cond * (A * rest - Q)
        want = s * torch.where(on | torch.tensor(not self.tail, device="cuda"), A * P - q, off)
        slack = s.abs() * torch.where(on, A * P * e_p + 2.0 ** -22 * (A * P + q),
                                      cond * ((A * rest - Q).abs() * e_p + 2 * e * A * rest + 2.0 ** -23 * (A * rest + Q)))
        if not self.tail:
            slack = s.abs() * (A * P * e_p + 2.0 ** -22 * (A * P + q))
        want[none] = 0
        half = torch.finfo(self.x.dtype).eps / 2
        full = torch.cat([v.double() for v in self.gx], 1)
        bound = slack + half * (want.abs() + slack) + 1e-37
        assert bool(((full[:, :self.V] - want).abs() <= bound).all())
        m = -(-self.V // self.p)
        assert bool((torch.cat([v[:, :m].double() for v in self.gx], 1)[:, self.V:] == 0).all())


def make(R, V, n, dtype, seed, tail, scale=2.5, peaked=False):
    g = torch.Generator("cuda").manual_seed(seed)
    t = scale * torch.randn(R, V, generator=g, device="cuda")
    if peaked:
        t[:, V // 3] += 20
    x = (t + 0.5 * torch.randn(R, V, generator=g, device="cuda")).to(DT[dtype])
    lp = torch.log_softmax(t.double(), 1)
    best = torch.topk(lp if tail else t.double(), n, 1)
    return x, best.indices, best.values


SIZES = [(1, 1, 1, 1), (1, 2, 3, 2), (2, 5, 37, 5), (4, 3, 1001, 32), (8, 7, 4096, 64), (3, 9, 20011, 256), (1, 4, 70000, 100),
         (8, 3, 131072, 32), (64, 2, 200, 7), (2, 900, 1000, 20), (1, 5000, 33, 3)]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("tail,tau", [(False, 1.0), (False, 2.5), (True, 1.0)])
@pytest.mark.parametrize("p,R,V,n", SIZES)
def test_loss_and_gradient(p, R, V, n, tail, tau, dtype):
    x, idx, val = make(R, V, n, dtype, V + n, tail)
    gl = torch.randn(R, device="cuda", generator=torch.Generator("cuda").manual_seed(R))
    with SC.SimComm(p) as c:
        a = Distill(x, idx, val, p, tau, tail)
        a.run(c)
        a.grad(c, gl)
        torch.cuda.synchronize()
        assert c.async_error() == SC.OK
        a.check()
        a.check_grad(gl)
        first = a.loss[0].clone()
        a.run(c)
        torch.cuda.synchronize()
        assert all(torch.equal(first, v) for v in a.loss)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("ld_extra,offset", [(1, 0), (3, 1), (8, 8)])
@pytest.mark.parametrize("tail", [False, True])
def test_rows_at_any_distance(tail, ld_extra, offset, dtype):
    x, idx, val = make(6, 5003, 40, dtype, 3, tail)
    gl = torch.ones(6, device="cuda")
    with SC.SimComm(3) as c:
        a = Distill(x, idx, val, 3, 1.0, tail, ld_extra, offset)
        a.run(c)
        a.grad(c, gl, 2, 1)
        torch.cuda.synchronize()
        a.check()
        a.check_grad(gl)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_peaked_rows_keep_the_rest(dtype):
    """Nearly all probability on a listed column: what is left beside it is a sum of its own."""
    x, idx, val = make(5, 8000, 16, dtype, 9, True, peaked=True)
    x[1, 8000 // 3] += 60  # the rest has e^-60 and less
    x[2] -= 3000
    gl = torch.ones(5, device="cuda")
    with SC.SimComm(2) as c:
        a = Distill(x, idx, val, 2, 1.0, True)
        a.run(c)
        a.grad(c, gl)
        torch.cuda.synchronize()
        a.check()
        a.check_grad(gl)


@pytest.mark.parametrize("tail", [False, True])
def test_open_places_repeated_columns_and_every_column(tail):
    V, n = 50, 50
    x, idx, val = make(6, V, n, "fp32", 4, tail)
    idx[0, 10:] = -1
    val[0, 10:] = math.nan  # not read where no column is given
    idx[1, :] = -1
    idx[2, 1::2] = idx[2, 0::2]          # every column twice
    val[2] -= math.log(4)
    val[3, 7:] = -inf
    idx[4, 5] = idx[4, 0]
    gl = torch.rand(6, device="cuda") + 0.5
    with SC.SimComm(4) as c:
        a = Distill(x, idx, val, 4, 1.0, tail)
        a.run(c)
        a.grad(c, gl)
        torch.cuda.synchronize()
        assert c.async_error() == SC.OK
        a.val = torch.nan_to_num(a.val, nan=0.0)
        a.check()
        a.check_grad(gl)
        if not tail:  # no teacher: no loss, no gradient
            assert float(a.loss[0][1]) == 0 and all(bool((v[1] == 0).all()) for v in a.gx)


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_masked_far_and_special_rows(dtype, tail):
    low = torch.finfo(DT[dtype]).min
    x, idx, val = make(12, 3000, 8, dtype, 5, tail)
    x[0, ::2] = -inf
    x[1, ::2] = low
    x[2] = -inf
    x[3] = low
    x[4] += 30000
    x[5] = x[5] * 1e30
    x[6, int(idx[6, 2])] = -inf          # the teacher wants what the student masks
    x[7, 100] = math.nan
    x[8, 200] = inf
    x[9, int(idx[9, 0])] = math.nan
    val[10, 3] = math.nan
    on = torch.zeros(3000, dtype=torch.bool, device="cuda")
    on[idx[11]] = True
    x[11, ~on] = -inf                    # nothing but listed columns
    gl = torch.ones(12, device="cuda")
    with SC.SimComm(3) as c:
        a = Distill(x, idx, val, 3, 1.0, tail)
        a.run(c)
        a.grad(c, gl)
        torch.cuda.synchronize()
    bad = [7, 8, 9, 10]
    for r in range(3):
        assert bool(a.loss[r][bad].isnan().all())
    full = torch.cat(a.gx, 1)[:, :3000]
    assert all(bool(full[t].isnan().any()) for t in bad)
    assert bool(full[7].isnan().all()) and bool(full[10].isnan().all())
    keep = [t for t in range(12) if t not in bad]
    b = Distill(x[keep], idx[keep], val[keep], 3, 1.0, tail)
    b.loss = [v[keep] for v in a.loss]
    b.gx = [v[keep] for v in a.gx]
    b.check()
    assert float(b.loss[0][6]) == inf
    if tail:  # the class of the rest has q but no P
        assert float(b.loss[0][7]) == inf
    b.check_grad(gl[keep])


def test_gradient_against_differences():
    for tail, tau in ((False, 1.7), (True, 1.0)):
        x, idx, val = make(3, 60, 6, "fp32", 8, tail)
        gl = torch.tensor([1.0, -2.0, 0.5], device="cuda")
        with SC.SimComm(2) as c:
            a = Distill(x, idx, val, 2, tau, tail)
            a.run(c)
            a.grad(c, gl)
            torch.cuda.synchronize()
        full = torch.cat(a.gx, 1)[:, :60].double()
        for seed in range(3):
            d = torch.randn(3, 60, dtype=torch.float64, device="cuda", generator=torch.Generator("cuda").manual_seed(seed))
            step, f = 1e-4, []
            for s in (step, -step):
                b = Distill(x.double() + s * d, idx, val, 1, tau, tail)
                f.append(float((b.exact()[-1] * gl.double()).sum()))
            num = (f[0] - f[1]) / (2 * step)
            assert abs(num - float((full * d).sum())) <= 1e-5 * float((full * d).abs().sum())


def test_as_a_graph_with_a_second_one_of_the_same_scratch():
    calls = []
    for R, V in ((3, 20000), (7, 50000)):
        x, idx, val = make(R, V, 16, "bf16", R, True)
        calls.append((Distill(x, idx, val, 2, 1.0, True), torch.rand(R, device="cuda")))
    with SC.SimComm(2) as c:
        stream, graphs = torch.cuda.Stream(), []
        for a, g in reversed(calls):
            a.run(c)
            a.grad(c, g)
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=stream):
                a.run(c)
                c.distill_backward(a.logits, a.V, a.idx, a.val, a.stats, g, a.gx, tail=True)
            graphs.append(graph)
        for a, g in calls:
            a.x = a.x.flip(1)
            for dst, src in zip(a.logits, shards(a.x, 2)):
                dst.copy_(src)
            for t in a.loss + a.gx:
                t.fill_(3)
        for _ in range(2):
            for graph in graphs:
                graph.replay()
        torch.cuda.synchronize()
        assert c.async_error() == SC.OK
        for a, g in calls:
            a.check()
            a.check_grad(g)
        del graph, graphs


def test_refusals_and_bad_columns():
    x, idx, val = make(4, 500, 8, "fp32", 1, False)
    with SC.SimComm(2) as c:
        a = Distill(x, idx, val, 2)
        for tau in (0.0, -1.0, math.nan, inf):
            with pytest.raises(SC.SimCommError, match="temperature"):
                c.distill(a.logits, 500, a.idx, a.val, a.loss, temperature=tau)
        with pytest.raises(SC.SimCommError, match="temperature"):
            c.distill(a.logits, 500, a.idx, a.val, a.loss, temperature=2.0, tail=True)
        with pytest.raises(SC.SimCommError, match="top_n"):
            c.distill(a.logits, 500, torch.zeros(4, 257, dtype=torch.int32, device="cuda"), torch.zeros(4, 257, device="cuda"), a.loss)
        with pytest.raises(SC.SimCommError, match="two output"):
            c.distill(a.logits, 500, a.idx, a.val, [a.loss[0], a.loss[0]])
        with pytest.raises(SC.SimCommError, match="overlap"):
            c.distill_backward(a.logits, 500, a.idx, a.val, a.stats, torch.ones(4, device="cuda"), a.logits)
        before = c.launch_count()
        c.distill([v[:0] for v in a.logits], 500, a.idx[:0], a.val[:0], [v[:0] for v in a.loss])
        assert c.launch_count() == before
        for value in (500, -2):
            a.idx[1, 3] = value
            a.run(c)
            torch.cuda.synchronize()
            assert c.async_error() == SC.INVALID_ARG
            c.reset()
            a.idx[1, 3] = 0
            a.run(c)
            a.idx[1, 3] = value
            a.grad(c, torch.ones(4, device="cuda"))
            torch.cuda.synchronize()
            assert c.async_error() == SC.INVALID_ARG
            c.reset()
        a.idx[1, 3] = 0
        a.run(c)
        torch.cuda.synchronize()
        a.check()
