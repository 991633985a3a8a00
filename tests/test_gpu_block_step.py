"""The norm, the adapters, the score adjustment and the distillation run together with the operators beside them, as they
are used: what one leaves on the ranks is what the next takes.

  decode: attention output (4-bit, row parallel) with the requests' adapters -> the ranks' sum is whole, so the norm of one
  rank's rows with the residual -> vocabulary head (4-bit, column parallel) -> penalties, biases, grammar -> log probabilities
  training: a teacher's log probabilities -> the distillation loss of the student's scores and its gradient -> the norm's
"""
import math

import pytest
import torch

from collective_communication_primitives_b200 import simcomm as SC
from test_gpu_adapters import Adapted
from test_gpu_moe_layer import make_weights
from test_gpu_rmsnorm import EPS

pytestmark = pytest.mark.gpu
BF, I32 = torch.bfloat16, torch.int32


def close(got, want, half):
    """Each operator's output from what the operator before it left: four times the rounding of its type relative to the
    largest output (the single operators' tests hold the element-wise bounds)."""
    fin = want.isfinite()
    if not torch.equal(got.double()[~fin], want[~fin]):
        return False
    return not bool(fin.any()) or float((got.double() - want)[fin].abs().max()) <= 4 * half * float(want[fin].abs().max())


class Step:
    """T tokens of as many requests, after a block's attention, on p ranks."""

    def __init__(self, p, T, H, V, S, R, seed=0):
        g = torch.Generator("cuda").manual_seed(seed)
        randn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        ints = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=g, device="cuda", dtype=I32)  # noqa: E731
        new = lambda *s, t=torch.float32: [torch.empty(*s, dtype=t, device="cuda") for _ in range(p)]  # noqa: E731
        self.p, self.T, self.V = p, T, V
        self.x = [randn(T, H // p).to(BF) for _ in range(p)]
        self.w, self.ws, self.wd = zip(*[make_weights(g, (H,), H // p, 32) for _ in range(p)])
        self.ad = Adapted(p, T, H, H, S, R, "row", "fp32", "fp32", seed=seed, whole=False)
        self.ad.x = self.x
        self.ad.X = torch.cat(self.x, 1)
        self.proj, self.sum = new(T, H), new(T, H)
        self.res, self.weight = randn(T, H), 1 + 0.1 * randn(H)
        self.total, self.y = [torch.empty(T, H, device="cuda")], [torch.empty(T, H, device="cuda")]
        self.hidden = new(T, H, t=BF)
        self.head, self.heads, self.headd = zip(*[make_weights(g, (V // p,), H, 64) for _ in range(p)])
        self.logits = new(T, V // p)
        self.hist, self.len = ints(0, V, T, 30), ints(0, 31, T)
        self.rep, self.freq, self.pres = 1 + torch.rand(T, device="cuda"), torch.rand(T, device="cuda"), torch.rand(T, device="cuda")
        self.mask, self.mask_row = ints(-2 ** 31, 2 ** 31 - 1, 2, V // 32), ints(-1, 2, T)
        self.ids = ints(0, V, T)
        self.changed = new(T, V // p)
        self.lp, self.lse, self.ti, self.tl = new(T), new(T), new(T, 4, t=I32), new(T, 4)

    def run(self, c, one):
        c.linear_w4(self.x, self.w, self.ws, self.proj, parallel="row")
        c.adapters(self.x, self.ad.ad, self.ad.a, self.ad.b, self.sum, base=self.proj, scale=self.ad.sc, parallel="row")
        one.rmsnorm(self.sum[:1], self.weight, EPS, out=self.y, residual=self.res, total=self.total)
        for h in self.hidden:
            h.copy_(self.y[0])
        c.linear_w4(self.hidden, self.head, self.heads, self.logits, parallel="column")
        c.adjust_logits(self.logits, self.V, self.changed, history=self.hist, history_len=self.len, repetition=self.rep,
                        frequency=self.freq, presence=self.pres, mask=self.mask, mask_row=self.mask_row)
        c.logprobs(self.changed, self.ids, self.V, self.lp, lse=self.lse, top_idx=self.ti, top_logprob=self.tl)

    def check(self):
        proj = sum(a.double() @ w.t() for a, w in zip(self.x, self.wd))
        assert all(close(v, proj, 2.0 ** -16) for v in self.proj)
        self.ad.base64 = self.proj[0]
        y, err = self.ad.exact()
        assert all(bool(((v.double() - y).abs() <= err + 2.0 ** -23 * y.abs()).all()) for v in self.sum)
        h = self.sum[0].double() + self.res.double()
        assert close(self.total[0], h, 2.0 ** -23)
        assert close(self.y[0], h / torch.sqrt(h.square().mean(1, keepdim=True) + EPS) * self.weight.double(), 2.0 ** -21)
        logits = torch.cat([self.hidden[0].double() @ w.t() for w in self.headd], 1)
        x = torch.cat(self.logits, 1).double()
        assert close(x, logits, 2.0 ** -16)
        for t in range(self.T):
            ids = self.hist[t, :int(self.len[t])].long()
            u, n = torch.unique(ids, return_counts=True)
            r = self.rep[t].double()
            x[t, u] = torch.where(x[t, u] > 0, x[t, u] / r, x[t, u] * r) - self.freq[t].double() * n - self.pres[t].double()
            if int(self.mask_row[t]) >= 0:
                words = self.mask[int(self.mask_row[t])].long()
                x[t, torch.stack([(words >> i) & 1 for i in range(32)], 1).view(-1) == 0] = -math.inf
        got = torch.cat(self.changed, 1)
        assert close(got, x, 2.0 ** -22)
        lp = torch.log_softmax(got.double(), 1)
        assert close(self.lp[1], lp.gather(1, self.ids.long()[:, None])[:, 0], 2.0 ** -21)
        top = torch.sort(got, dim=1, descending=True, stable=True).indices[:, :4]
        assert torch.equal(self.ti[0].long(), top)


@pytest.mark.parametrize("p,T,H,V,S,R", [(2, 3, 256, 1024, 4, 8), (4, 20, 512, 4096, 6, 16), (8, 70, 256, 2048, 3, 20)])
def test_decode_step(p, T, H, V, S, R):
    s = Step(p, T, H, V, S, R)
    with SC.SimComm(p) as c, SC.SimComm(1) as one:
        for _ in range(2):
            s.run(c, one)
            torch.cuda.synchronize()
            assert c.async_error() == SC.OK and one.async_error() == SC.OK
            s.check()


def test_decode_step_as_a_graph_with_trace():
    s = Step(4, 8, 512, 4096, 5, 16)
    with SC.SimComm(4) as c, SC.SimComm(1) as one:
        for k in (c, one):
            k.set_option("trace", 1)
        s.run(c, one)
        torch.cuda.synchronize()
        got = c.trace_read()
        assert [r["coll"] for r in got] == ["linear_w4", "adapters", "linear_w4", "adjust_logits", "logprobs"]
        assert [r["launches"] for r in got] == [1, 2, 1, 1, 1]
        assert [(r["coll"], r["n"]) for r in one.trace_read()] == [("rmsnorm", 8)]
        for k in (c, one):
            k.set_option("trace", 0)
        stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            s.run(c, one)
        for a in s.x:
            a.copy_(torch.randn_like(a))
        s.ad.X = torch.cat(s.x, 1)
        s.hist.copy_(torch.roll(s.hist, 1, 0))
        for _ in range(3):
            graph.replay()
        torch.cuda.synchronize()
        assert c.async_error() == SC.OK and one.async_error() == SC.OK
        s.check()
        del graph


@pytest.mark.parametrize("tail", [False, True])
def test_training_step_from_a_teachers_alternatives(tail):
    """The teacher's alternatives as the log probabilities leave them, the student's scores from normed rows of two ranks'
    partial sums: the gradient down to those partial sums and the norm's weight, against float64."""
    p, T, H, V, n = 2, 12, 64, 101, 6
    g = torch.Generator("cuda").manual_seed(3)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    new = lambda *s, t=torch.float32: [torch.empty(*s, dtype=t, device="cuda") for _ in range(p)]  # noqa: E731
    m = -(-V // p)

    def sharded(x):
        out = [torch.zeros(T, m, device="cuda") for _ in range(p)]
        for r in range(p):
            part = x[:, r * m:(r + 1) * m]
            out[r][:, :part.shape[1]] = part
        return out
    teacher, rows, res, weight, proj = 2 * randn(T, V), [randn(T, H) for _ in range(p)], randn(T, H), 1 + 0.1 * randn(H), randn(H, V) / 8
    none = torch.full((T,), -1, dtype=I32, device="cuda")
    lp, ti, tl, total, y = new(T), new(T, n, t=I32), new(T, n), new(T, H), new(T, H)
    loss, stats, gl = new(T), new(T, 8), torch.full((T,), 1 / T, device="cuda")
    gx, gw = new(T, H), new(H)
    with SC.SimComm(p) as c:
        c.logprobs(sharded(teacher), none, V, lp, top_idx=ti, top_logprob=tl)
        c.rmsnorm(rows, weight, EPS, out=y, residual=res, total=total)
        scores = sharded(y[0] @ proj)
        c.distill(scores, V, ti[0], tl[0], loss, stats=stats, tail=tail)
        gs = [torch.empty_like(v) for v in scores]
        c.distill_backward(scores, V, ti[0], tl[0], stats, gl, gs, tail=tail)
        # a column-parallel product's backward leaves each rank its columns' part of the sum
        full = [torch.zeros(T, p * m, device="cuda") for _ in range(p)]
        for r in range(p):
            full[r][:, r * m:(r + 1) * m] = gs[r]
        c.rmsnorm_backward([f[:, :V] @ proj.t() for f in full], total[0], weight, EPS, gx, grad_weight=gw)
        torch.cuda.synchronize()
        assert c.async_error() == SC.OK
    xs = [v.double().requires_grad_() for v in rows]
    w = weight.double().requires_grad_()
    h = sum(xs) + res.double()
    z = torch.log_softmax((h / torch.sqrt(h.square().mean(1, keepdim=True) + EPS) * w) @ proj.double(), 1)
    best = torch.topk(torch.log_softmax(teacher.double(), 1), n, 1)
    assert torch.equal(best.indices.int(), ti[0])
    at = z.gather(1, best.indices)
    if tail:
        q = best.values.exp()
        left = 1 - q.sum(1)
        rest = 1 - at.exp().sum(1)
        want = (q * (best.values - at)).sum(1) + left * (left.log() - rest.log())
    else:
        lq = torch.log_softmax(best.values, 1)
        want = (lq.exp() * (lq - at)).sum(1)
    (want.sum() / T).backward()
    # two fp32 products of up to 101 terms lie between: their rounding, relative to the largest value
    slack = lambda v: 256 * 2.0 ** -23 * float(v.abs().max())  # noqa: E731
    assert float((loss[0].double() - want.detach()).abs().max()) <= slack(z.detach())
    for r in range(p):
        assert float((gx[r].double() - xs[r].grad).abs().max()) <= slack(xs[r].grad)
        assert float((gw[r].double() - w.grad).abs().max()) <= slack(w.grad)


def test_two_communicators_at_once_on_two_streams():
    a, b = Step(2, 6, 256, 1024, 4, 8, seed=1), Step(4, 9, 512, 2048, 3, 12, seed=2)
    with SC.SimComm(2) as c, SC.SimComm(4) as d, SC.SimComm(1) as e, SC.SimComm(1) as f:
        s, t = torch.cuda.Stream(), torch.cuda.Stream()
        torch.cuda.synchronize()
        for _ in range(5):
            with torch.cuda.stream(s):
                a.run(c, e)
            with torch.cuda.stream(t):
                b.run(d, f)
        torch.cuda.synchronize()
        assert all(k.async_error() == SC.OK for k in (c, d, e, f))
        a.check()
        b.check()
