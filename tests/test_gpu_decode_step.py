"""The tail of a decode step and a training step, the operators run together as they are used: the shards that one
leaves on the ranks are what the next takes, without a copy in between.

  attention output (4-bit, summed over the ranks) -> router scores -> router -> expert layer -> vocabulary head
  (4-bit, its rows on the ranks) -> log probabilities of the sampled tokens, entropy, alternatives
"""
import pytest
import torch

from collective_communication_primitives_b200 import simcomm as SC
from test_gpu_moe_layer import make_weights

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


class Step:
    """One block's weights and buffers on p ranks; every rank holds the same T tokens after the row-parallel sum,
    and routes its own T / p of them to the experts."""

    def __init__(self, p, T, H, F, E, k, V, seed=0):
        g = torch.Generator("cuda").manual_seed(seed)
        randn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.p, self.T, self.k, self.E, self.V = p, T, k, E, V
        self.attn = [randn(T, H // p).to(BF) for _ in range(p)]
        wo = [make_weights(g, (H,), H // p, 32) for _ in range(p)]
        self.wo, self.wos, self.wod = zip(*wo)
        self.hidden = [torch.empty(T, H, dtype=BF, device="cuda") for _ in range(p)]
        self.gate = (randn(H, E) * H ** -0.5).to(BF)
        up = [make_weights(g, (E // p, 2 * F), H, 64) for _ in range(p)]
        down = [make_weights(g, (E // p, H), F, 64) for _ in range(p)]
        self.up, self.ups, upd = zip(*up)
        self.down, self.downs, downd = zip(*down)
        self.upd, self.downd = torch.cat(upd), torch.cat(downd)
        head = [make_weights(g, (V // p,), H, 128) for _ in range(p)]
        self.head, self.heads, self.headd = zip(*head)
        n = T // p
        self.idx = [torch.empty(n, k, dtype=torch.int32, device="cuda") for _ in range(p)]
        self.w = [torch.empty(n, k, device="cuda") for _ in range(p)]
        self.scores = [torch.empty(n, E, device="cuda") for _ in range(p)]
        self.mixed = [torch.empty(n, H, dtype=BF, device="cuda") for _ in range(p)]
        self.all = [torch.empty(T, H, dtype=BF, device="cuda") for _ in range(p)]
        self.logits = [torch.empty(T, V // p, device="cuda") for _ in range(p)]
        self.ids = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
        new = lambda *s, t=torch.float32: [torch.empty(*s, dtype=t, device="cuda") for _ in range(p)]  # noqa: E731
        self.lp, self.en, self.lse, self.ti, self.tl = new(T), new(T), new(T), new(T, 5, t=torch.int32), new(T, 5)

    def run(self, c):
        n = self.T // self.p
        c.linear_w4(self.attn, self.wo, self.wos, self.hidden, parallel="row")
        mine = [h[r * n:(r + 1) * n] for r, h in enumerate(self.hidden)]
        for r in range(self.p):
            torch.matmul(mine[r].float(), self.gate.float(), out=self.scores[r])
        c.moe_route(self.scores, self.idx, self.w)
        c.moe_layer(mine, self.idx, self.w, self.E, self.up, self.down, self.mixed, up_scale=self.ups,
                    down_scale=self.downs, residual=mine)
        c.allgather(self.mixed, self.all)
        c.linear_w4(self.all, self.head, self.heads, self.logits, parallel="column")
        c.logprobs(self.logits, self.ids, self.V, self.lp, entropy=self.en, lse=self.lse, top_idx=self.ti,
                   top_logprob=self.tl)

    def check(self):
        """Each operator's output from what the operator before it left: its own error alone, at four times the
        rounding of its type relative to the largest output (the single operators' tests hold the element-wise
        bounds), the picks exactly."""
        close = lambda got, want, half: float((got.double() - want).abs().max()) <= 4 * half * float(want.abs().max())  # noqa: E731
        hidden = sum(a.double() @ w.t() for a, w in zip(self.attn, self.wod))
        assert all(close(h, hidden, 2.0 ** -8) for h in self.hidden)
        x = torch.cat([h[r * (self.T // self.p):(r + 1) * (self.T // self.p)] for r, h in enumerate(self.hidden)]).double()
        s = torch.cat(self.scores).double()
        want_idx = torch.sort(s, dim=1, descending=True, stable=True).indices[:, :self.k]
        assert torch.equal(torch.cat(self.idx).long(), want_idx)
        w = torch.softmax(s, 1).gather(1, want_idx)
        w = w / w.sum(1, keepdim=True)
        assert close(torch.cat(self.w), w, 2.0 ** -20)
        out, F = x.clone(), self.downd.shape[2]
        for t in range(self.T):
            for q in range(self.k):
                e = int(want_idx[t, q])
                a = self.upd[e] @ x[t]
                out[t] += w[t, q] * (self.downd[e] @ (torch.nn.functional.silu(a[:F]) * a[F:]))
        assert close(torch.cat(self.mixed), out, 2.0 ** -8)
        assert all(torch.equal(v, torch.cat(self.mixed)) for v in self.all)
        logits = torch.cat([self.all[0].double() @ w.t() for w in self.headd], 1)
        got = torch.cat(self.logits, 1)
        assert close(got, logits, 2.0 ** -18)
        lp = torch.log_softmax(got.double(), 1)
        assert close(self.lp[1], lp.gather(1, self.ids.long()[:, None])[:, 0], 2.0 ** -21)
        assert close(self.en[0], -(lp.exp() * lp).sum(1), 2.0 ** -20)
        top = torch.sort(got, dim=1, descending=True, stable=True).indices[:, :5]
        assert torch.equal(self.ti[0].long(), top) and close(self.tl[0], lp.gather(1, top), 2.0 ** -21)


@pytest.mark.parametrize("p,T,H,F,E,k,V", [(2, 2, 256, 128, 8, 2, 1024), (4, 8, 512, 256, 16, 4, 4096), (8, 8, 256, 64, 8, 2, 2048)])
def test_decode_step(p, T, H, F, E, k, V):
    s = Step(p, T, H, F, E, k, V)
    with SC.SimComm(p) as c:
        for _ in range(2):
            s.run(c)
            torch.cuda.synchronize()
            assert c.async_error() == SC.OK
            s.check()


def test_decode_step_as_a_graph_with_trace():
    s = Step(4, 8, 512, 256, 16, 4, 4096)
    with SC.SimComm(4) as c:
        c.set_option("trace", 1)
        s.run(c)
        torch.cuda.synchronize()
        names = [r["coll"] for r in c.trace_read()]
        assert names == ["linear_w4", "moe_route", "moe_layer", "allgather", "linear_w4", "logprobs"]
        c.set_option("trace", 0)
        stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            s.run(c)
        for a in s.attn:
            a.copy_(torch.randn_like(a))
        for _ in range(3):
            graph.replay()
        torch.cuda.synchronize()
        assert c.async_error() == SC.OK
        s.check()
        del graph


def test_two_graphs_of_one_communicator_in_turn():
    """They share the communicator's scratch: replayed one after the other, each is right."""
    a, b = Step(2, 4, 256, 128, 8, 2, 1024, seed=1), Step(2, 8, 512, 192, 16, 4, 2048, seed=2)
    with SC.SimComm(2) as c:
        stream = torch.cuda.Stream()
        graphs = []
        for s in (a, b):
            s.run(c)
            torch.cuda.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=stream):
                s.run(c)
            graphs.append(g)
        for _ in range(4):
            for g in graphs:
                g.replay()
        torch.cuda.synchronize()
        a.check()
        b.check()
        del graphs, g


def test_training_step_of_router_and_loss():
    """The gradient of a loss through the log probabilities and through the router's weights, against float64."""
    p, T, E, k, V = 2, 6, 16, 3, 101
    g = torch.Generator("cuda").manual_seed(7)
    scores = [torch.randn(T, E, generator=g, device="cuda") for _ in range(p)]
    proj = torch.randn(k, V, generator=g, device="cuda")
    ids = torch.randint(0, V, (p * T,), generator=g, device="cuda", dtype=torch.int32)
    ids[3] = -1
    idx = [torch.empty(T, k, dtype=torch.int32, device="cuda") for _ in range(p)]
    w = [torch.empty(T, k, device="cuda") for _ in range(p)]
    m = -(-V // p)
    with SC.SimComm(p) as c:
        c.moe_route(scores, idx, w)
        logits = torch.cat(w) @ proj  # a stand-in for the layers between router and head
        shards = [torch.zeros(p * T, m, device="cuda") for _ in range(p)]
        for r in range(p):
            part = logits[:, r * m:(r + 1) * m]
            shards[r][:, :part.shape[1]] = part
        lp, lse, en = ([torch.empty(p * T, device="cuda") for _ in range(p)] for _ in range(3))
        c.logprobs(shards, ids, V, lp, lse=lse, entropy=en)
        gl = torch.full((p * T,), -1.0 / (p * T), device="cuda")  # the loss: minus the mean of the log probabilities
        gx = [torch.empty_like(s) for s in shards]
        c.logprobs_backward(shards, ids, V, lse, gl, gx)
        gw = (torch.cat(gx, 1)[:, :V] @ proj.t()).view(p, T, k)
        gs = [torch.empty_like(s) for s in scores]
        c.moe_route_backward(scores, idx, list(gw), gs)
        torch.cuda.synchronize()
        assert c.async_error() == SC.OK
    x = torch.cat(scores).double().requires_grad_()
    q = torch.softmax(x, 1).gather(1, torch.cat(idx).long())
    z = (q / q.sum(1, keepdim=True)) @ proj.double()
    keep = ids >= 0
    loss = -torch.log_softmax(z, 1).gather(1, ids.clamp(min=0).long()[:, None])[:, 0][keep].sum() / (p * T)
    loss.backward()
    assert abs(float(loss.detach()) + float(lp[0].sum()) / (p * T)) < 1e-5
    # two fp32 products of up to 101 terms lie between: their rounding, relative to the largest gradient
    assert float((torch.cat(gs).double() - x.grad).abs().max()) <= 256 * 2.0 ** -23 * float(x.grad.abs().max())
