"""GPU tests of the expert layer for few tokens against float64, and against the dispatch and combine.

Per element, with S_a = the sum of the magnitudes of a product's terms: a sum of K exact products in fp32
errs by at most K 2^-23 S (a matrix instruction may truncate), silu(g) u passes that on with |silu'| <= 1.1
plus 2^-20 of itself (exponential, quotient, product), its rounding to bf16 is 2^-8 of it, the second sum
adds F 2^-23 of its terms, the weighted sum (k + 1) 2^-24 of its own, and the output's rounding 2^-8.
"""
import pytest
import torch

from collective_communication_primitives_b200 import simcomm as SC

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def pack4(q):
    """uint8 [..., K] values 0..15 -> packed [..., K/2]."""
    return (q[..., 0::2] | (q[..., 1::2] << 4)).contiguous()


def make_weights(g, lead, K, group):
    """(tensor, scale or None, float64 values) of weights [*lead][K] of about 1/sqrt(K)."""
    if not group:
        w = (torch.randn(*lead, K, generator=g, device="cuda") * K ** -0.5).to(BF)
        return w, None, w.double()
    q = torch.randint(0, 16, (*lead, K), generator=g, device="cuda", dtype=torch.uint8)
    s = ((0.5 + torch.rand(*lead, K // group, generator=g, device="cuda")) * K ** -0.5 / 4.6).to(BF)
    return pack4(q), s, (q.double() - 8) * s.double().repeat_interleave(group, -1)


class Layer:
    def __init__(self, p, T, E, k, H, F, group=0, residual=True, seed=0, idx=None, offset=0):
        g = torch.Generator("cuda").manual_seed(seed)
        self.p, self.T, self.E, self.k, self.H, self.F = p, T, E, k, H, F

        def rows(scale=1.0):
            flat = (scale * torch.randn(T * H + offset, generator=g, device="cuda")).to(BF)
            return flat[offset:].view(T, H)
        self.x = [rows() for _ in range(p)]
        if idx is None:
            idx = torch.stack([torch.randperm(E, generator=g, device="cuda")[:k] for _ in range(p * T)]).view(p, T, k)
        self.idx = [i.contiguous() for i in idx.int()]
        self.w = [torch.randn(T, k, generator=g, device="cuda") for _ in range(p)]
        up = [make_weights(g, (E // p, 2 * F), H, group) for _ in range(p)]
        down = [make_weights(g, (E // p, H), F, group) for _ in range(p)]
        self.up, self.us, self.upd = [u[0] for u in up], [u[1] for u in up], torch.cat([u[2] for u in up])
        self.down, self.ds, self.downd = [d[0] for d in down], [d[1] for d in down], torch.cat([d[2] for d in down])
        self.group = group
        self.res = [rows() for _ in range(p)] if residual else None
        self.out = [torch.full((T, H), 3.0, dtype=BF, device="cuda") for _ in range(p)]

    def scales(self):
        return {"up_scale": self.us, "down_scale": self.ds} if self.group else {}

    def run(self, c, **more):
        c.moe_layer(self.x, self.idx, self.w, self.E, self.up, self.down, self.out, residual=self.res, **self.scales(),
                    **more)

    def check(self, out=None, y_rounding=0.0):
        """y_rounding: the relative rounding of the experts' outputs before the weighted sum."""
        p, T, k, H, F = self.p, self.T, self.k, self.H, self.F
        x = torch.cat(self.x).double()
        idx, w = torch.cat(self.idx).long(), torch.cat(self.w).double()
        want = torch.cat(self.res).double() if self.res else torch.zeros(p * T, H, dtype=torch.float64, device="cuda")
        mag, slack = want.abs(), torch.zeros_like(want)
        for e in torch.unique(idx).tolist():
            t, s = torch.nonzero(idx == e, as_tuple=True)
            up, down = self.upd[e], self.downd[e]
            a, am = x[t] @ up.t(), x[t].abs() @ up.abs().t()
            gate, u = a[:, :F], a[:, F:]
            silu = gate * torch.sigmoid(gate)
            h = silu * u
            dh = H * 2.0 ** -23 * (1.1 * u.abs() * am[:, :F] + silu.abs() * am[:, F:]) + h.abs() * (2.0 ** -8 + 2.0 ** -20)
            y, ym = h @ down.t(), h.abs() @ down.abs().t()
            dy = (dh + F * 2.0 ** -23 * h.abs()) @ down.abs().t()
            ws = w[t, s][:, None]
            want.index_add_(0, t, ws * y)
            mag.index_add_(0, t, ws.abs() * y.abs())
            slack.index_add_(0, t, ws.abs() * dy)
        got = torch.cat(self.out if out is None else out).double()
        bound = slack + ((k + 2) * 2.0 ** -24 + y_rounding) * mag
        bound = bound + 2.0 ** -8 * (want.abs() + bound)
        bad = (got - want).abs() > bound
        assert not bool(bad.any()), f"{int(bad.sum())} of {bad.numel()}, worst {float(((got - want).abs() / bound).max())}"


CASES = [
    # p, T, E, k, H, F, group, residual
    (1, 1, 1, 1, 8, 8, 0, False), (1, 1, 8, 2, 64, 32, 0, True), (2, 3, 8, 2, 40, 24, 0, True),
    (8, 1, 64, 2, 256, 128, 0, True), (4, 9, 16, 4, 104, 72, 0, False), (2, 40, 4, 3, 136, 88, 0, True),
    (1, 300, 8, 4, 64, 48, 0, True),                                   # over 100 assignments per expert
    (1, 1, 4, 2, 1, 1, 0, True), (2, 5, 6, 3, 33, 17, 0, True), (1, 3, 2, 2, 1001, 129, 0, False),  # rows of odd length
    (64, 1, 128, 8, 32, 16, 0, True), (3, 7, 4095, 5, 16, 8, 0, True),
    (1, 1, 2, 1, 32, 32, 32, True), (2, 3, 8, 2, 64, 96, 32, False), (4, 17, 8, 3, 128, 64, 64, True),
    (2, 1, 8, 2, 256, 128, 128, True), (1, 70, 4, 2, 384, 128, 128, False), (2, 9, 4, 2, 512, 256, 256, True),
    (1, 33, 4, 4, 160, 224, 32, True),
    (1, 512, 4096, 8, 16, 8, 0, True), (2, 256, 4096, 8, 32, 32, 32, False),  # as many assignments as there may be
]


@pytest.mark.parametrize("p,T,E,k,H,F,group,residual", CASES)
def test_layer(p, T, E, k, H, F, group, residual):
    a = Layer(p, T, E, k, H, F, group, residual, seed=p + T + E + H)
    with SC.SimComm(p) as c:
        a.run(c)
        torch.cuda.synchronize()
        assert c.async_error() == SC.OK
    a.check()


TENSOR_CASES = [
    # p, T, E, k, H, F, residual: rows of 16-byte units
    (1, 1, 1, 1, 8, 8, False), (1, 1, 8, 2, 64, 32, True), (2, 3, 8, 2, 40, 24, True), (8, 1, 64, 2, 256, 128, True),
    (4, 9, 16, 4, 104, 72, False), (2, 40, 4, 3, 136, 88, True), (1, 300, 8, 4, 64, 48, True), (4, 33, 16, 4, 1000, 712, False),
    (1, 700, 4, 4, 200, 264, True), (64, 1, 128, 8, 32, 16, True), (2, 64, 8, 8, 512, 384, True), (1, 20, 2, 1, 2048, 1024, True),
]


@pytest.mark.parametrize("p,T,E,k,H,F,residual", TENSOR_CASES)
def test_layer_on_the_tensor_cores(p, T, E, k, H, F, residual):
    a = Layer(p, T, E, k, H, F, 0, residual, seed=p + T + E + H)
    with SC.SimComm(p) as c:
        c.set_option("moe_layer_tensor", 1)
        for _ in range(2):
            a.run(c)
            torch.cuda.synchronize()
            assert c.async_error() == SC.OK
            a.check()


def test_both_kernels_take_turns_on_one_communicator():
    a, b = Layer(2, 40, 4, 3, 136, 88, seed=1), Layer(2, 64, 8, 4, 256, 128, seed=2)
    with SC.SimComm(2) as c:
        for option in (0, 1, 0, 1, -1):
            c.set_option("moe_layer_tensor", option)
            for x in (a, b):
                x.run(c)
            torch.cuda.synchronize()
            a.check()
            b.check()


@pytest.mark.parametrize("group", [0, 32])
def test_every_token_on_one_expert_and_an_id_twice(group):
    T, E, k = 67, 8, 2
    idx = torch.full((2, T, k), 5, device="cuda")
    a = Layer(2, T, E, k, 64, 64, group, seed=3, idx=idx)
    with SC.SimComm(2) as c:
        a.run(c)
        torch.cuda.synchronize()
    a.check()


def test_counts_around_the_token_tiles():
    """Experts with 1, 8, 9, 16, 17, 32, 33 and 65 assignments in one call, in no order."""
    counts = [1, 8, 9, 16, 17, 32, 33, 65]
    ids = torch.repeat_interleave(torch.arange(8), torch.tensor(counts))
    ids = ids[torch.randperm(len(ids), generator=torch.Generator().manual_seed(1))].cuda()
    a = Layer(1, len(ids), 8, 1, 72, 40, seed=5, idx=ids.view(1, -1, 1))
    with SC.SimComm(1) as c:
        for _ in range(3):
            a.run(c)
            torch.cuda.synchronize()
            a.check()


@pytest.mark.parametrize("group", [0, 32])
def test_addresses_that_are_not_aligned(group):
    a = Layer(2, 5, 4, 2, 64, 32, group, seed=9, offset=3)
    with SC.SimComm(2) as c:
        a.run(c)
        torch.cuda.synchronize()
    a.check()


def test_same_bits_on_every_call_in_place_and_alone():
    """Repeated calls, a residual that is the output, and one rank's tokens by themselves: the same bits."""
    a = Layer(4, 6, 16, 2, 128, 96, seed=2)
    with SC.SimComm(4) as c:
        a.run(c)
        torch.cuda.synchronize()
        first = [o.clone() for o in a.out]
        for _ in range(5):
            a.run(c)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(first, a.out))
        for o, r in zip(a.out, a.res):
            o.copy_(r)
        res, a.res = a.res, a.out
        a.run(c)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(first, a.out))
        a.res = res
    for rank in range(4):
        with SC.SimComm(4, rank=rank) as v:
            out = torch.zeros_like(a.out[rank])
            only = lambda t: [t[r] if r == rank else None for r in range(4)]  # noqa: E731
            v.moe_layer(only(a.x), only(a.idx), only(a.w), a.E, a.up, a.down,
                        [out if r == rank else None for r in range(4)], residual=only(a.res))
            torch.cuda.synchronize()
            a.check([first[r] if r != rank else out for r in range(4)])


def test_agrees_with_dispatch_experts_and_combine():
    """The layer in three steps: routes, rows moved to the experts' ranks, the experts in torch, the combine."""
    p, T, E, k, H, F = 4, 11, 8, 2, 64, 48
    a = Layer(p, T, E, k, H, F, seed=4)
    cap = p * T * k
    recv = [torch.zeros(cap, H, dtype=BF, device="cuda") for _ in range(p)]
    pos = [torch.empty(T, k, dtype=torch.int32, device="cuda") for _ in range(p)]
    ec = torch.empty(p, E, dtype=torch.int64, device="cuda")
    out = [torch.empty(T, H, dtype=BF, device="cuda") for _ in range(p)]
    with SC.SimComm(p) as c:
        c.moe_dispatch(a.x, a.idx, E, recv, route_pos=pos, expert_counts=ec)
        counts = ec.cpu()
        for j in range(p):
            at = 0
            for i in range(p):
                for e in range(j * (E // p), (j + 1) * (E // p)):
                    n = int(counts[i, e])
                    rows = recv[j][at:at + n].double() @ a.upd[e].t()
                    h = (torch.nn.functional.silu(rows[:, :F]) * rows[:, F:]).to(BF)
                    recv[j][at:at + n] = (h.double() @ a.downd[e].t()).to(BF)
                    at += n
        c.moe_combine(recv, a.idx, pos, a.w, E, out, residual=a.res)
        a.run(c)
        torch.cuda.synchronize()
    a.check()
    a.check(out, y_rounding=2.0 ** -8)


def test_nan_and_inf_stay_in_their_token():
    a = Layer(1, 6, 4, 2, 64, 32, seed=8, residual=False)
    a.x[0][2, 5] = float("nan")
    a.x[0][4, 0] = float("inf")
    with SC.SimComm(1) as c:
        a.run(c)
        torch.cuda.synchronize()
    out = a.out[0]
    assert bool(out[2].isnan().all()) and not bool(out[4].isfinite().all())
    for t in (0, 1, 3, 5):
        assert bool(out[t].isfinite().all())


@pytest.mark.parametrize("group", [0, 64])
def test_two_communicators_at_once(group):
    """Each kernel holds every SM it asks for until its grid barriers are passed; two of them take turns."""
    a, b = Layer(2, 12, 16, 4, 512, 1024, group, seed=31), Layer(4, 5, 8, 2, 1024, 640, group, seed=32)
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    with SC.SimComm(2) as ca, SC.SimComm(4) as cb:
        a.run(ca)
        b.run(cb)
        torch.cuda.synchronize()
        for _ in range(20):
            a.run(ca, stream=sa)
            b.run(cb, stream=sb)
        torch.cuda.synchronize()
        assert ca.async_error() == SC.OK and cb.async_error() == SC.OK
    a.check()
    b.check()


def test_graph_replays_with_new_tokens_and_calls_between():
    a = Layer(2, 4, 8, 2, 64, 32, seed=6)
    b = Layer(2, 40, 8, 4, 64, 32, seed=7)
    with SC.SimComm(2) as c:
        a.run(c)
        torch.cuda.synchronize()
        graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(graph, stream=s):
            a.run(c)
        b.run(c)  # needs more scratch: the graph keeps the old
        torch.cuda.synchronize()
        b.check()
        for seed in (11, 12):
            n = Layer(2, 4, 8, 2, 64, 32, seed=seed)
            for dst, src in zip(a.x + a.idx + a.w, n.x + n.idx + n.w):
                dst.copy_(src)
            graph.replay()
            torch.cuda.synchronize()
            a.check()
        del graph
    with SC.SimComm(2) as c:
        graph = torch.cuda.CUDAGraph()
        with pytest.raises(SC.SimCommError) as e:
            with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
                a.run(c)  # its scratch does not exist yet
        assert e.value.status == SC.UNSUPPORTED


def test_a_bad_expert_is_reported_and_nothing_is_written():
    a = Layer(2, 4, 8, 2, 64, 32, seed=6)
    with SC.SimComm(2) as c:
        for bad in (-1, 8, 2 ** 31 - 1):
            keep = int(a.idx[1][3, 1])
            a.idx[1][3, 1] = bad
            a.run(c)
            torch.cuda.synchronize()
            assert c.async_error() == SC.INVALID_ARG
            assert all(bool((o == 3.0).all()) for o in a.out)
            c.reset()
            a.idx[1][3, 1] = keep
        a.run(c)
        torch.cuda.synchronize()
        assert c.async_error() == SC.OK
        a.check()


def test_refusals():
    a = Layer(2, 4, 8, 2, 64, 32, 32)
    with SC.SimComm(2) as c:
        with pytest.raises(SC.SimCommError, match="overlap"):
            c.moe_layer(a.x, a.idx, a.w, 8, a.up, a.down, [a.x[0], a.out[1]], **a.scales())
        with pytest.raises(SC.SimCommError, match="residual"):
            c.moe_layer(a.x, a.idx, a.w, 8, a.up, a.down, a.out, residual=[a.out[1], a.out[0]], **a.scales())
        big = torch.zeros(1025, 2, dtype=torch.int32, device="cuda")
        with pytest.raises(SC.SimCommError, match="4096") as e:
            c.moe_layer([torch.zeros(1025, 64, dtype=BF, device="cuda")] * 2, [big] * 2, [big.float()] * 2, 8, a.up, a.down,
                        [torch.zeros(1025, 64, dtype=BF, device="cuda") for _ in range(2)], **a.scales())
        assert e.value.status == SC.UNSUPPORTED
        with pytest.raises(ValueError):
            c.moe_layer(a.x, a.idx, a.w, 8, a.up, a.down, a.out, up_scale=a.us)
        with pytest.raises(ValueError):
            c.moe_layer(a.x, a.idx, a.w, 16, a.up, a.down, a.out, **a.scales())
        with pytest.raises(TypeError):
            c.moe_layer(a.x, a.idx, a.w, 8, a.up, a.down, a.out)  # 4-bit weights without scales
        with pytest.raises(SC.SimCommError, match="16|aligned"):
            off = [torch.zeros(u.numel() + 1, dtype=torch.uint8, device="cuda")[1:].view(u.shape) for u in a.up]
            c.moe_layer(a.x, a.idx, a.w, 8, off, a.down, a.out, **a.scales())
        n = c.launch_count()
        c.moe_layer([t[:0] for t in a.x], [t[:0] for t in a.idx], [t[:0] for t in a.w], 8, a.up, a.down,
                    [t[:0] for t in a.out], **a.scales())
        assert c.launch_count() == n
