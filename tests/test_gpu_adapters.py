"""GPU tests of the low-rank adapters against float64.

Whole-number inputs make every step exact (sums below 2^24, A x below 2^16, which two bf16 parts hold), so the result must be
the exact one, rounded once. For others: a matrix instruction adds 16 products and a sum, each cut below the last bit of
the largest: 17 * 2^-23 of the magnitudes at most, K / 16 instructions for A x and R / 8 for B (A x); the two parts of A x lose
2^-16 of it; the joins of at most 8 warps and 16 parts, the scale and the base round once each.
"""
import math

import pytest
import torch

from collective_communication_primitives_b200 import simcomm as SC

pytestmark = pytest.mark.gpu
DT = {"fp32": torch.float32, "bf16": torch.bfloat16}
BF = torch.bfloat16


class Adapted:
    def __init__(self, p, T, N, K, S, R, parallel, base="fp32", out="fp32", seed=0, whole=True, runs=1, ranks=None, scale=True,
                 offset=0):
        g = torch.Generator("cuda").manual_seed(seed)
        self.p, self.T, self.N, self.K, self.S, self.R, self.parallel = p, T, N, K, S, R, parallel
        self.row, self.bt, self.ot = parallel == "row", base and DT[base], DT[out]
        if whole:
            num = lambda *s: torch.randint(-3, 4, s, generator=g, device="cuda").float()  # noqa: E731
        else:
            num = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.X, self.A, self.B = num(T, K).to(BF), num(S, R, K).to(BF), num(S, N, R).to(BF)
        self.base64 = num(T, N).to(self.bt) if base else None
        pick = torch.randint(-1, S, (-(-T // runs),), generator=g, device="cuda", dtype=torch.int32)
        self.ad = pick.repeat_interleave(runs)[:T].contiguous()
        self.rk = None if ranks is None else torch.tensor(ranks, dtype=torch.int32, device="cuda")
        self.sc = (2.0 ** torch.randint(-2, 2, (S,), generator=g, device="cuda")) if scale else None

        def place(t):  # at an offset, with a margin
            b = torch.full((t.numel() + offset + 16,), 7.0, device="cuda").to(t.dtype)
            v = b[offset:offset + t.numel()].view(t.shape)
            v.copy_(t)
            return v
        cut = lambda t, d: [place(v) for v in t.chunk(p, d)]  # noqa: E731
        every = lambda t: [place(t) for _ in range(p)]  # noqa: E731
        if self.row:
            self.x, self.a, self.b = cut(self.X, 1), cut(self.A, 2), every(self.B)
            self.base = every(self.base64) if base else None
        else:
            self.x, self.a, self.b = every(self.X), every(self.A), cut(self.B, 1)
            self.base = cut(self.base64, 1) if base else None
        n = N if self.row else N // p
        self.raw = [torch.full((T * n + offset + 64,), 5.0, device="cuda").to(self.ot) for _ in range(p)]
        self.out = [b[32 + offset:32 + offset + T * n].view(T, n) for b in self.raw]
        self.offset = offset

    def run(self, c, **more):
        c.adapters(self.x, self.ad, self.a, self.b, self.out, base=self.base, rank=self.rk, scale=self.sc,
                   parallel=self.parallel, **more)

    def exact(self):
        """(result, sum of magnitudes that the error bounds refer to)"""
        y = torch.zeros(self.T, self.N, dtype=torch.float64, device="cuda")
        mag = torch.zeros_like(y)
        for e in range(self.S):
            t = torch.nonzero(self.ad == e)[:, 0]
            r = self.R if self.rk is None else int(self.rk[e])
            x, a, b = self.X[t].double(), self.A[e, :r].double(), self.B[e, :, :r].double()
            s = 1.0 if self.sc is None else float(self.sc[e])
            u, um = x @ a.t(), x.abs() @ a.abs().t()
            y[t] += s * (u @ b.t())
            mag[t] += s * ((self.K / 16 + self.p) * 17 * 2.0 ** -23 + 26 * 2.0 ** -24) * (um @ b.abs().t())
            mag[t] += s * ((r / 8 + 1) * 17 * 2.0 ** -23 + 2.0 ** -16 + 2.0 ** -23) * (u.abs() @ b.abs().t())
        if self.base64 is not None:
            y += self.base64.double()
        return y, mag + 2.0 ** -24 * y.abs()

    def check(self, exact):
        y, err = self.exact()
        parts = [y] * self.p if self.row else list(y.chunk(self.p, 1))
        errs = [err] * self.p if self.row else list(err.chunk(self.p, 1))
        h = torch.finfo(self.ot).eps / 2
        for got, want, e, raw in zip(self.out, parts, errs, self.raw):
            if exact:
                assert torch.equal(got, want.float().to(self.ot))
            else:
                assert bool(((got.double() - want).abs() <= e + h * (want.abs() + e)).all())
            edge = 32 + self.offset
            assert bool((raw[:edge].float() == 5).all()) and bool((raw[edge + got.numel():].float() == 5).all())


SIZES = [(1, 1, 8, 8, 1, 1), (2, 3, 16, 32, 2, 4), (4, 8, 64, 128, 3, 8), (2, 9, 40, 200, 5, 16), (8, 32, 256, 1024, 40, 16),
         (1, 64, 130, 72, 7, 17), (2, 65, 66, 48, 4, 20), (4, 100, 128, 256, 9, 64), (2, 300, 24, 40, 2, 128),
         (1, 33, 20, 64, 3, 256), (2, 515, 136, 96, 6, 32), (1, 1100, 17, 33, 3, 5), (8, 70, 8, 24, 2, 100)]


@pytest.mark.parametrize("parallel", ["row", "column"])
@pytest.mark.parametrize("p,T,N,K,S,R", SIZES)
def test_whole_numbers_are_exact(p, T, N, K, S, R, parallel):
    with SC.SimComm(p) as c:
        for base, out, runs, scale in (("fp32", "bf16", 1, True), ("bf16", "bf16", 20, False), (None, "fp32", 7, True),
                                       ("bf16", "fp32", 1, False)):
            a = Adapted(p, T, N, K, S, R, parallel, base, out, seed=T + N, runs=runs, scale=scale)
            a.run(c)
            torch.cuda.synchronize()
            assert c.async_error() == SC.OK
            a.check(exact=True)


@pytest.mark.parametrize("parallel", ["row", "column"])
@pytest.mark.parametrize("p,T,N,K,S,R", [(2, 5, 64, 256, 3, 16), (4, 200, 256, 512, 8, 24), (8, 600, 128, 1024, 3, 64)])
def test_random_numbers(p, T, N, K, S, R, parallel):
    with SC.SimComm(p) as c:
        a = Adapted(p, T, N, K, S, R, parallel, seed=T, whole=False, runs=11)
        a.run(c)
        torch.cuda.synchronize()
        a.check(exact=False)


@pytest.mark.parametrize("parallel", ["row", "column"])
@pytest.mark.parametrize("T", [6, 90])
def test_adapters_of_different_ranks(T, parallel):
    """What lies behind an adapter's own rank is not read as numbers: here NaN; a rank of 0 adds nothing."""
    with SC.SimComm(2) as c:
        a = Adapted(2, T, 36, 64, 6, 40, parallel, seed=T, ranks=[0, 1, 15, 17, 39, 40])
        for r in range(2):
            for e, k in enumerate(a.rk.tolist()):
                a.a[r][e, k:] = math.nan
                a.b[r][e, :, k:] = math.nan
        a.run(c)
        torch.cuda.synchronize()
        a.check(exact=True)


@pytest.mark.parametrize("parallel", ["row", "column"])
@pytest.mark.parametrize("offset", [1, 2, 4])
def test_unaligned_buffers(offset, parallel):
    with SC.SimComm(2) as c:
        for T in (5, 80):
            a = Adapted(2, T, 32, 64, 3, 16, parallel, "bf16", "bf16", seed=T, offset=offset)
            a.run(c)
            torch.cuda.synchronize()
            a.check(exact=True)


@pytest.mark.parametrize("parallel", ["row", "column"])
def test_in_place_and_no_adapter_at_all(parallel):
    with SC.SimComm(2) as c:
        a = Adapted(2, 40, 64, 64, 4, 8, parallel, "fp32", "fp32", seed=1)
        for o, b in zip(a.out, a.base):
            o.copy_(b)
        a.base = a.out
        a.run(c)
        torch.cuda.synchronize()
        a.check(exact=True)
        a = Adapted(2, 40, 64, 64, 4, 8, parallel, "bf16", "fp32", seed=1)
        a.ad.fill_(-1)
        a.run(c)
        torch.cuda.synchronize()
        a.check(exact=True)


def test_infinities_and_nan_stay_with_their_tokens():
    with SC.SimComm(1) as c:
        a = Adapted(1, 20, 16, 32, 2, 8, "row", seed=3)
        a.ad.copy_(torch.tensor([0, 1] * 10, dtype=torch.int32))
        a.x[0][3, 5] = math.nan
        a.x[0][8, 1] = math.inf
        a.a[0][0, :, 1] = 1
        a.b[0][0] = 1
        a.run(c)
        torch.cuda.synchronize()
        got = a.out[0]
        assert bool(got[3].isnan().all()) and bool((got[8] == math.inf).all())
        a.X, a.A, a.B = a.x[0], a.a[0], a.b[0]
        keep = torch.tensor([t not in (3, 8) for t in range(20)], device="cuda")
        y, _ = a.exact()
        assert torch.equal(got[keep], y[keep].float())


def test_a_tokens_result_does_not_depend_on_the_others():
    with SC.SimComm(2) as c:
        for T in (40, 200, 700):
            a = Adapted(2, T, 64, 512, 5, 16, "row", seed=T, whole=False)
            a.run(c)
            first = [o.clone() for o in a.out]
            keep = torch.rand(T, device="cuda", generator=torch.Generator("cuda").manual_seed(1)) < 0.5
            a.ad[~keep] = torch.roll(a.ad, 1)[~keep]
            a.run(c)
            torch.cuda.synchronize()
            assert all(torch.equal(u[keep], v[keep]) for u, v in zip(first, a.out))


def test_as_a_graph_with_other_adapters_and_a_second_graph():
    p = 2
    a, b = (Adapted(p, T, 64, 128, 5, 16, "row", seed=T) for T in (12, 130))
    with SC.SimComm(p) as c:
        stream, graphs = torch.cuda.Stream(), []
        for s in (b, a):
            s.run(c)
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=stream):
                s.run(c)
            graphs.append(graph)
        for s in (a, b):
            s.ad.copy_(torch.roll(s.ad, 3))
            for o in s.out:
                o.fill_(0)
        for _ in range(2):
            for graph in graphs:
                graph.replay()
        torch.cuda.synchronize()
        a.check(exact=True)
        b.check(exact=True)
        del graph, graphs


def test_refusals_and_bad_indices():
    with SC.SimComm(2) as c:
        a = Adapted(2, 6, 32, 64, 3, 16, "row", "bf16", "fp32")
        with pytest.raises(SC.SimCommError, match="overlap"):
            c.adapters(a.x, a.ad, a.a, a.b, a.out, base=a.out[::-1])
        with pytest.raises(SC.SimCommError, match="max_rank"):
            big = [torch.zeros(1, 257, 32, dtype=BF, device="cuda")] * 2
            c.adapters(a.x, a.ad, big, [torch.zeros(1, 32, 257, dtype=BF, device="cuda")] * 2, a.out)
        with pytest.raises(SC.SimCommError, match="UNSUPPORTED"):
            i = [torch.zeros(6, 32, dtype=torch.int32, device="cuda") for _ in range(2)]
            c.adapters(a.x, a.ad, a.a, a.b, i)
        before = c.launch_count()
        none = [t[:0] for t in a.x]
        c.adapters(none, a.ad[:0], a.a, a.b, [o[:0] for o in a.out])
        assert c.launch_count() == before
        for value in (3, -2):
            a.ad[2] = value
            a.run(c)
            torch.cuda.synchronize()
            assert c.async_error() == SC.INVALID_ARG
            with pytest.raises(SC.SimCommError):
                a.run(c)
            c.reset()
        a.ad[2] = 0
        for value in (17, -1):
            a.rk = torch.tensor([value, 2, 3], dtype=torch.int32, device="cuda")
            a.run(c)
            torch.cuda.synchronize()
            assert c.async_error() == SC.INVALID_ARG
            c.reset()
        a.rk = None
        a.run(c)
        torch.cuda.synchronize()
        a.check(exact=True)
