"""GPU tests of the root-mean-square norm with its AllReduce, residual and 8-bit rows, and of its gradient, against float64.

u = 2^-24. A sum of the ranks' p values and a residual errs by p u of the sum of their magnitudes (e_h). The sum of a
row's H squares runs in chains of at most 32 per thread and 12 joins (rows of more than 16,384 elements: H / 1024), each
term with one rounding, and what e_h does to it: r = 1 / sqrt(..) errs by half of that and 4 u. Each product rounds once
more. Outputs are off by half a step of their type beyond that: bf16 2^-8 of the value, fp32 2^-24, e4m3 2^-4 (2^-10 of the
scale where the value is subnormal).
"""
import math

import pytest
import torch

from collective_communication_primitives_b200 import simcomm as SC

pytestmark = pytest.mark.gpu
DT = {"fp32": torch.float32, "bf16": torch.bfloat16}
U = 2.0 ** -24
EPS = 1e-5
E4 = torch.float8_e4m3fn


def half(t):
    return torch.finfo(t).eps / 2


def guarded(p, *shape, dtype, offset=0, fill=3.0):
    """p buffers with a margin on both sides; (views, whether the margins are intact)."""
    n = math.prod(shape)
    raw = [torch.full((n + 64 + offset,), fill, device="cuda").to(dtype) for _ in range(p)]
    views = [b[32 + offset:32 + offset + n].view(shape) for b in raw]

    def intact():
        return all(bool((b[:32 + offset].float() == fill).all() and (b[32 + offset + n:].float() == fill).all()) for b in raw)
    return views, intact


class Norm:
    def __init__(self, p, T, H, dtype, residual=True, group=0, seed=0, offset=0, scale=1.0):
        g = torch.Generator("cuda").manual_seed(seed)
        rn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.p, self.T, self.H, self.dt, self.group = p, T, H, DT[dtype], group
        new = lambda *s, t=self.dt, o=offset: guarded(p, *s, dtype=t, offset=o)  # noqa: E731
        self.x = new(T, H)[0]
        for x in self.x:
            x.copy_(scale * rn(T, H))
        self.res = (2 * scale * rn(T, H)).to(self.dt) if residual else None
        self.w = (1 + 0.3 * rn(H)).to(self.dt)
        self.total, self.ok_total = new(T, H)
        self.y, self.ok_y = new(T, H)
        if group:
            self.q, self.ok_q = guarded(p, T, H, dtype=torch.uint8, offset=offset)
            self.scale, self.ok_scale = guarded(p, T, H // group, dtype=torch.float32)
        else:
            self.q = self.scale = None

    def run(self, c, **more):
        c.rmsnorm(self.x, self.w, EPS, out=self.y, residual=self.res, total=self.total, q=self.q, scale=self.scale, **more)

    def exact(self, res=None):
        res = self.res if res is None else res
        parts = [x.double() for x in self.x] + ([] if res is None else [res.double()])
        h, mag = sum(parts), sum(v.abs() for v in parts)
        e_h = self.p * U * mag
        ms = h.square().mean(1, keepdim=True)
        r = 1 / torch.sqrt(ms + EPS)
        chain = 32 + 12 if self.H <= 16384 else self.H / 1024 + 12
        e_r = 0.5 * ((chain + 1) * U + 2 * (h.abs() * e_h).mean(1, keepdim=True) / (ms + EPS)) + 4 * U
        y = h * r * self.w.double()
        e_y = self.w.double().abs() * r * e_h + y.abs() * (e_r + 3 * U)
        return h, e_h, y, e_y

    def check(self, res=None):
        h, e_h, y, e_y = self.exact(res)
        assert self.ok_total() and self.ok_y()
        for r in range(self.p):
            assert bool(((self.total[r].double() - h).abs() <= e_h + half(self.dt) * (h.abs() + e_h)).all())
            assert bool(((self.y[r].double() - y).abs() <= e_y + half(self.dt) * (y.abs() + e_y)).all())
        if not self.group:
            return
        assert self.ok_q() and self.ok_scale()
        part = lambda t: t.view(self.T, -1, self.group)  # noqa: E731
        want = part(y).abs().amax(2) / 448
        off = part(e_y).amax(2) / 448 + 2 * U * want
        for r in range(self.p):
            s = self.scale[r].double()
            assert bool(((s - want).abs() <= off).all())
            got = self.q[r].view(E4).double() * s.repeat_interleave(self.group, 1)
            step = s.repeat_interleave(self.group, 1)
            assert bool(((got - y).abs() <= e_y + half(E4) * (y.abs() + e_y) + 2.0 ** -10 * step + 2 * U * y.abs()).all())
            assert bool((part(self.q[r].view(E4).float()).abs().amax(2)[want > 0] == 448).all())


SHAPES = [(1, 1, 1), (1, 3, 7), (2, 5, 64), (3, 2, 129), (4, 33, 1001), (8, 1, 4096), (8, 17, 4096), (2, 9, 8200),
          (1, 3, 16384), (2, 2, 16392), (1, 2, 40000), (64, 2, 96), (8, 300, 256), (5, 4, 8191)]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("p,T,H", SHAPES)
def test_norm(p, T, H, dtype):
    with SC.SimComm(p) as c:
        for residual in (True, False):
            a = Norm(p, T, H, dtype, residual, seed=T)
            a.run(c)
            torch.cuda.synchronize()
            assert c.async_error() == SC.OK
            a.check()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("p,T,H,group", [(1, 3, 32, 32), (2, 5, 4096, 32), (8, 4, 4096, 64), (4, 7, 4096, 128), (2, 3, 4096, 256),
                                         (2, 3, 4096, 1024), (2, 3, 4096, 4096), (4, 5, 1001, 1001), (1, 2, 40960, 128),
                                         (1, 2, 40960, 40960), (3, 9, 96, 32), (1, 1, 8192, 2048), (2, 70, 2048, 512), (1, 4, 7, 7),
                                         (2, 3, 16384, 8192), (1, 2, 32768, 16384)])
def test_8_bit_rows(p, T, H, group, dtype):
    with SC.SimComm(p) as c:
        a = Norm(p, T, H, dtype, True, group, seed=H)
        a.run(c)
        torch.cuda.synchronize()
        a.check()
        # 8 bits alone, no other output
        q, s = [torch.empty_like(v) for v in a.q], [torch.empty_like(v) for v in a.scale]
        c.rmsnorm(a.x, a.w, EPS, residual=a.res, q=[v.view(E4) for v in q], scale=s)
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(q + s, a.q + a.scale))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("offset", [1, 4])
def test_unaligned_rows(offset, dtype):
    with SC.SimComm(2) as c:
        for H, group in ((256, 32), (4096, 128), (8192, 64), (96, 96)):
            a = Norm(2, 5, H, dtype, True, group, offset=offset)
            a.run(c)
            torch.cuda.synchronize()
            a.check()


def test_outputs_alone_and_the_sum_alone():
    with SC.SimComm(4) as c:
        a = Norm(4, 6, 512, "bf16", seed=1)
        a.run(c)
        only = [torch.empty_like(v) for v in a.total]
        c.rmsnorm(a.x, a.w, EPS, residual=a.res, total=only)
        y = [torch.empty_like(v) for v in a.y]
        c.rmsnorm(a.x, a.w, EPS, out=y, residual=a.res)
        torch.cuda.synchronize()
        a.check()
        assert all(torch.equal(u, v) for u, v in zip(only + y, a.total + a.y))


@pytest.mark.parametrize("H", [512, 1001, 40000])
def test_residual_in_place(H):
    with SC.SimComm(3) as c:
        a = Norm(3, 4, H, "bf16", seed=2)
        res = a.res.clone()
        a.total[1].copy_(a.res)
        c.rmsnorm(a.x, a.w, EPS, out=a.y, residual=a.total[1], total=a.total)
        torch.cuda.synchronize()
        a.check(res)


@pytest.mark.parametrize("H", [64, 1001, 20000])
def test_rows_with_zeros_infinities_nan_and_huge_values(H):
    p = 2
    x = [torch.randn(7, H, device="cuda") for _ in range(p)]
    for v in x:
        v[0] = 0
        v[3] *= 1e25          # squares pass fp32
        v[5] *= 1e-25         # squares vanish beside eps
    x[0][1, 3], x[1][2, 5] = math.nan, math.inf
    x[0][6] = 3e38 / p
    x[1][6] = 0
    w = torch.randn(H, device="cuda")
    new = lambda *s, t=torch.float32: [torch.empty(*s, dtype=t, device="cuda") for _ in range(p)]  # noqa: E731
    total, y, q, s = new(7, H), new(7, H), new(7, H, t=E4), new(7, 1)
    with SC.SimComm(p) as c:
        c.rmsnorm(x, w, EPS, total=total, out=y, q=q, scale=s)
        torch.cuda.synchronize()
    h = sum(v.double() for v in x)
    want = h / torch.sqrt(h.square().mean(1, keepdim=True) + EPS) * w.double()
    got = y[1].double()
    assert bool((got[0] == 0).all()) and bool((q[0][0].float() == 0).all()) and float(s[0][0]) == 0
    assert bool(got[1].isnan().all()) and bool(s[1][1].isnan().all()) and bool(q[1][1].float().isnan().all())
    assert bool(got[2, 5].isnan()) and bool((got[2, torch.arange(H, device="cuda") != 5] == 0).all())
    for t in (3, 4, 5, 6):  # the bound of check() for two ranks, its sum of squares in chains of H / 1024 at most
        bound = (2 + 64 + H / 1024) * U * want[t].abs() + w.double().abs() * 2 * U * sum(v[t].double().abs() for v in x) \
            / torch.sqrt(h[t].square().mean() + EPS)
        assert bool(((got[t] - want[t]).abs() <= bound).all()), t


class Back:
    def __init__(self, p, T, H, dtype, past=True, seed=0, offset=0, scale=1.0):
        g = torch.Generator("cuda").manual_seed(seed)
        rn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.p, self.T, self.H, self.dt = p, T, H, DT[dtype]
        self.gy = guarded(p, T, H, dtype=self.dt, offset=offset)[0]
        for v in self.gy:
            v.copy_(rn(T, H))
        self.h = (scale * (rn(T, H) + 0.3)).to(self.dt)
        self.w = (1 + 0.3 * rn(H)).to(self.dt)
        self.past = rn(T, H).to(self.dt) if past else None
        self.gx, self.ok_x = guarded(p, T, H, dtype=self.dt, offset=offset)
        self.gw, self.ok_w = guarded(p, H, dtype=torch.float32)

    def run(self, c, weight=True, **more):
        c.rmsnorm_backward(self.gy, self.h, self.w, EPS, self.gx, grad_total=self.past, grad_weight=self.gw if weight else None,
                           **more)

    def check(self, weight=True, sms=148):
        h, w = self.h.double(), self.w.double()
        g = sum(v.double() for v in self.gy)
        e_g = self.p * U * sum(v.double().abs() for v in self.gy)
        chain = 32 + 12 if self.H <= 16384 else self.H / 1024 + 12
        r = 1 / torch.sqrt(h.square().mean(1, keepdim=True) + EPS)
        u = h * r
        e_u = u.abs() * ((chain + 10) * U)
        along = (w * g * u).mean(1, keepdim=True)
        e_a = ((w * g * u).abs() * ((2 * chain + 14) * U) + (w * u).abs() * e_g).mean(1, keepdim=True)
        want = r * (w * g - u * along)
        part = (w * g).abs() + (u * along).abs()
        err = r * (w.abs() * e_g + e_u * along.abs() + u.abs() * e_a + part * ((chain + 8) * U))
        if self.past is not None:
            want = want + self.past.double()
            err = err + U * (want.abs() + self.past.double().abs())
        dw = (g * u).sum(0)
        rows = -(-self.T // min(self.T, 2 * sms))
        e_w = (u.abs() * e_g + g.abs() * e_u + (g * u).abs() * (rows + 2 * sms / 8 + 12) * U).sum(0) + U * dw.abs()
        assert self.ok_x() and self.ok_w()
        for k in range(self.p):
            assert bool(((self.gx[k].double() - want).abs() <= err + half(self.dt) * (want.abs() + err)).all())
            if weight:
                assert bool(((self.gw[k].double() - dw).abs() <= e_w).all())


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("p,T,H", SHAPES + [(2, 1000, 264), (1, 700, 33)])
def test_gradient(p, T, H, dtype):
    with SC.SimComm(p) as c:
        for past in (True, False):
            a = Back(p, T, H, dtype, past, seed=T)
            a.run(c)
            torch.cuda.synchronize()
            assert c.async_error() == SC.OK
            a.check()
            first = [v.clone() for v in a.gx + a.gw]
            a.run(c)
            torch.cuda.synchronize()
            assert all(torch.equal(u, v) for u, v in zip(first, a.gx + a.gw))
        a.run(c, weight=False)
        torch.cuda.synchronize()
        a.check(weight=False)


@pytest.mark.parametrize("offset", [1, 4])
def test_gradient_of_unaligned_rows(offset):
    with SC.SimComm(2) as c:
        for dtype in ("fp32", "bf16"):
            a = Back(2, 37, 512, dtype, offset=offset)
            a.run(c)
            torch.cuda.synchronize()
            a.check()


@pytest.mark.parametrize("H", [64, 1001, 20000])
def test_gradient_at_huge_rows(H):
    """Rows whose squares pass fp32: u is what it is for the row scaled down, the gradient as much smaller."""
    with SC.SimComm(1) as c:
        a = Back(1, 3, H, "fp32", past=False, seed=5)
        b = Back(1, 3, H, "fp32", past=False, seed=5)
        b.h *= 2.0 ** 80
        a.h *= 2.0 ** 20  # eps is nothing beside either
        a.run(c)
        b.run(c)
        torch.cuda.synchronize()
    # the same operations on numbers scaled by powers of two, but for eps, which moves r by eps / (2 mean h^2) at most
    tiny = 2 * U
    assert bool(((a.gw[0] - b.gw[0]).abs() <= 3 * 16 * tiny * (a.gy[0] * 8).abs().sum(0)).all())
    assert bool((b.gx[0].abs() > 0).any()) and bool(b.gx[0].isfinite().all())
    rel = (b.gx[0].double() * 2.0 ** 60 - a.gx[0].double()).norm() / a.gx[0].double().norm()
    assert float(rel) < 1e-5


def test_gradient_against_differences():
    """(f(h + d) - f(h - d)) / 2 in float64 along random directions, f the loss sum(gy y) through the norm."""
    p, T, H = 2, 4, 96
    a = Back(p, T, H, "fp32", past=True, seed=11)
    with SC.SimComm(p) as c:
        a.run(c)
        torch.cuda.synchronize()
    g, w, h, past = sum(v.double() for v in a.gy), a.w.double(), a.h.double(), a.past.double()
    f = lambda h, w: float((g * h / torch.sqrt(h.square().mean(1, keepdim=True) + EPS) * w).sum() + (past * h).sum())  # noqa: E731
    for seed in range(3):
        d = torch.randn(T, H, dtype=torch.float64, device="cuda", generator=torch.Generator("cuda").manual_seed(seed))
        step = 1e-4
        num = (f(h + step * d, w) - f(h - step * d, w)) / (2 * step)
        scale = float((a.gx[0].double() * d).abs().sum())
        assert abs(num - float((a.gx[0].double() * d).sum())) <= 1e-5 * scale
        dw = d[0]
        num = (f(h, w + step * dw) - f(h, w - step * dw)) / (2 * step)
        assert abs(num - float((a.gw[0].double() * dw).sum())) <= 1e-5 * float((a.gw[0].double() * dw).abs().sum())


def test_forward_and_backward_as_a_graph_on_another_stream():
    p = 4
    a, b = Norm(p, 64, 1024, "bf16", True, 128, seed=3), Back(p, 64, 1024, "bf16", seed=4)
    with SC.SimComm(p) as c:
        stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        stream.wait_stream(torch.cuda.current_stream())
        a.run(c, stream=stream)
        b.run(c, stream=stream)
        stream.synchronize()
        a.check()
        b.check()
        with torch.cuda.graph(graph, stream=stream):
            a.run(c)
            b.run(c)
        for x in a.x + b.gy:
            x.copy_(torch.randn_like(x))
        for t in a.total + a.y + b.gx + b.gw:
            t.fill_(9)
        for _ in range(2):
            graph.replay()
        torch.cuda.synchronize()
        assert c.async_error() == SC.OK
        a.check()
        b.check()
        del graph


def test_refusals():
    with SC.SimComm(2) as c:
        a = Norm(2, 4, 96, "fp32", group=32)
        for eps in (0.0, -1.0, math.nan, math.inf, 1e-39):
            with pytest.raises(SC.SimCommError, match="eps"):
                c.rmsnorm(a.x, a.w, eps, out=a.y)
        with pytest.raises(SC.SimCommError, match="no output"):
            c.rmsnorm(a.x, a.w, EPS)
        with pytest.raises(SC.SimCommError, match="group"):
            c.rmsnorm(a.x, a.w, EPS, q=a.q, scale=[torch.empty(4, 2, device="cuda") for _ in range(2)])  # groups of 48
        with pytest.raises(SC.SimCommError, match="overlap"):
            c.rmsnorm(a.x, a.w, EPS, out=a.x)
        with pytest.raises(SC.SimCommError, match="overlap"):
            c.rmsnorm(a.x, a.w, EPS, out=a.y, total=a.y)
        with pytest.raises(SC.SimCommError, match="residual"):
            c.rmsnorm(a.x, a.w, EPS, out=a.y, residual=a.y[0])
        with pytest.raises(SC.SimCommError, match="UNSUPPORTED"):
            i = [torch.zeros(4, 8, dtype=torch.int32, device="cuda") for _ in range(4)]
            c.rmsnorm(i[:2], torch.zeros(8, dtype=torch.int32, device="cuda"), EPS, out=i[2:])
        b = Back(2, 4, 96, "fp32")
        with pytest.raises(SC.SimCommError, match="overlap"):
            c.rmsnorm_backward(b.gy, b.h, b.w, EPS, b.gy)
        with pytest.raises(SC.SimCommError, match="overlap"):
            c.rmsnorm_backward(b.gy, b.h, b.w, EPS, [b.gx[0], b.h])
        # no rows: nothing is done
        none = [torch.empty(0, 96, device="cuda") for _ in range(2)]
        before = c.launch_count()
        c.rmsnorm(none, a.w, EPS, out=none)
        c.rmsnorm_backward(none, none[0], a.w, EPS, none, grad_weight=b.gw)
        assert c.launch_count() == before
        torch.cuda.synchronize()
        assert bool((b.gw[0] == 3).all())
        assert c.async_error() == SC.OK
