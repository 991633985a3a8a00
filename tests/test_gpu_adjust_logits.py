"""GPU tests of penalties, biases and masks on sharded scores against float64.

Scores that no rule touches must keep their bits; masked ones are -inf. Of the others each of at most five operations in
fp32 rounds by 2^-24 of the largest number that occurs, and the result by half a step of its type.
"""
import math

import pytest
import torch

from collective_communication_primitives_b200 import simcomm as SC
from test_gpu_logprobs import shards

pytestmark = pytest.mark.gpu
DT = {"fp32": torch.float32, "bf16": torch.bfloat16}
I32 = torch.int32


class Adjust:
    def __init__(self, p, R, V, dtype, L=0, bias=0, masked=False, seed=0, ld_extra=0, offset=0, prompt=True, own_mask=False,
                 ld_history=None):
        g = torch.Generator("cuda").manual_seed(seed)
        rand = lambda *s: torch.rand(*s, generator=g, device="cuda")  # noqa: E731
        ints = lambda lo, hi, s: torch.randint(lo, hi, s, generator=g, device="cuda", dtype=I32)  # noqa: E731
        self.p, self.R, self.V, self.ld_extra, self.offset = p, R, V, ld_extra, offset
        x = (3 * torch.randn(R, V, generator=g, device="cuda")).to(DT[dtype])
        x[rand(R, V) < 0.02] = -math.inf
        x[rand(R, V) < 0.02] = 0
        self.x = x
        self.logits = shards(x, p, ld_extra, offset)
        self.out = shards(torch.full_like(x, 4), p, ld_extra, offset, fill=11.0)
        self.kw = {}
        if L:
            h = (V * rand(R, L) ** 3).int().clamp_(max=V - 1)
            h[rand(R, L) < 0.05] = -1
            n = ints(0, L + 1, (R,))
            n[0] = L
            if R > 1:
                n[1] = 0
            self.kw |= {"history": h, "history_len": n, "repetition": 0.5 + rand(R), "frequency": rand(R) - 0.3, "presence": rand(R)}
            if prompt:
                self.kw["prompt_len"] = (n * rand(R)).int()
        if bias:
            n = ints(0, bias + 1, (R,))
            n[R // 2] = bias
            start = torch.zeros(R + 1, dtype=I32, device="cuda")
            start[1:] = n.cumsum(0)
            total = int(start[-1]) + 3  # entries behind the last row's
            self.kw |= {"bias_start": start, "bias_token": ints(-1, V, (total,)), "bias_value": 2 * torch.randn(total, generator=g, device="cuda")}
        if masked:
            words = -(-V // 32) + 2
            M = R if own_mask else max(1, R // 3)
            self.kw["mask"] = ints(-2 ** 31, 2 ** 31 - 1, (M, words))
            if M > 1:
                self.kw["mask"][1] = 0
            if not own_mask:
                self.kw["mask_row"] = ints(-1, M, (R,))

    def run(self, c, in_place=False, **more):
        c.adjust_logits(self.logits, self.V, self.logits if in_place else self.out, **self.kw, **more)

    def want(self):
        """(float64 result, which scores a rule touches, bound of the fp32 steps)"""
        x, k = self.x.double(), self.kw
        touched = torch.zeros_like(x, dtype=torch.bool)
        big = torch.where(x.isfinite(), x.abs(), 0)
        if "history" in k:
            for t in range(self.R):
                n = int(k["history_len"][t])
                m = int(k["prompt_len"][t]) if "prompt_len" in k else 0
                ids = k["history"][t, :n].long()
                new = ids[m:][ids[m:] >= 0]
                ids = torch.unique(ids[ids >= 0])
                touched[t, ids] = True
                if "repetition" in k:
                    rp = k["repetition"][t].double()
                    x[t, ids] = torch.where(x[t, ids] > 0, x[t, ids] / rp, x[t, ids] * rp)
                    big[t, ids] = torch.maximum(big[t, ids], torch.where(x[t, ids].isfinite(), x[t, ids].abs(), 0))
                ids, times = torch.unique(new, return_counts=True)
                f = k["frequency"][t].double() if "frequency" in k else 0.0
                q = k["presence"][t].double() if "presence" in k else 0.0
                x[t, ids] -= f * times + q
                big[t, ids] += abs(f) * times + abs(q)
        if "bias_start" in k:
            for t in range(self.R):
                last = {}
                for i in range(int(k["bias_start"][t]), int(k["bias_start"][t + 1])):
                    last[int(k["bias_token"][i])] = float(k["bias_value"][i])
                for v, b in last.items():
                    if v >= 0:
                        x[t, v] += b
                        touched[t, v] = True
                        big[t, v] += abs(b)
        ok = torch.ones_like(touched)
        if "mask" in k:
            bits = torch.stack([(k["mask"].long() >> i) & 1 for i in range(32)], 2).flatten(1)[:, :self.V] != 0
            row = k.get("mask_row", torch.arange(self.R, device="cuda"))
            ok = bits[row.clamp(min=0).long()] | (row < 0)[:, None]
        return torch.where(ok, x, -math.inf), touched, ok, 5 * 2.0 ** -24 * big

    def check(self, got=None):
        want, touched, ok, err = self.want()
        got = self.out if got is None else got
        m = -(-self.V // self.p)
        full = torch.cat([v for v in got], 1)[:, :self.V]
        keep = ok & ~touched
        raw = torch.int32 if full.dtype == torch.float32 else torch.int16
        assert torch.equal(full.contiguous().view(raw)[keep], self.x.view(raw)[keep])
        assert bool((full[~ok] == -math.inf).all())
        at = ok & touched
        half = torch.finfo(full.dtype).eps / 2
        g, w, e = full[at].double(), want[at], err[at]
        fin = w.isfinite()
        assert torch.equal(g[~fin], w[~fin])
        assert bool(((g - w).abs()[fin] <= (e + half * (w.abs() + e))[fin]).all())
        for r in range(self.p):  # padding columns are not written
            own = max(0, min(m, self.V - r * m))
            assert bool((got[r][:, own:].float() == (11 if got is self.out else 77)).all())


SIZES = [(1, 1, 1), (2, 3, 37), (4, 5, 1001), (8, 2, 4096), (3, 7, 20011), (8, 9, 32), (1, 2, 70000), (8, 3, 131072), (64, 2, 200)]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("p,R,V", SIZES)
def test_every_rule(p, R, V, dtype):
    with SC.SimComm(p) as c:
        for L, bias, masked in ((50, 0, False), (0, 9, False), (0, 0, True), (333, 40, True), (1, 1, True)):
            a = Adjust(p, R, V, dtype, L, bias, masked, seed=V + L)
            a.run(c)
            torch.cuda.synchronize()
            assert c.async_error() == SC.OK
            a.check()
            assert torch.equal(torch.cat(a.logits, 1)[:, :V].view(torch.int8), a.x.view(torch.int8))
            a.run(c, in_place=True)
            torch.cuda.synchronize()
            a.check(a.logits)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("ld_extra,offset", [(1, 0), (3, 1), (0, 5), (8, 8)])
def test_rows_at_any_distance(ld_extra, offset, dtype):
    with SC.SimComm(3) as c:
        a = Adjust(3, 6, 5003, dtype, 77, 12, True, seed=1, ld_extra=ld_extra, offset=offset)
        a.run(c)
        torch.cuda.synchronize()
        a.check()
        # aligned in, unaligned out
        b = Adjust(3, 6, 5003, dtype, 77, 12, True, seed=1, ld_extra=ld_extra)
        b.out = a.out
        b.run(c)
        torch.cuda.synchronize()
        b.check()
        a.run(c, in_place=True)
        torch.cuda.synchronize()
        a.check(a.logits)


@pytest.mark.parametrize("L", [5000, 40000])
def test_long_histories_and_rows_of_one_token(L):
    with SC.SimComm(2) as c:
        a = Adjust(2, 3, 30000, "fp32", L, seed=2)
        a.kw["history"][0] = 12345  # one token, all the time
        a.kw["frequency"].fill_(2.0 ** -10)
        a.run(c)
        torch.cuda.synchronize()
        a.check()


def test_rules_one_by_one():
    with SC.SimComm(2) as c:
        for leave in (("repetition",), ("frequency",), ("presence",), ("repetition", "presence"), ("frequency", "presence", "prompt_len")):
            a = Adjust(2, 4, 500, "fp32", 60, seed=3)
            for k in leave:
                a.kw.pop(k)
            a.run(c)
            torch.cuda.synchronize()
            a.check()
        a = Adjust(2, 4, 500, "bf16", masked=True, own_mask=True, seed=4)  # a mask to each row
        a.run(c)
        torch.cuda.synchronize()
        a.check()
        a = Adjust(2, 4, 500, "bf16", seed=4)  # no rule: a copy
        a.run(c)
        torch.cuda.synchronize()
        a.check()


def test_the_last_bias_of_a_token_counts_and_masked_nan_is_masked():
    x = torch.tensor([[math.nan, math.inf, -math.inf, 1.0, -0.0, 2.0, 3.0, 4.0]], device="cuda")
    out = [torch.empty_like(x)]
    i = lambda *v: torch.tensor(v, dtype=I32, device="cuda")  # noqa: E731
    with SC.SimComm(1) as c:
        c.adjust_logits([x], 8, out, bias_start=i(0, 6), bias_token=i(3, 5, 3, -1, 2, 3),
                        bias_value=torch.tensor([1.0, 2.0, 4.0, 8.0, 5.0, 16.0], device="cuda"), mask=i(0b11111110).view(1, 1))
        torch.cuda.synchronize()
        assert out[0].tolist() == [[-math.inf, math.inf, -math.inf, 17.0, -0.0, 4.0, 3.0, 4.0]]
        assert math.copysign(1, float(out[0][0, 4])) == -1
        # an infinite bias against a token
        c.adjust_logits([x], 8, out, bias_start=i(0, 1), bias_token=i(6), bias_value=torch.tensor([-math.inf], device="cuda"))
        torch.cuda.synchronize()
        assert float(out[0][0, 6]) == -math.inf and bool(out[0][0, 0].isnan())


def test_as_a_graph_on_another_stream():
    p = 2
    a = Adjust(p, 5, 3000, "bf16", 64, 8, True, seed=6)
    with SC.SimComm(p) as c:
        stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        stream.wait_stream(torch.cuda.current_stream())
        a.run(c, stream=stream)
        stream.synchronize()
        a.check()
        with torch.cuda.graph(graph, stream=stream):
            a.run(c)
        a.kw["history"].copy_(torch.roll(a.kw["history"], 7, 1))
        a.kw["mask_row"].copy_(torch.roll(a.kw["mask_row"], 1))
        for o in a.out:
            o.fill_(0 if o.shape[1] * p == a.V else 11)
        graph.replay()
        torch.cuda.synchronize()
        a.check()
        del graph


def test_refusals_and_bad_indices():
    with SC.SimComm(2) as c:
        a = Adjust(2, 4, 500, "fp32", 16, 4, True, seed=7)
        with pytest.raises(SC.SimCommError, match="in place"):
            c.adjust_logits(a.logits, 500, a.logits[::-1])
        with pytest.raises(SC.SimCommError, match="two output"):
            c.adjust_logits(a.logits, 500, [a.out[0], a.out[0]])
        with pytest.raises(SC.SimCommError, match="ld_mask"):
            c.adjust_logits(a.logits, 500, a.out, mask=a.kw["mask"][:, :15].contiguous())
        with pytest.raises(SC.SimCommError, match="masks"):
            c.adjust_logits(a.logits, 500, a.out, mask=a.kw["mask"][:1].contiguous())
        with pytest.raises(SC.SimCommError, match="UNSUPPORTED"):
            i = [torch.zeros(4, 250, dtype=I32, device="cuda") for _ in range(4)]
            c.adjust_logits(i[:2], 500, i[2:])
        before = c.launch_count()
        c.adjust_logits([x[:0] for x in a.logits], 500, [x[:0] for x in a.out])
        assert c.launch_count() == before

        def bad(key, at, value):
            old = a.kw[key].clone()
            a.kw[key][at] = value
            a.run(c)
            torch.cuda.synchronize()
            assert c.async_error() == SC.INVALID_ARG, key
            with pytest.raises(SC.SimCommError):
                a.run(c)
            c.reset()
            a.kw[key].copy_(old)
        bad("history", (0, 3), 500)
        bad("history", (0, 3), -2)
        bad("history_len", 2, 17)
        bad("history_len", 2, -1)
        bad("prompt_len", 0, 17)
        bad("prompt_len", 0, -1)
        bad("bias_token", int(a.kw["bias_start"][2]), 500)
        bad("bias_start", 4, a.kw["bias_token"].shape[0] + 1)
        bad("bias_start", 0, -1)
        bad("bias_start", 2, 10 ** 6)
        bad("mask_row", 1, a.kw["mask"].shape[0])
        bad("mask_row", 1, -2)
        a.run(c)
        torch.cuda.synchronize()
        a.check()
