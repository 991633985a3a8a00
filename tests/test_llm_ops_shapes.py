"""The binding refuses tensors of the right number of elements in the wrong shape: a transposed matrix, scales with
groups and rows exchanged, picks slot by slot."""
import struct

import pytest
import torch

from collective_communication_primitives_b200 import simcomm as SC

BF, U8, I32 = torch.bfloat16, torch.uint8, torch.int32


class Lib:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append(name)
            return SC.OK
        return call


def fake(p=2):
    c = object.__new__(SC.SimComm)
    c.p, c.rank, c._device, c._h = p, None, -1, None  # a CPU tensor's device number is -1
    c._pack, c._torch, c._L = struct.Struct(f"{p}P").pack, torch, Lib()
    c._launch_stream = lambda stream: 0
    return c


def two(*shape, t=torch.float32):
    return [torch.zeros(*shape, dtype=t) for _ in range(2)]


def turned(ts, *order):
    """The same elements in another order of axes, contiguous."""
    return [t.permute(*order).contiguous() for t in ts]


def refuses(call, name, args, kw, **wrong):
    """The call goes through as it is, and not with any of the wrong tensors (by position or keyword)."""
    c = fake()
    getattr(c, call)(*args.values(), **kw)
    assert c._L.calls == [name]
    for key, value in wrong.items():
        a, k = dict(args), dict(kw)
        (a if key in a else k)[key] = value
        with pytest.raises(ValueError, match=key):
            getattr(c, call)(*a.values(), **k)
    assert c._L.calls == [name]


def test_flat_tensors_and_vectors_of_any_shape_are_taken():
    c = fake()
    x, idx, w = two(6, 8), two(6, 2, t=I32), two(6, 2)
    c.moe_route(x, idx, [t.view(-1) for t in w])
    c.logprobs(two(6, 10), torch.zeros(2, 3, dtype=I32), 20, [t.view(6, 1) for t in two(6)])
    assert c._L.calls == ["coll_moe_route", "coll_logprobs"]


def test_router():
    T, E, k = 6, 8, 2
    a = {"logits": two(T, E), "topk_idx": two(T, k, t=I32), "topk_weight": two(T, k)}
    refuses("moe_route", "coll_moe_route", a, {}, topk_weight=turned(a["topk_weight"], 1, 0))
    a = {"logits": two(T, E), "topk_idx": two(T, k, t=I32), "grad_weight": two(T, k), "grad_logits": two(T, E)}
    refuses("moe_route_backward", "coll_moe_route_backward", a, {}, grad_weight=turned(a["grad_weight"], 1, 0),
            grad_logits=turned(a["grad_logits"], 1, 0))


@pytest.mark.parametrize("parallel", ["row", "column"])
def test_linear(parallel):
    T, N, K, groups = 5, 12, 128, 2
    a = {"x": two(T, K, t=BF), "w": two(N, K // 2, t=U8), "scale": two(N, groups, t=BF), "out": two(T, N, t=BF)}
    mixed = [a["scale"][0], a["scale"][1].t().contiguous()]
    refuses("linear_w4", "coll_linear_w4", a, {"parallel": parallel}, out=turned(a["out"], 1, 0), scale=mixed,
            w=[a["w"][0], a["w"][1].view(N // 2, K)])


@pytest.mark.parametrize("group", [0, 32])
def test_expert_layer(group):
    T, E, k, H, F = 5, 4, 2, 64, 96
    per, wt = (2, U8) if group else (1, BF)
    a = {"x": two(T, H, t=BF), "topk_idx": two(T, k, t=I32), "topk_weight": two(T, k), "experts": E,
         "w_up": two(E // 2, 2 * F, H // per, t=wt), "w_down": two(E // 2, H, F // per, t=wt), "out": two(T, H, t=BF)}
    kw = {"residual": two(T, H, t=BF)}
    wrong = {"topk_weight": turned(a["topk_weight"], 1, 0), "w_down": turned(a["w_down"], 0, 2, 1),
             "residual": turned(kw["residual"], 1, 0), "out": turned(a["out"], 1, 0)}
    if group:
        kw.update(up_scale=two(E // 2, 2 * F, H // group, t=BF), down_scale=two(E // 2, H, F // group, t=BF))
        wrong["down_scale"] = turned(kw["down_scale"], 0, 2, 1)
    refuses("moe_layer", "coll_moe_layer", a, kw, **wrong)


def test_log_probabilities():
    R, V, n = 6, 20, 3
    a = {"logits": two(R, V // 2), "tokens": torch.zeros(R, dtype=I32), "vocab": V, "logprob": two(R)}
    kw = {"entropy": two(R), "lse": two(R), "top_idx": two(R, n, t=I32), "top_logprob": two(R, n)}
    refuses("logprobs", "coll_logprobs", a, kw, top_logprob=turned(kw["top_logprob"], 1, 0),
            logits=[a["logits"][0], a["logits"][1].view(V // 2, R)])
    a = {"logits": two(R, V // 2), "tokens": torch.zeros(R, dtype=I32), "vocab": V, "lse": two(R),
         "grad_logprob": torch.zeros(R), "grad_logits": two(R, V // 2)}
    refuses("logprobs_backward", "coll_logprobs_backward", a, {}, grad_logits=[a["grad_logits"][0], torch.zeros(V // 2, R)])
