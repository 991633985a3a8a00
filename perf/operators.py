"""The language-model operators of the simulated communicator, as measured cases.

Four operators, each over p logical ranks that live in one GPU's memory:

  route      the router of an expert layer: softmax over the experts' scores, the k best, their weights,
             and the gradient of the scores
  moe        a whole expert layer (gate, up and down products, weighted sum, residual) for a few tokens
  linear     few tokens times a matrix of 4-bit weights with group scales, its shards on the ranks: split
             by rows of the matrix ("column" parallel) or along the sum ("row" parallel, all-reduced)
  logprobs   log probabilities of given tokens, entropy and top alternatives over a vocabulary whose
             columns are sharded over the ranks, and the gradient of the scores

`run` computes them in plain torch operations (own = False) or with the library's calls (own = True).
"""
import functools
import math

import torch

own = False

DT = {"fp32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # one decode step's router: a token on each of 8 ranks, top 2 of 64 experts
        {"name": "route decode", "op": "route", "p": 8, "T": 1, "E": 64, "k": 2, "dtype": "fp32", "normalise": True,
         "backward": False},
        # the router in front of the dispatch of 8 x 8192 tokens
        {"name": "route prefill", "op": "route", "p": 8, "T": 8192, "E": 64, "k": 2, "dtype": "bf16",
         "normalise": True, "backward": False},
        # a training step's router, forward and backward, an odd token count, many experts
        {"name": "route train", "op": "route", "p": 4, "T": 4099, "E": 256, "k": 8, "dtype": "fp32",
         "normalise": False, "backward": True},
        # one decode step of an expert layer: a token on each of 8 ranks
        {"name": "moe decode", "op": "moe", "p": 8, "T": 1, "E": 64, "k": 2, "H": 4096, "F": 2048, "group": 0,
         "residual": True},
        # the same layer with 4-bit experts, 16 tokens on each rank
        {"name": "moe 4-bit", "op": "moe", "p": 8, "T": 16, "E": 64, "k": 2, "H": 4096, "F": 2048, "group": 128,
         "residual": True},
        # a small odd layer: ragged sizes, no residual
        {"name": "moe odd", "op": "moe", "p": 4, "T": 33, "E": 16, "k": 4, "H": 1000, "F": 712, "group": 0,
         "residual": False},
        # the largest batch: 64 tokens on each rank, 8 experts each
        {"name": "moe batch", "op": "moe", "p": 8, "T": 64, "E": 64, "k": 8, "H": 4096, "F": 2048, "group": 0,
         "residual": True},
        # an attention output projection for one token, summed over 8 ranks
        {"name": "linear row one", "op": "linear", "p": 8, "T": 1, "N": 4096, "K": 4096, "group": 128,
         "parallel": "row", "out": "bf16"},
        # the vocabulary head for 16 tokens, its rows on 8 ranks
        {"name": "linear head", "op": "linear", "p": 8, "T": 16, "N": 131072, "K": 4096, "group": 64,
         "parallel": "column", "out": "fp32"},
        # the sampled tokens of a decode step, with alternatives
        {"name": "logprobs decode", "op": "logprobs", "p": 8, "R": 8, "V": 131072, "dtype": "fp32", "top": 8,
         "masked": True, "backward": False},
        # scoring a batch of sequences
        {"name": "logprobs score", "op": "logprobs", "p": 8, "R": 2048, "V": 131072, "dtype": "bf16", "top": 4,
         "masked": False, "backward": False},
        # a training step's loss with an entropy term: an odd vocabulary, padding rows
        {"name": "logprobs train", "op": "logprobs", "p": 4, "R": 1023, "V": 50257, "dtype": "fp32", "top": 0,
         "masked": False, "backward": True},
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "moe", "linear", "logprobs"])
    p = rng.choice([1, 2, 4, 8])
    if op == "route":
        E = p * _log(rng, max(1, 8 // p), 512 // p)
        return {"op": op, "p": p, "T": _log(rng, 1, 65536 // p), "E": E, "k": rng.randint(1, min(8, E)),
                "dtype": rng.choice(["fp32", "bf16"]), "normalise": rng.random() < 0.5,
                "backward": rng.random() < 0.5}
    if op == "moe":
        group = rng.choice([0, 0, 32, 64, 128])
        E = p * _log(rng, max(1, 8 // p), 64 // p)
        k = rng.randint(1, 4)
        unit = group or rng.choice([8, 8, 1])
        return {"op": op, "p": p, "T": _log(rng, 1, 128 // p), "E": E, "k": k,
                "H": unit * _log(rng, max(1, 256 // unit), 4096 // unit),
                "F": unit * _log(rng, max(1, 128 // unit), 2048 // unit), "group": group,
                "residual": rng.random() < 0.5}
    if op == "linear":
        parallel, group = rng.choice(["row", "column"]), rng.choice([32, 64, 128])
        rows = _log(rng, 64, 32768)
        if parallel == "row":
            return {"op": op, "p": p, "T": _log(rng, 1, 64), "N": rows,
                    "K": p * group * _log(rng, 1, max(1, 8192 // (p * group))), "group": group, "parallel": parallel,
                    "out": rng.choice(["fp32", "bf16"])}
        return {"op": op, "p": p, "T": _log(rng, 1, 64), "N": p * max(1, rows // p),
                "K": group * _log(rng, 2, 8192 // group), "group": group, "parallel": parallel,
                "out": rng.choice(["fp32", "bf16"])}
    V = _log(rng, 1000, 131072)
    return {"op": op, "p": p, "R": _log(rng, 1, max(1, min(2048, 60_000_000 // V))), "V": V,
            "dtype": rng.choice(["fp32", "bf16"]), "top": rng.choice([0, 1, 5, 20]), "masked": rng.random() < 0.5,
            "backward": rng.random() < 0.5}


# ---- inputs ----------------------------------------------------------------------------------------


def _experts(g, n, E, k):
    """k distinct experts for each of n tokens."""
    return torch.rand(n, E, generator=g, device="cuda").topk(k, dim=1).indices.to(torch.int32).contiguous()


def _w4(g, rows, K, group):
    """Packed 4-bit weights [..., K/2] (element 2i in the low half of byte i, value q - 8) and their bf16
    scales [..., K/group], for weights of about 1/sqrt(K)."""
    q = torch.randint(0, 256, (*rows, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    s = (0.5 + torch.rand(*rows, K // group, generator=g, device="cuda")) / (4.6 * math.sqrt(K))
    return q, s.to(torch.bfloat16)


def prepare(case, seed):
    g = torch.Generator("cuda")
    g.manual_seed(seed)
    p, op = case["p"], case["op"]
    randn = functools.partial(torch.randn, generator=g, device="cuda")
    s = dict(case)
    if op == "route":
        T, E, k, dt = case["T"], case["E"], case["k"], DT[case["dtype"]]
        s["logits"] = [randn(T, E).to(dt) for _ in range(p)]
        s["idx"] = [torch.empty(T, k, dtype=torch.int32, device="cuda") for _ in range(p)]
        s["weight"] = [torch.empty(T, k, device="cuda") for _ in range(p)]
        if case["backward"]:
            s["grad_weight"] = [randn(T, k) for _ in range(p)]
            s["grad_logits"] = [torch.empty(T, E, dtype=dt, device="cuda") for _ in range(p)]
    elif op == "moe":
        T, E, k, H, F, group = (case[n] for n in ("T", "E", "k", "H", "F", "group"))
        n, e = p * T, E // p
        s["x"] = [randn(T, H).to(torch.bfloat16) for _ in range(p)]
        s["idx"] = list(_experts(g, n, E, k).view(p, T, k))
        w = 0.05 + torch.rand(n, k, generator=g, device="cuda")
        s["weight"] = list((w / w.sum(1, keepdim=True)).view(p, T, k))
        if group:
            s["w_up"], s["up_scale"] = map(list, zip(*[_w4(g, (e, 2 * F), H, group) for _ in range(p)]))
            s["w_down"], s["down_scale"] = map(list, zip(*[_w4(g, (e, H), F, group) for _ in range(p)]))
        else:
            s["w_up"] = [randn(e, 2 * F, H, dtype=torch.bfloat16).mul_(H ** -0.5) for _ in range(p)]
            s["w_down"] = [randn(e, H, F, dtype=torch.bfloat16).mul_(F ** -0.5) for _ in range(p)]
            s["up_scale"] = s["down_scale"] = None
        s["res"] = [randn(T, H).to(torch.bfloat16) for _ in range(p)] if case["residual"] else None
        s["out"] = [torch.empty(T, H, dtype=torch.bfloat16, device="cuda") for _ in range(p)]
    elif op == "linear":
        T, N, K, group = (case[n] for n in ("T", "N", "K", "group"))
        row = case["parallel"] == "row"
        rows, cols = (N, K // p) if row else (N // p, K)
        if row:
            s["x"] = [randn(T, cols).to(torch.bfloat16) for _ in range(p)]
        else:
            x = randn(T, cols).to(torch.bfloat16)
            s["x"] = [x.clone() for _ in range(p)]
        s["w"], s["scale"] = map(list, zip(*[_w4(g, (rows,), cols, group) for _ in range(p)]))
        s["out_t"] = [torch.empty(T, rows, dtype=DT[case["out"]], device="cuda") for _ in range(p)]
    else:
        R, V, dt, top = case["R"], case["V"], DT[case["dtype"]], case["top"]
        m = -(-V // p)
        s["logits"] = [(2.5 * randn(R, m)).to(dt) for _ in range(p)]
        if case["masked"]:  # a grammar's mask: about half of the columns of each row
            for x in s["logits"]:
                x.masked_fill_(torch.rand(R, m, generator=g, device="cuda") < 0.5, -math.inf)
        ids = torch.randint(0, V, (R,), generator=g, device="cuda", dtype=torch.int32)
        if case["masked"]:  # a sampled token is an allowed one: here the first allowed column at or after a draw
            full = torch.cat(s["logits"], 1)[:, :V]
            far = torch.arange(V, device="cuda").expand(R, V)
            ids = torch.where((full > -math.inf) & (far >= ids[:, None]), far, V).amin(1).clamp_(max=V - 1).int()
        if case["backward"]:  # padding rows carry no token
            ids = torch.where(torch.rand(R, generator=g, device="cuda") < 0.1, -1, ids).int()
            s["grad_logprob"] = randn(R) / R
            s["grad_entropy"] = 0.01 * randn(R) / R
            s["grad_logits"] = [torch.empty(R, m, dtype=dt, device="cuda") for _ in range(p)]
        s["ids"] = ids.contiguous()
        for n in ("logprob", "entropy", "lse"):
            s[n] = [torch.empty(R, device="cuda") for _ in range(p)]
        s["top_idx"] = [torch.empty(R, top, dtype=torch.int32, device="cuda") for _ in range(p)] if top else None
        s["top_logprob"] = [torch.empty(R, top, device="cuda") for _ in range(p)] if top else None
    return s


# ---- the plain forms -------------------------------------------------------------------------------


def _ordered_top(x, k):
    """The k largest of each row of fp32 values, the lowest index first among equals: the best whole-number
    keys, whose upper half follows the value's order and whose lower half falls with the index."""
    u = (x + 0.0).view(torch.int32)
    order = (u ^ ((u >> 31) & 0x7FFFFFFF)).long() << 32
    last = x.shape[-1] - 1
    key = torch.topk(order + torch.arange(last, -1, -1, device=x.device), k, dim=-1).values
    idx = last - (key & 0xFFFFFFFF)
    return x.gather(-1, idx), idx


def _plain_route(s):
    x = torch.stack(s["logits"]).float()
    e = torch.exp(x - x.amax(-1, keepdim=True))
    prob = e / e.sum(-1, keepdim=True)
    _, idx = _ordered_top(x, s["k"])
    w = prob.gather(-1, idx)
    total = w.sum(-1, keepdim=True)
    out = {"weight": list(w / total if s["normalise"] else w), "idx": list(idx.int())}
    if s["backward"]:
        gw = torch.stack(s["grad_weight"])
        if s["normalise"]:
            q = w / total
            gx = torch.zeros_like(x).scatter_(-1, idx, q * (gw - (gw * q).sum(-1, keepdim=True)))
        else:
            gx = torch.zeros_like(x).scatter_(-1, idx, gw)
            gx = prob * (gx - (gw * w).sum(-1, keepdim=True))
        out["grad_logits"] = list(gx.to(DT[s["dtype"]]))
    return out


def _dequantised(q, scale):
    """fp32 weights of packed 4-bit ones: (q - 8) times the scale of its group."""
    w = torch.stack((q & 15, q >> 4), -1).flatten(-2).float() - 8
    return (w.unflatten(-1, (scale.shape[-1], -1)) * scale.float()[..., None]).flatten(-2)


def _plain_moe(s):
    x, F = torch.cat(s["x"]).float(), s["F"]
    up, down = torch.cat(s["w_up"]), torch.cat(s["w_down"])
    if s["group"]:
        up, down = _dequantised(up, torch.cat(s["up_scale"])), _dequantised(down, torch.cat(s["down_scale"]))
    share = torch.zeros(x.shape[0], s["E"], device="cuda")
    share.scatter_add_(1, torch.cat(s["idx"]).long(), torch.cat(s["weight"]))
    gu = torch.matmul(x, up.float().transpose(1, 2))  # every expert on every token: [E][tokens][2F]
    h = gu[..., :F] / (1 + torch.exp(-gu[..., :F])) * gu[..., F:]
    y = torch.matmul(h, down.float().transpose(1, 2))
    out = (share.t()[..., None] * y).sum(0)
    if s["res"] is not None:
        out = out + torch.cat(s["res"]).float()
    return list(out.to(torch.bfloat16).view(s["p"], s["T"], s["H"]))


def _plain_linear(s):
    w = _dequantised(torch.stack(s["w"]), torch.stack(s["scale"]))
    y = torch.matmul(torch.stack(s["x"]).float(), w.transpose(1, 2))
    if s["parallel"] == "row":
        return [y.sum(0).to(DT[s["out"]])] * s["p"]
    return list(y.to(DT[s["out"]]))


def _plain_logprobs(s):
    p, V, ids = s["p"], s["V"], s["ids"].long()
    x = torch.cat(s["logits"], 1)[:, :V].float()
    top = x.amax(1)
    e = torch.exp(x - top[:, None])
    total = e.sum(1)
    lse = top + torch.log(total)
    prob = e / total[:, None]
    logp = x - lse[:, None]
    held = torch.where(prob > 0, logp, 0)
    entropy = -(prob * held).sum(1)
    given = ids >= 0
    lp = torch.where(given, logp.gather(1, ids.clamp(min=0)[:, None])[:, 0], 0)
    out = {"logprob": [lp] * p, "entropy": [entropy] * p}
    if s["top"]:
        v, i = _ordered_top(x, s["top"])
        out["top_idx"], out["top_logprob"] = [i.int()] * p, [v - lse[:, None]] * p
    if s["backward"]:
        gl, ge = torch.where(given, s["grad_logprob"], 0), s["grad_entropy"]
        gx = -prob * (gl[:, None] + ge[:, None] * (held + entropy[:, None]))
        gx.scatter_add_(1, ids.clamp(min=0)[:, None], gl[:, None])
        m = s["logits"][0].shape[1]
        pad = torch.zeros(gx.shape[0], p * m - V, device="cuda")
        out["grad_logits"] = list(torch.cat((gx, pad), 1).to(DT[s["dtype"]]).split(m, 1))
    return out


# ---- the library's calls ---------------------------------------------------------------------------


@functools.lru_cache(None)
def _comm(p):
    from collective_communication_primitives_b200.simcomm import SimComm
    return SimComm(p)


def _own_route(s):
    c = _comm(s["p"])
    c.moe_route(s["logits"], s["idx"], s["weight"], normalise=s["normalise"])
    out = {"weight": s["weight"], "idx": s["idx"]}
    if s["backward"]:
        c.moe_route_backward(s["logits"], s["idx"], s["grad_weight"], s["grad_logits"], normalise=s["normalise"])
        out["grad_logits"] = s["grad_logits"]
    return out


def _own_moe(s):
    _comm(s["p"]).moe_layer(s["x"], s["idx"], s["weight"], s["E"], s["w_up"], s["w_down"], s["out"],
                            up_scale=s["up_scale"], down_scale=s["down_scale"], residual=s["res"])
    return s["out"]


def _own_linear(s):
    _comm(s["p"]).linear_w4(s["x"], s["w"], s["scale"], s["out_t"], parallel=s["parallel"])
    return s["out_t"]


def _own_logprobs(s):
    c = _comm(s["p"])
    c.logprobs(s["logits"], s["ids"], s["V"], s["logprob"], entropy=s["entropy"], lse=s["lse"],
               top_idx=s["top_idx"], top_logprob=s["top_logprob"])
    out = {"logprob": s["logprob"], "entropy": s["entropy"]}
    if s["top"]:
        out["top_idx"], out["top_logprob"] = s["top_idx"], s["top_logprob"]
    if s["backward"]:
        c.logprobs_backward(s["logits"], s["ids"], s["V"], s["lse"], s["grad_logprob"], s["grad_logits"],
                            entropy=s["entropy"], grad_entropy=s["grad_entropy"])
        out["grad_logits"] = s["grad_logits"]
    return out


def run(state):
    op = state["op"]
    if own:
        return {"route": _own_route, "moe": _own_moe, "linear": _own_linear, "logprobs": _own_logprobs}[op](state)
    return {"route": _plain_route, "moe": _plain_moe, "linear": _plain_linear, "logprobs": _plain_logprobs}[op](state)


# ---- what a pass cannot do without -----------------------------------------------------------------


def work(case):
    p, op = case["p"], case["op"]
    if op == "route":
        n, E, k = p * case["T"], case["E"], case["k"]
        d = 4 if case["dtype"] == "fp32" else 2
        forward = n * (E * d + 8 * k)
        # the gradient needs the picked scores, or all of them where the weights are shares of the whole
        grad = n * ((k if case["normalise"] else E) * d + 8 * k + E * d) if case["backward"] else 0
        return {"bytes": forward + grad, "flops": 4 * n * E * (1 + case["backward"])}
    if op == "moe":
        n, E, k, H, F, group = p * case["T"], case["E"], case["k"], case["H"], case["F"], case["group"]
        met = E * (1 - (1 - k / E) ** n)  # experts that some token picks, when tokens pick alike
        per = 0.5 + 2 / group if group else 2
        return {"bytes": int(met * 3 * H * F * per + n * H * 2 * (2 + case["residual"]) + 8 * n * k),
                "flops": 6 * n * k * H * F}
    if op == "linear":
        T, N, K = case["T"], case["N"], case["K"]
        row = case["parallel"] == "row"
        out = T * N * (4 if case["out"] == "fp32" else 2) * (p if row else 1)
        return {"bytes": int(N * K * (0.5 + 2 / case["group"])) + T * K * 2 * (1 if row else p) + out,
                "flops": 2 * T * N * K}
    R, V, d = case["R"], case["V"], 4 if case["dtype"] == "fp32" else 2
    grads = 2 * R * V * d if case["backward"] else 0  # the scores again, and their gradient
    return {"bytes": R * V * d + grads + 4 * R + p * R * (8 + 8 * case["top"]), "flops": (8 if grads else 4) * R * V}


# ---- from the definitions, in 64 bits --------------------------------------------------------------


def _ints4(q):
    """The whole numbers that packed 4-bit weights stand for, in 64 bits."""
    out = torch.empty(*q.shape[:-1], 2 * q.shape[-1], dtype=torch.float64, device=q.device)
    out[..., 0::2] = torch.remainder(q.to(torch.int16), 16).double() - 8
    out[..., 1::2] = torch.div(q.to(torch.int16), 16, rounding_mode="floor").double() - 8
    return out


def _exact_weight(w, scale, group):
    return _ints4(w) * scale.double().repeat_interleave(group, -1) if group else w.double()


def exact(case, seed):
    s = prepare(case, seed)
    p, op = case["p"], case["op"]
    if op == "route":
        ws, gs = [], []
        for r in range(p):
            x = s["logits"][r].double()
            prob = torch.softmax(x, 1)
            picked = torch.zeros_like(x, dtype=torch.bool)
            cols = []
            for _ in range(case["k"]):  # the best that is left, the first among equals
                left = x.masked_fill(picked, -math.inf)
                first = (left == left.amax(1, keepdim=True)).int().argmax(1, keepdim=True)
                picked.scatter_(1, first, True)
                cols.append(first)
            idx = torch.cat(cols, 1)
            w = prob.gather(1, idx)
            if case["normalise"]:
                w = w / w.sum(1, keepdim=True)
            ws.append(w)
            if case["backward"]:
                gw = s["grad_weight"][r].double()
                up = torch.zeros_like(x).scatter_(1, idx, gw)
                base = torch.zeros_like(x).scatter_(1, idx, w) if case["normalise"] else prob
                gs.append(base * (up - (gw * w).sum(1, keepdim=True)))
        out = {"weight": ws, "idx": [None] * p}
        if case["backward"]:
            out["grad_logits"] = gs
        return out
    if op == "moe":
        T, E, H, F, group = (case[n] for n in ("T", "E", "H", "F", "group"))
        x, idx, w = torch.cat(s["x"]).double(), torch.cat(s["idx"]).long(), torch.cat(s["weight"]).double()
        out = torch.cat(s["res"]).double() if case["residual"] else torch.zeros(p * T, H, dtype=torch.float64,
                                                                                 device="cuda")
        for e in torch.unique(idx).tolist():
            j, q = divmod(e, E // p)
            up = _exact_weight(s["w_up"][j][q], s["up_scale"][j][q] if group else None, group)
            down = _exact_weight(s["w_down"][j][q], s["down_scale"][j][q] if group else None, group)
            t, slot = torch.nonzero(idx == e, as_tuple=True)
            a = x[t] @ up.t()
            y = (a[:, :F] * torch.sigmoid(a[:, :F]) * a[:, F:]) @ down.t()
            out.index_add_(0, t, w[t, slot][:, None] * y)
        return list(out.view(p, T, H))
    if op == "linear":
        ys = [s["x"][r].double() @ _exact_weight(s["w"][r], s["scale"][r], case["group"]).t() for r in range(p)]
        return [torch.stack(ys).sum(0)] * p if case["parallel"] == "row" else ys
    R, V, top = case["R"], case["V"], case["top"]
    m = -(-V // p)
    x = torch.cat([v.double() for v in s["logits"]], 1)[:, :V]
    logp = torch.log_softmax(x, 1)
    prob = logp.exp()
    entropy = -torch.special.xlogy(prob, prob).sum(1)
    ids = s["ids"].long()
    at = torch.arange(V, device="cuda")[None, :] == ids[:, None]
    out = {"logprob": [logp.masked_fill(~at, 0).sum(1)] * p, "entropy": [entropy] * p}
    if top:
        out["top_idx"] = [None] * p
        out["top_logprob"] = [torch.topk(logp, top, 1).values] * p
    if case["backward"]:
        gl, ge = s["grad_logprob"].double() * (ids >= 0), s["grad_entropy"].double()
        gx = gl[:, None] * (at.double() - prob)
        gx -= ge[:, None] * (torch.special.xlogy(prob, prob) + prob * entropy[:, None])
        full = torch.zeros(R, p * m, dtype=torch.float64, device="cuda")
        full[:, :V] = gx
        out["grad_logits"] = list(full.split(m, 1))
    return out
