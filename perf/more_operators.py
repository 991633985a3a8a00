"""More operators of a model's step on the simulated communicator, as measured cases.

Over p logical ranks that live in one GPU's memory:

  norm       rows that lie on the ranks as partial sums: all-reduced, the residual added, root-mean-square norm,
             if asked in 8 bits with scales; and the gradient
  adapters   low-rank adapters of many requests at once, added to what a shared projection gave
  adjust     penalties for repeated tokens, biases and grammar masks on scores whose columns are on the ranks
  distill    loss against a teacher's best logits, over a vocabulary whose columns are on the ranks; and the gradient

`run` computes them in plain torch operations (own = False) or with the library's calls (own = True).
"""
import functools
import math

import torch

own = False

DT = {"fp32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-5


def listed():
    return [
        # between two products of a decode step: one token's partial sums of 8 ranks
        {"name": "norm decode", "op": "norm", "p": 8, "T": 1, "H": 4096, "dtype": "bf16", "residual": True, "group": 0,
         "backward": False},
        # in front of a dispatch of 8-bit rows: a prompt's tokens, a scale per 128 columns
        {"name": "norm 8-bit", "op": "norm", "p": 8, "T": 2048, "H": 4096, "dtype": "bf16", "residual": True,
         "group": 128, "backward": False},
        # odd sizes, fp32, 8-bit rows with one scale each, no residual
        {"name": "norm odd", "op": "norm", "p": 4, "T": 333, "H": 1001, "dtype": "fp32", "residual": False,
         "group": 1001, "backward": False},
        # a training step, forward and backward with the weight's gradient
        {"name": "norm train", "op": "norm", "p": 8, "T": 2048, "H": 4096, "dtype": "bf16", "residual": True, "group": 0,
         "backward": True},
        # a decode step of 32 requests, each with its own adapter, beside an attention output projection
        {"name": "adapters decode", "op": "adapters", "p": 8, "T": 32, "N": 4096, "K": 4096, "S": 64, "R": 16,
         "parallel": "row", "base": "fp32", "out": "bf16", "runs": 1},
        # prompts of some requests, tokens in runs, beside a column-parallel projection
        {"name": "adapters prompt", "op": "adapters", "p": 8, "T": 4099, "N": 4096, "K": 4096, "S": 8, "R": 64,
         "parallel": "column", "base": "bf16", "out": "bf16", "runs": 700},
        # a decode step of 8 requests under a grammar: long histories, biases
        {"name": "adjust decode", "op": "adjust", "p": 8, "R": 8, "V": 131072, "dtype": "fp32", "history": 4096,
         "bias": 16, "masked": True},
        # a large batch of requests, short histories, a mask for some
        {"name": "adjust batch", "op": "adjust", "p": 8, "R": 256, "V": 131072, "dtype": "bf16", "history": 1024,
         "bias": 0, "masked": True},
        # an odd vocabulary whose shards end in padding, many biases
        {"name": "adjust odd", "op": "adjust", "p": 4, "R": 33, "V": 50257, "dtype": "fp32", "history": 333,
         "bias": 300, "masked": False},
        # a few rows against a teacher's 32 best, the rest of the vocabulary as one more class
        {"name": "distill few", "op": "distill", "p": 8, "R": 16, "V": 131072, "dtype": "fp32", "n": 32,
         "tail": True, "temperature": 1.0, "backward": True},
        # a training step on an odd vocabulary, some rows without a teacher
        {"name": "distill odd", "op": "distill", "p": 4, "R": 1023, "V": 50257, "dtype": "fp32", "n": 20,
         "tail": False, "temperature": 2.0, "backward": True},
        # the largest training step
        {"name": "distill train", "op": "distill", "p": 8, "R": 2048, "V": 131072, "dtype": "bf16", "n": 32,
         "tail": True, "temperature": 1.0, "backward": True},
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "adapters", "adjust", "distill"])
    p = rng.choice([1, 2, 4, 8])
    if op == "norm":
        unit = rng.choice([1, 8, 128])
        H = unit * _log(rng, max(1, 64 // unit), 8192 // unit)
        backward = rng.random() < 0.4
        groups = [0, H] + [g for g in (32, 64, 128) if H % g == 0]
        return {"op": op, "p": p, "T": _log(rng, 1, max(1, min(16384 // p, 60_000_000 // (p * H)))), "H": H,
                "dtype": rng.choice(["fp32", "bf16"]), "residual": rng.random() < 0.7,
                "group": 0 if backward else rng.choice(groups), "backward": backward}
    if op == "adapters":
        unit = p * rng.choice([1, 8, 64])
        T = _log(rng, 1, 4096)
        return {"op": op, "p": p, "T": T, "N": unit * _log(rng, max(1, 64 // unit), 8192 // unit),
                "K": unit * _log(rng, max(1, 64 // unit), 8192 // unit), "S": _log(rng, 1, 64 if T <= 256 else 12),
                "R": rng.choice([4, 8, 16, 16, 32, 64, rng.randint(1, 64)]), "parallel": rng.choice(["row", "column"]),
                "base": rng.choice(["fp32", "bf16"]), "out": rng.choice(["fp32", "bf16"]),
                "runs": rng.choice([1, 1 + T // 3])}
    V = _log(rng, 1000, 131072)
    if op == "adjust":
        return {"op": op, "p": p, "R": _log(rng, 1, max(1, min(256, 30_000_000 // V))), "V": V,
                "dtype": rng.choice(["fp32", "bf16"]), "history": _log(rng, 1, 16384),
                "bias": rng.choice([0, 1, 20, 300]), "masked": rng.random() < 0.5}
    return {"op": op, "p": p, "R": _log(rng, 1, max(1, min(2048, 60_000_000 // V))), "V": V,
            "dtype": rng.choice(["fp32", "bf16"]), "n": _log(rng, 1, 128), "tail": rng.random() < 0.5,
            "temperature": 1.0, "backward": rng.random() < 0.6} | ({} if rng.random() < 0.5 else
                                                                   {"tail": False, "temperature": 2.5})


# ---- inputs ----------------------------------------------------------------------------------------


def _each(p, *shape, dtype=torch.float32):
    return [torch.empty(*shape, dtype=dtype, device="cuda") for _ in range(p)]


def prepare(case, seed):
    g = torch.Generator("cuda")
    g.manual_seed(seed)
    p, op = case["p"], case["op"]
    randn = functools.partial(torch.randn, generator=g, device="cuda")
    rand = functools.partial(torch.rand, generator=g, device="cuda")
    randint = functools.partial(torch.randint, generator=g, device="cuda", dtype=torch.int32)
    s = dict(case)
    if op == "norm":
        T, H, dt, group = case["T"], case["H"], DT[case["dtype"]], case["group"]
        s["x"] = [(p ** -0.5 * randn(T, H)).to(dt) for _ in range(p)]
        s["res"] = (2 * randn(T, H)).to(dt) if case["residual"] else None
        s["w"] = (1 + 0.2 * randn(H)).to(dt)
        s["total"] = _each(p, T, H, dtype=dt)
        if group:
            s["q"], s["scale"] = _each(p, T, H, dtype=torch.float8_e4m3fn), _each(p, T, H // group)
        else:
            s["y"] = _each(p, T, H, dtype=dt)
        if case["backward"]:
            s["gy"] = [randn(T, H).to(dt) for _ in range(p)]
            s["gt"] = randn(T, H).to(dt)
            s["gx"], s["gw"] = _each(p, T, H, dtype=dt), _each(p, H)
    elif op == "adapters":
        T, N, K, S, R = (case[n] for n in ("T", "N", "K", "S", "R"))
        row = case["parallel"] == "row"
        bf = torch.bfloat16
        x = randn(T, K).to(bf)
        a = (randn(S, R, K) * K ** -0.5).to(bf)
        b = (randn(S, N, R) * R ** -0.5).to(bf)
        base = randn(T, N).to(DT[case["base"]])
        cut = lambda t, d: [v.contiguous() for v in t.chunk(p, d)]  # noqa: E731
        copies = lambda t: [t.clone() for _ in range(p)]  # noqa: E731
        s["x"], s["a"] = (cut(x, 1), cut(a, 2)) if row else (copies(x), copies(a))
        s["b"], s["base_t"] = (copies(b), copies(base)) if row else (cut(b, 1), cut(base, 1))
        s["out_t"] = _each(p, T, N if row else N // p, dtype=DT[case["out"]])
        # runs of tokens of one request; about one run in sixteen has no adapter
        runs = -(-T // case["runs"])
        pick = randint(0, S, (runs,))
        pick = torch.where(rand(runs) < 1 / 16, -1, pick).int()
        s["adapter"] = pick.repeat_interleave(case["runs"])[:T].contiguous()
        s["scales"] = 0.5 + rand(S)
    elif op == "adjust":
        R, V, dt, L, nb = case["R"], case["V"], DT[case["dtype"]], case["history"], case["bias"]
        m = -(-V // p)
        s["logits"] = [(2.5 * randn(R, m)).to(dt) for _ in range(p)]
        s["out"] = [torch.zeros(R, m, dtype=dt, device="cuda") for _ in range(p)]  # padding columns stay 0
        # tokens of a text: a few common ones, a long tail
        s["seen"] = (V * rand(R, L) ** 4).int().clamp_(max=V - 1)
        s["len"] = randint(L // 2, L + 1, (R,))
        s["prompt"] = (s["len"] * rand(R)).int()
        s["rep"], s["freq"], s["pres"] = 1 + 0.3 * rand(R), 0.5 * rand(R), 0.5 * rand(R)
        if nb:  # a request's biases name distinct tokens, here at equal distances
            step = V // nb if V >= nb else 1
            at = torch.arange(nb, device="cuda") * step
            s["bias_start"] = torch.arange(0, R * nb + 1, nb, device="cuda", dtype=torch.int32)
            s["bias_token"] = (at + randint(0, step, (R, nb))).int().view(-1).contiguous()
            s["bias_value"] = 3 * randn(R * nb)
        if case["masked"]:  # grammars: each allows a share of the vocabulary; some rows have none
            words, n = -(-V // 32), max(1, R // 4)
            bits = torch.zeros(n, words, dtype=torch.int32, device="cuda")
            share = 0.02 + 0.9 * rand(n, 1)
            for i in range(32):
                bits |= (rand(n, words) < share).int() << i
            s["mask"], s["mask_row"] = bits, randint(-1, n, (R,))
    else:
        R, V, dt, n = case["R"], case["V"], DT[case["dtype"]], case["n"]
        m = -(-V // p)
        x = 2.5 * randn(R, p * m)
        s["logits"] = [v.to(dt).contiguous() for v in x.chunk(p, 1)]
        # the teacher's scores: like the student's, a little off
        t = x.add_(0.7 * randn(R, p * m))[:, :V]
        best = torch.topk(t, n, 1)
        s["top_idx"] = best.indices.int()
        s["top_value"] = (best.values - torch.logsumexp(t, 1, keepdim=True)).contiguous()
        del x, t
        if case["backward"]:  # rows without a teacher (padding), places it left open
            s["top_idx"][rand(R) < 0.05] = -1
            s["top_idx"][:, n - 1][rand(R) < 0.1] = -1
            s["grad_loss"] = (0.5 + rand(R)) / R
            s["grad_logits"] = _each(p, R, m, dtype=dt)
        s["loss"], s["stats"] = _each(p, R), _each(p, R, 8)
    return s


# ---- the plain forms -------------------------------------------------------------------------------


def _plain_norm(s):
    p, dt, H = s["p"], DT[s["dtype"]], s["H"]
    h = torch.stack(s["x"]).float().sum(0)
    if s["res"] is not None:
        h = h + s["res"].float()
    w = s["w"].float()
    y = h * torch.rsqrt((h * h).mean(1, keepdim=True) + EPS) * w
    total = h.to(dt)
    out = {"total": [total] * p}
    if s["group"]:
        part = y.view(y.shape[0], -1, s["group"])
        scale = part.abs().amax(2) / 448
        q = (part / scale[..., None]).to(torch.float8_e4m3fn)
        out["q"], out["scale"] = [q.view(y.shape)] * p, [scale] * p
    else:
        out["y"] = [y.to(dt)] * p
    if s["backward"]:
        h = total.float()
        g = torch.stack(s["gy"]).float().sum(0)
        r = torch.rsqrt((h * h).mean(1, keepdim=True) + EPS)
        wg = w * g
        gx = r * wg - h * (r * r * r * (wg * h).sum(1, keepdim=True) / H) + s["gt"].float()
        out["gx"], out["gw"] = [gx.to(dt)] * p, [(g * h * r).sum(0)] * p
    return out


def _plain_adapters(s):
    p, T, S, R = s["p"], s["T"], s["S"], s["R"]
    row, dt = s["parallel"] == "row", DT[s["out"]]
    # every adapter on every token, then each token's own
    if row:
        u = torch.cat(s["x"], 1).float() @ torch.cat(s["a"], 2).float().view(S * R, -1).t()
    else:
        u = s["x"][0].float() @ s["a"][0].float().view(S * R, -1).t()
    mine = s["adapter"][:, None] == torch.arange(S, device="cuda")
    u = (u.view(T, S, R) * (mine * s["scales"])[..., None]).view(T, S * R)
    if row:
        delta = u @ s["b"][0].float().transpose(1, 2).reshape(S * R, -1)
        return list((torch.stack(s["base_t"]).float() + delta).to(dt))
    delta = u @ torch.stack(s["b"]).float().transpose(2, 3).reshape(p, S * R, -1)
    return list((torch.stack(s["base_t"]).float() + delta).to(dt))


def _plain_adjust(s):
    R, V, L = s["R"], s["V"], s["history"]
    x = torch.cat(s["logits"], 1)[:, :V].float()
    at = torch.arange(L, device="cuda")
    held = at < s["len"][:, None]
    new = held & (at >= s["prompt"][:, None])
    seen = s["seen"].long()
    count = torch.zeros(R, V, device="cuda").scatter_add_(1, seen, new.float())
    any_ = torch.zeros(R, V, device="cuda").scatter_add_(1, seen, held.float()) > 0
    rep = s["rep"][:, None]
    x = torch.where(any_, torch.where(x > 0, x / rep, x * rep), x)
    x = x - s["freq"][:, None] * count - s["pres"][:, None] * (count > 0)
    if s["bias"]:
        x = x.scatter_add(1, s["bias_token"].view(R, -1).long(), s["bias_value"].view(R, -1))
    if s["masked"]:
        bits = s["mask"][s["mask_row"].clamp(min=0).long()]
        allowed = ((bits[:, :, None] >> torch.arange(32, device="cuda")) & 1).view(R, -1)[:, :V] != 0
        x = torch.where(allowed | (s["mask_row"] < 0)[:, None], x, -math.inf)
    x = torch.cat((x, torch.zeros(R, s["p"] * s["logits"][0].shape[1] - V, device="cuda")), 1)
    return list(x.to(DT[s["dtype"]]).chunk(s["p"], 1))


def _plain_distill(s):
    p, V, tau = s["p"], s["V"], s["temperature"]
    m = s["logits"][0].shape[1]
    x = torch.cat(s["logits"], 1)[:, :V].float() / tau
    top = x.amax(1, keepdim=True)
    e = torch.exp(x - top)
    total = e.sum(1, keepdim=True)
    ids, given = s["top_idx"].clamp(min=0).long(), s["top_idx"] >= 0
    lp = x.gather(1, ids) - top - torch.log(total)
    v = torch.where(given, s["top_value"] / tau, -math.inf)
    if s["tail"]:
        lq, q = v, torch.exp(v)
        taken = torch.zeros_like(x, dtype=torch.bool)
        taken.scatter_(1, torch.where(given, ids, ids.amax(1, keepdim=True)), given.any(1, keepdim=True).expand_as(ids))
        rest = torch.where(taken, 0, e).sum(1) / total[:, 0]
        left = 1 - q.sum(1)
        left = torch.where(left < 2.0 ** -20, 0, left)
    else:
        high = v.amax(1, keepdim=True)
        high = torch.where(high > -math.inf, high, 0)
        z = torch.exp(v - high)
        zs = z.sum(1, keepdim=True)
        q = torch.where(zs > 0, z / zs, 0)
        lq = v - high - torch.log(zs)
    loss = torch.where(q > 0, q * (lq - lp), 0).sum(1)
    if s["tail"]:
        loss = loss + torch.where(left > 0, left * (torch.log(left) - torch.log(rest)), 0)
    out = {"loss": [loss] * p}
    if s["backward"]:
        weight = q.sum(1, keepdim=True)
        if s["tail"]:
            weight = weight + left[:, None] * torch.where(taken, 1, 1 - 1 / rest[:, None])
        gx = e / total * weight
        gx.scatter_add_(1, ids, torch.where(given, -q, 0))
        gx = gx * (s["grad_loss"][:, None] / tau)
        pad = torch.zeros(gx.shape[0], p * m - V, device="cuda")
        out["grad_logits"] = list(torch.cat((gx, pad), 1).to(DT[s["dtype"]]).split(m, 1))
    return out


# ---- the library's calls ---------------------------------------------------------------------------


@functools.lru_cache(None)
def _comm(p):
    from collective_communication_primitives_b200.simcomm import SimComm
    return SimComm(p)


def _own_norm(s):
    c = _comm(s["p"])
    out = {"total": s["total"]}
    if s["group"]:
        c.rmsnorm(s["x"], s["w"], EPS, residual=s["res"], total=s["total"], q=s["q"], scale=s["scale"])
        out["q"], out["scale"] = s["q"], s["scale"]
    else:
        c.rmsnorm(s["x"], s["w"], EPS, out=s["y"], residual=s["res"], total=s["total"])
        out["y"] = s["y"]
    if s["backward"]:
        c.rmsnorm_backward(s["gy"], s["total"][0], s["w"], EPS, s["gx"], grad_total=s["gt"], grad_weight=s["gw"])
        out["gx"], out["gw"] = s["gx"], s["gw"]
    return out


def _own_adapters(s):
    _comm(s["p"]).adapters(s["x"], s["adapter"], s["a"], s["b"], s["out_t"], base=s["base_t"], scale=s["scales"],
                           parallel=s["parallel"])
    return s["out_t"]


def _own_adjust(s):
    more = {}
    if s["bias"]:
        more |= {"bias_start": s["bias_start"], "bias_token": s["bias_token"], "bias_value": s["bias_value"]}
    if s["masked"]:
        more |= {"mask": s["mask"], "mask_row": s["mask_row"]}
    _comm(s["p"]).adjust_logits(s["logits"], s["V"], s["out"], history=s["seen"], history_len=s["len"],
                                prompt_len=s["prompt"], repetition=s["rep"], frequency=s["freq"], presence=s["pres"],
                                **more)
    return s["out"]


def _own_distill(s):
    c = _comm(s["p"])
    c.distill(s["logits"], s["V"], s["top_idx"], s["top_value"], s["loss"], stats=s["stats"],
              temperature=s["temperature"], tail=s["tail"])
    out = {"loss": s["loss"]}
    if s["backward"]:
        c.distill_backward(s["logits"], s["V"], s["top_idx"], s["top_value"], s["stats"], s["grad_loss"],
                           s["grad_logits"], temperature=s["temperature"], tail=s["tail"])
        out["grad_logits"] = s["grad_logits"]
    return out


def run(state):
    op = state["op"]
    if own:
        return {"norm": _own_norm, "adapters": _own_adapters, "adjust": _own_adjust, "distill": _own_distill}[op](state)
    return {"norm": _plain_norm, "adapters": _plain_adapters, "adjust": _plain_adjust,
            "distill": _plain_distill}[op](state)


# ---- what a pass cannot do without -----------------------------------------------------------------


def work(case):
    p, op = case["p"], case["op"]
    if op == "norm":
        T, H, d = case["T"], case["H"], 4 if case["dtype"] == "fp32" else 2
        rows = T * H * d
        out = p * T * (H + 4 * (H // case["group"])) if case["group"] else p * rows
        total = p * rows + case["residual"] * rows + H * d + p * rows + out
        if case["backward"]:  # the ranks' gradients, the stored sum and its gradient; both gradients out
            total += p * rows + 2 * rows + H * d + p * rows + p * 4 * H
        return {"bytes": total, "flops": T * H * (p + 5) * (2 if case["backward"] else 1)}
    if op == "adapters":
        T, N, K, S, R = (case[n] for n in ("T", "N", "K", "S", "R"))
        row = case["parallel"] == "row"
        runs = -(-T // case["runs"])
        met = S * (1 - (1 - 15 / 16 / S) ** runs)  # adapters that some run of tokens has
        ends = (4 if case["base"] == "fp32" else 2) + (4 if case["out"] == "fp32" else 2)
        copies = p if row else 1
        return {"bytes": int(2 * met * R * (K + N)) + 2 * T * K + T * N * ends * copies + 4 * T,
                "flops": 2 * T * R * (K + N)}
    if op == "adjust":
        R, V, d = case["R"], case["V"], 4 if case["dtype"] == "fp32" else 2
        mask = max(1, R // 4) * V // 8 if case["masked"] else 0
        return {"bytes": 2 * R * V * d + 3 * R * case["history"] + 8 * R * case["bias"] + mask, "flops": 3 * R * V}
    R, V, d = case["R"], case["V"], 4 if case["dtype"] == "fp32" else 2
    grads = 2 * R * V * d if case["backward"] else 0  # the scores again, and their gradient
    return {"bytes": R * V * d + grads + 8 * R * case["n"] + p * R * 36, "flops": (6 if grads else 3) * R * V}


# ---- from the definitions, in 64 bits --------------------------------------------------------------


def _e4m3(v):
    """The nearest value with 3 bits behind the leading one, exponents from -6 up, ties to even."""
    e = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6)))
    step = torch.exp2(e - 3)
    return (torch.round(v / step) * step).clamp(-448, 448)


def exact(case, seed):
    s = prepare(case, seed)
    p, op = case["p"], case["op"]
    if op == "norm":
        h = s["res"].double() if case["residual"] else torch.zeros(case["T"], case["H"], dtype=torch.float64, device="cuda")
        for x in s["x"]:
            h = h + x.double()
        w = s["w"].double()
        y = w * h / torch.sqrt(h.square().mean(1, keepdim=True) + EPS)
        out = {"total": [h] * p}
        if case["group"]:
            qs, scales = [], []
            for part in y.split(case["group"], 1):
                scales.append(part.abs().max(1).values / 448)
                qs.append(_e4m3(part / scales[-1][:, None]))
            out["q"], out["scale"] = [torch.cat(qs, 1)] * p, [torch.stack(scales, 1)] * p
        else:
            out["y"] = [y] * p
        if case["backward"]:  # at the stored, rounded sum
            h = h.to(DT[case["dtype"]]).double()
            g = sum(v.double() for v in s["gy"])
            norm = torch.sqrt(h.square().mean(1, keepdim=True) + EPS)
            unit = h / norm
            along = (w * g * unit).mean(1, keepdim=True)
            out["gx"] = [(w * g - unit * along) / norm + s["gt"].double()] * p
            out["gw"] = [(g * unit).sum(0)] * p
        return out
    if op == "adapters":
        row = case["parallel"] == "row"
        outs = [b.double() for b in s["base_t"]]
        for i in range(case["S"]):
            t = torch.nonzero(s["adapter"] == i)[:, 0]
            if not len(t):
                continue
            if row:
                u = sum(s["x"][r][t].double() @ s["a"][r][i].double().t() for r in range(p))
            for r in range(p):
                if not row:
                    u = s["x"][r][t].double() @ s["a"][r][i].double().t()
                outs[r][t] += s["scales"][i].double() * (u @ s["b"][r][i].double().t())
        return outs
    if op == "adjust":
        R, V = case["R"], case["V"]
        x = torch.cat([v.double() for v in s["logits"]], 1)[:, :V].contiguous()
        for t in range(R):
            n, k = int(s["len"][t]), int(s["prompt"][t])
            ids = s["seen"][t, :n].long()
            met = torch.unique(ids)
            rep = s["rep"][t].double()
            x[t, met] = torch.where(x[t, met] > 0, x[t, met] / rep, x[t, met] * rep)
            met, times = torch.unique(ids[k:], return_counts=True)
            x[t, met] -= s["freq"][t].double() * times + s["pres"][t].double()
            if case["bias"]:
                at = slice(int(s["bias_start"][t]), int(s["bias_start"][t + 1]))
                x[t, s["bias_token"][at].long()] += s["bias_value"][at].double()
            if case["masked"] and int(s["mask_row"][t]) >= 0:
                words = s["mask"][int(s["mask_row"][t])].long() & 0xFFFFFFFF
                bits = torch.stack([torch.div(words, 2 ** i, rounding_mode="floor") % 2 for i in range(32)], 1)
                x[t, bits.view(-1)[:V] == 0] = -math.inf
        m = s["logits"][0].shape[1]
        full = torch.zeros(R, p * m, dtype=torch.float64, device="cuda")
        full[:, :V] = x
        return list(full.split(m, 1))
    R, V, tau = case["R"], case["V"], case["temperature"]
    m = -(-V // p)
    x = torch.cat([v.double() for v in s["logits"]], 1)[:, :V] / tau
    logp = torch.log_softmax(x, 1)
    del x
    given = s["top_idx"] >= 0
    teacher = torch.zeros(R, V + 1, dtype=torch.float64, device="cuda")  # one more column takes what is not given
    ids = torch.where(given, s["top_idx"], V).long()
    v = s["top_value"].double().masked_fill(~given, -math.inf) / tau
    q = v.exp() if case["tail"] else torch.nan_to_num(torch.softmax(v, 1), nan=0.0)
    teacher.scatter_add_(1, ids, q)
    teacher = teacher[:, :V]
    loss = (torch.special.xlogy(teacher, teacher) - teacher * logp).sum(1)
    slope = logp.exp()
    if case["tail"]:
        listed_ = torch.zeros(R, V + 1, dtype=torch.bool, device="cuda").scatter_(1, ids, True)[:, :V]
        rest = slope.masked_fill(listed_, 0).sum(1, keepdim=True)
        left = 1 - teacher.sum(1, keepdim=True)
        left = torch.where(left < 2.0 ** -20, torch.zeros_like(left), left)
        loss += (torch.special.xlogy(left, left) - torch.special.xlogy(left, rest))[:, 0]
        slope = slope * (teacher.sum(1, keepdim=True) + left - torch.where(listed_, 0, left / rest))
    else:
        slope = slope * teacher.sum(1, keepdim=True)
    out = {"loss": [loss] * p}
    if case["backward"]:
        full = torch.zeros(R, p * m, dtype=torch.float64, device="cuda")
        full[:, :V] = (slope - teacher) * s["grad_loss"].double()[:, None] / tau
        out["grad_logits"] = list(full.split(m, 1))
    return out
