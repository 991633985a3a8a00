"""Argument checks of the norm, the adapters, the score adjustment and the distillation that need no GPU: NULL
communicators, the binding's checks of tensors and shapes, the layout of the struct of rules, and the rank views' meetings."""
import ctypes
import inspect
import os
import struct
import subprocess

import pytest
import torch

from collective_communication_primitives_b200 import build as B
from collective_communication_primitives_b200 import ranks
from collective_communication_primitives_b200 import simcomm as SC

BF, F, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    B.build()
    return SC.load_library()


def test_null_communicators_are_refused(lib):
    assert lib.coll_rmsnorm(None, None, None, None, 4, 8, 1e-5, 1, None, None, None, None, 0, None) == SC.INVALID_ARG
    assert lib.coll_rmsnorm_backward(None, None, None, None, None, 4, 8, 1e-5, 1, None, None, None) == SC.INVALID_ARG
    assert lib.coll_adapters(None, None, None, None, None, None, None, 1, 8, 4, 8, 8, 1, None, 1, 1, None, None) == SC.INVALID_ARG
    assert lib.coll_adjust_logits(None, None, 8, 4, 8, 1, None, None, 8, None) == SC.INVALID_ARG
    assert lib.coll_distill(None, None, 8, None, None, 2, 4, 8, 1, 1.0, 0, None, None, None) == SC.INVALID_ARG
    assert lib.coll_distill_backward(None, None, 8, None, None, 2, 4, 8, 1, 1.0, 0, None, None, None, 8, None) == SC.INVALID_ARG


def test_rules_layout_matches_the_header(tmp_path):
    fields = [name for name, _ in SC.LogitRules._fields_]
    src = tmp_path / "layout.c"
    body = "".join(f'    printf("%zu ", offsetof(coll_logit_rules_t, {f}));\n' for f in fields)
    src.write_text("#include <stddef.h>\n#include <stdio.h>\n#include \"simcomm.h\"\nint main(void) {\n" + body +
                   '    printf("%zu\\n", sizeof(coll_logit_rules_t));\n    return 0;\n}\n')
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()]
    assert got == [getattr(SC.LogitRules, f).offset for f in fields] + [ctypes.sizeof(SC.LogitRules)]


class Lib:
    def __init__(self, log, status=SC.OK):
        self.log, self.status = log, status

    def __getattr__(self, name):
        def call(*args):
            self.log.append(name)
            return self.status
        return call


def whole(p=2):
    c = object.__new__(SC.SimComm)
    c.p, c.rank, c._device, c._h = p, None, -1, None  # a CPU tensor's device number is -1
    c._pack, c._torch, c.log = struct.Struct(f"{p}P").pack, torch, []
    c._L = Lib(c.log)
    c._launch_stream = lambda stream: 0
    return c


def view(p=2, rank=1, status=SC.OK):
    c = object.__new__(ranks.RankComm)
    c.p, c.rank, c._device, c._h = p, rank, -1, None
    c._pack, c._torch, c.log = struct.Struct(f"{p}P").pack, torch, []
    c._L = Lib(c.log, status)
    c._check = lambda rc: (_ for _ in ()).throw(SC.SimCommError(rc, "refused")) if rc else None
    c.sync = lambda stream=None: c.log.append(("sync", stream))
    c._launch_stream = lambda stream: 0
    return c


def two(*shape, t=F):
    return [torch.zeros(*shape, dtype=t) for _ in range(2)]


def one(*shape, t=F):
    return torch.zeros(*shape, dtype=t)


NORM = (dict(x=two(6, 32), weight=one(32), eps=1e-5),
        dict(out=two(6, 32), residual=one(6, 32), total=two(6, 32), q=two(6, 32, t=U8), scale=two(6, 1)))
BACK = (dict(grad_out=two(6, 32), h=one(6, 32), weight=one(32), eps=1e-5, grad_x=two(6, 32)),
        dict(grad_total=one(6, 32), grad_weight=two(32)))
ADAPT = (dict(x=two(6, 16, t=BF), adapter=one(6, t=I32), a=two(3, 4, 16, t=BF), b=two(3, 8, 4, t=BF), out=two(6, 8)),
         dict(base=two(6, 8, t=BF), rank=one(3, t=I32), scale=one(3)))
RULES = dict(history=one(6, 9, t=I32), history_len=one(6, t=I32), prompt_len=one(6, t=I32), repetition=one(6), frequency=one(6),
             presence=one(6), bias_start=one(7, t=I32), bias_token=one(5, t=I32), bias_value=one(5), mask=one(2, 1, t=I32),
             mask_row=one(6, t=I32))
ADJUST = (dict(logits=two(6, 10), vocab=20, out=two(6, 10)), RULES)
DISTILL = (dict(logits=two(6, 10), vocab=20, top_idx=one(6, 3, t=I32), top_value=one(6, 3), loss=two(6)), dict(stats=two(6, 8)))
DBACK = (dict(logits=two(6, 10), vocab=20, top_idx=one(6, 3, t=I32), top_value=one(6, 3), stats=two(6, 8), grad_loss=one(6),
              grad_logits=two(6, 10)), {})
CALLS = {"rmsnorm": NORM, "rmsnorm_backward": BACK, "adapters": ADAPT, "adjust_logits": ADJUST, "distill": DISTILL,
         "distill_backward": DBACK}


def turned(t):
    """As many elements in another shape, or, of a vector, one more."""
    if isinstance(t, list):
        return [turned(v) for v in t]
    if t.dim() == 1:
        return torch.zeros(t.shape[0] + 1, dtype=t.dtype)
    return torch.zeros(*reversed(t.shape), dtype=t.dtype) if t.shape[0] != t.shape[-1] else torch.zeros(t.shape[0] * 2, dtype=t.dtype)


@pytest.mark.parametrize("name", CALLS)
def test_wrong_shapes_types_and_strides_are_refused(name):
    args, kw = CALLS[name]
    c = whole()
    getattr(c, name)(*args.values(), **kw)
    assert c.log == ["coll_" + name]
    # those whose shape says what the call's sizes are: another shape contradicts another argument
    for key, good in {**args, **kw}.items():
        if not isinstance(good, (list, torch.Tensor)):
            continue
        for wrong in (turned(good), [v.double() for v in good] if isinstance(good, list) else good.double()):
            if key == "mask" and wrong.dtype is I32:  # its shape is its own: rows and words
                continue
            a, k = dict(args), dict(kw)
            (a if key in a else k)[key] = wrong
            with pytest.raises((ValueError, TypeError)):
                getattr(c, name)(*a.values(), **k)
        if isinstance(good, list):
            a, k = dict(args), dict(kw)
            (a if key in a else k)[key] = good[:1]
            with pytest.raises((ValueError, TypeError)):
                getattr(c, name)(*a.values(), **k)
    c._device = 0
    with pytest.raises(ValueError, match="device"):
        getattr(c, name)(*args.values(), **kw)
    assert c.log == ["coll_" + name]


def test_arguments_that_go_together():
    c = whole()
    with pytest.raises(ValueError, match="scale"):
        c.rmsnorm(*NORM[0].values(), q=NORM[1]["q"])
    with pytest.raises(ValueError, match="groups"):
        c.rmsnorm(*NORM[0].values(), q=NORM[1]["q"], scale=two(6, 5))
    with pytest.raises(ValueError, match="parallel"):
        c.adapters(*ADAPT[0].values(), parallel="both")
    for keys, match in ((("history",), "history"), (("repetition",), "penalties"), (("prompt_len",), "penalties"),
                        (("bias_start", "bias_token"), "bias"), (("mask_row",), "mask")):
        with pytest.raises(ValueError, match=match):
            c.adjust_logits(*ADJUST[0].values(), **{k: RULES[k] for k in keys})
    for name in ("adjust_logits", "distill", "distill_backward"):
        a = dict(CALLS[name][0], vocab=22)
        with pytest.raises(ValueError, match="columns per rank"):
            getattr(c, name)(*a.values())
    # rows at a distance are taken where scores are, and nowhere else
    wide = [torch.zeros(6, 16)[:, :10] for _ in range(2)]
    c.adjust_logits(wide, 20, wide)
    c.distill(wide, 20, *list(DISTILL[0].values())[2:])
    with pytest.raises(ValueError, match="contiguous"):
        c.rmsnorm([torch.zeros(6, 40)[:, :32] for _ in range(2)], one(32), 1e-5, out=two(6, 32))
    with pytest.raises(ValueError, match="contiguous"):
        c.adjust_logits(*ADJUST[0].values(), history=torch.zeros(6, 12, dtype=I32)[:, :9], history_len=one(6, t=I32))
    assert c.log == ["coll_adjust_logits", "coll_distill"]


def own(ts, other=None):
    return ts if not isinstance(ts, list) else [other, ts[1]]


PEERS = {"rmsnorm": ("x",), "rmsnorm_backward": ("grad_out",), "adapters": ("x", "a"), "distill": ("logits",)}


def of_view(name):
    args, kw = CALLS[name]
    take = lambda d: {k: own(v, 64 if k in PEERS.get(name, ()) else None) for k, v in d.items()}  # noqa: E731
    return take(args), take(kw)


@pytest.mark.parametrize("name", list(PEERS))
def test_calls_that_read_peers_meet_the_ranks_before_and_after(name):
    a, k = of_view(name)
    c = view()
    getattr(c, name)(*a.values(), **k)
    getattr(c, name)(*a.values(), **k, stream=5)
    assert c.log == [("sync", None), "coll_" + name, ("sync", None), ("sync", 5), "coll_" + name, ("sync", 5)]
    c = view(status=SC.INVALID_ARG)
    with pytest.raises(SC.SimCommError):
        getattr(c, name)(*a.values(), **k)
    assert c.log == [("sync", None), "coll_" + name, ("sync", None)]


def test_calls_on_own_memory_meet_nobody():
    c = view()
    for name in ("adjust_logits", "distill_backward"):
        a, k = of_view(name)
        getattr(c, name)(*a.values(), **k)
    args, kw = ADAPT
    c.adapters(*[own(v) for v in args.values()], **{k: own(v) for k, v in kw.items()}, parallel="column")
    assert c.log == ["coll_adjust_logits", "coll_distill_backward", "coll_adapters"]


@pytest.mark.parametrize("name", list(CALLS))
def test_arguments_are_those_of_the_whole_communicator(name):
    assert inspect.signature(getattr(ranks.RankComm, name)) == inspect.signature(getattr(SC.SimComm, name))
