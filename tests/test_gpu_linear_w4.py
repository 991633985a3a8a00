"""GPU tests of the 4-bit linear against float64.

The products of whole numbers and bf16 tokens are exact; summed in fp32 they err by at most
(group + group / 16) 2^-23 of their magnitudes within a group (a matrix instruction may truncate), the
scaled sums over the groups by another (K / group + 8) 2^-24, and the output's rounding by half a step.
"""
import pytest
import torch

from collective_communication_primitives_b200 import simcomm as SC
from test_gpu_moe_layer import make_weights

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
DT = {"fp32": torch.float32, "bf16": BF}


def make(p, T, N, K, group, parallel, out, seed=0, offset=0):
    g = torch.Generator("cuda").manual_seed(seed)
    row = parallel == "row"
    n, k = (N, K // p) if row else (N // p, K)
    xs = []
    first = torch.randn(T * k + offset, generator=g, device="cuda").to(BF)[offset:].view(T, k)
    for r in range(p):
        x = torch.randn(T * k + offset, generator=g, device="cuda").to(BF)[offset:].view(T, k) if row else first
        xs.append(x)
    w = [make_weights(g, (n,), k, group) for _ in range(p)]
    o = [torch.full((T, n), 5.0, dtype=DT[out], device="cuda") for _ in range(p)]
    return xs, [v[0] for v in w], [v[1] for v in w], [v[2] for v in w], o


def check(xs, wd, out, group, parallel):
    y = [x.double() @ w.t() for x, w in zip(xs, wd)]
    mag = [x.double().abs() @ w.abs().t() for x, w in zip(xs, wd)]
    K = xs[0].shape[1]
    if parallel == "row":
        y, mag, K = [sum(y)] * len(xs), [sum(mag)] * len(xs), K * len(xs)
    half = torch.finfo(out[0].dtype).eps / 2
    for o, v, m in zip(out, y, mag):
        g = min(group, 128)
        bound = m * ((g + g // 16) * 2.0 ** -23 + (K // g + 8) * 2.0 ** -24)
        bound = bound + half * (v.abs() + bound)
        bad = (o.double() - v).abs() > bound
        assert not bool(bad.any()), f"{int(bad.sum())} of {bad.numel()}"


CASES = [
    # p, T, N, K, group
    (1, 1, 1, 32, 32), (1, 1, 16, 64, 64), (2, 3, 34, 256, 128), (4, 8, 100, 512, 64), (8, 1, 256, 2048, 128),
    (8, 5, 8, 256, 32), (2, 9, 50, 384, 64), (1, 16, 33, 640, 128), (4, 17, 20, 1024, 256), (2, 33, 18, 128, 32),
    (1, 70, 15, 224, 32), (64, 2, 64, 4096, 64), (3, 1, 3, 96, 32), (1, 4, 5000, 128, 128), (2, 2, 40, 1024, 512),
    (1, 1, 24000, 96, 32), (1, 3, 7, 8192, 128),
    # more blocks than SMs: the last ones in pieces
    (2, 9, 40100, 1024, 64), (1, 20, 38000, 640, 32), (4, 1, 39000, 2048, 128), (1, 40, 20000, 512, 64),
]


@pytest.mark.parametrize("p,T,N,K,group", CASES)
@pytest.mark.parametrize("parallel", ["row", "column"])
@pytest.mark.parametrize("out", ["fp32", "bf16"])
def test_linear(p, T, N, K, group, parallel, out):
    N = -(-N // p) * p
    xs, w, s, wd, o = make(p, T, N, K, group, parallel, out, seed=T + N + K)
    with SC.SimComm(p) as c:
        c.linear_w4(xs, w, s, o, parallel=parallel)
        torch.cuda.synchronize()
        assert c.async_error() == SC.OK
    check(xs, wd, o, group, parallel)
    if parallel == "row":
        assert all(torch.equal(o[0], v) for v in o)


@pytest.mark.parametrize("group", [32, 64, 128])
def test_every_weight_value_in_every_place(group):
    """One-hot tokens read the matrix back: W[n][k] itself, exactly (q - 8 times a power of two)."""
    K = 256
    q = torch.arange(16 * K, device="cuda").view(16, K).add(torch.arange(K, device="cuda") // 16).remainder(16)
    from test_gpu_moe_layer import pack4
    scale = torch.exp2(torch.arange(16 * (K // group), device="cuda").view(16, -1).remainder(5).float()).to(BF)
    out = [torch.empty(K, 16, device="cuda")]
    with SC.SimComm(1) as c:
        c.linear_w4([torch.eye(K, device="cuda", dtype=BF)], [pack4(q.to(torch.uint8))], [scale], out)
        torch.cuda.synchronize()
    want = (q.float() - 8) * scale.float().repeat_interleave(group, 1)
    assert torch.equal(out[0], want.t())


@pytest.mark.parametrize("group", [32, 64, 128])
def test_addresses_that_are_not_aligned(group):
    xs, w, s, wd, o = make(2, 5, 24, 512, group, "row", "fp32", offset=1)
    with SC.SimComm(2) as c:
        c.linear_w4(xs, w, s, o)
        torch.cuda.synchronize()
    check(xs, wd, o, group, "row")


def test_nan_and_inf_stay_in_their_token_and_row():
    xs, w, s, wd, o = make(1, 4, 32, 128, 32, "row", "fp32")
    xs[0][1, 7] = float("nan")
    s[0][9, 1] = float("inf")
    with SC.SimComm(1) as c:
        c.linear_w4(xs, w, s, o)
        torch.cuda.synchronize()
    fin = o[0].isfinite()
    assert not bool(fin[1].any()) and not bool(fin[:, 9].any())
    fin[1], fin[:, 9] = True, True
    assert bool(fin.all())


def test_rows_behind_the_last_token_are_left_alone_and_views_agree():
    p, T, N, K = 4, 3, 32, 512
    xs, w, s, wd, o = make(p, T, N, K, 64, "row", "bf16")
    big = [torch.full((T + 5, N), 9.0, dtype=BF, device="cuda") for _ in range(p)]
    with SC.SimComm(p) as c:
        c.linear_w4(xs, w, s, [b[:T] for b in big])
        torch.cuda.synchronize()
    assert all(bool((b[T:] == 9).all()) for b in big)
    with SC.SimComm(p, rank=2) as v:
        v.linear_w4(xs, w, s, [None, None, o[2], None])
        torch.cuda.synchronize()
    assert torch.equal(o[2], big[2][:T])
    xs, w, s, wd, o = make(p, T, N, K, 64, "column", "bf16")
    with SC.SimComm(p) as c:
        c.linear_w4(xs, w, s, o, parallel="column")
    with SC.SimComm(p, rank=3) as v:
        mine = torch.empty_like(o[3])
        v.linear_w4([None] * 3 + [xs[3]], [None] * 3 + [w[3]], [None] * 3 + [s[3]], [None] * 3 + [mine], parallel="column")
        torch.cuda.synchronize()
    check([xs[3]], [wd[3]], [mine], 64, "column")


def test_graph_and_stream():
    xs, w, s, wd, o = make(2, 2, 64, 512, 128, "row", "fp32")
    with SC.SimComm(2) as c:
        graph, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(graph, stream=st):
            c.linear_w4(xs, w, s, o)
        for x in xs:
            x.copy_(torch.randn_like(x))
        graph.replay()
        torch.cuda.synchronize()
        check(xs, wd, o, 128, "row")
        del graph
        o2 = [torch.empty_like(v) for v in o]
        st.wait_stream(torch.cuda.current_stream())
        c.linear_w4(xs, w, s, o2, stream=st)
        st.synchronize()
        assert torch.equal(o2[0], o[0])


def test_refusals():
    xs, w, s, wd, o = make(2, 4, 32, 256, 64, "row", "bf16")
    L = SC.load_library()
    with SC.SimComm(2) as c:
        with pytest.raises(SC.SimCommError, match="overlap"):
            c.linear_w4(xs, w, s, [o[0], o[0]])
        with pytest.raises(SC.SimCommError, match="overlap"):
            c.linear_w4([xs[0], o[1].view(-1)[:128].repeat(4).view(4, 128)], w, s,
                        [w[1].view(BF).view(-1)[:128].view(4, 32), o[1]])
        with pytest.raises(SC.SimCommError, match="power of two"):
            c.linear_w4(xs, w, [v[:, :1].expand(-1, 8).contiguous() for v in s], o)  # group 16
        with pytest.raises(ValueError):
            c.linear_w4(xs, w, [v[:, :1].expand(-1, 3).contiguous() for v in s], o)
        with pytest.raises(ValueError):
            c.linear_w4(xs, w, s, o, parallel="diagonal")
        with pytest.raises(SC.SimCommError) as e:
            c.linear_w4(xs, w, s, [torch.zeros(4, 32, dtype=torch.int32, device="cuda") for _ in range(2)])
        assert e.value.status == SC.UNSUPPORTED
        with pytest.raises(TypeError):
            c.linear_w4([x.float() for x in xs], w, s, o)
        args = lambda n, k, group, par=1: L.coll_linear_w4(  # noqa: E731
            c._h, None, None, None, 4, n, k, group, par, 2, None, None)
        assert args(32, 0, 32) == SC.INVALID_ARG and args(32, 1 << 25, 32) == SC.INVALID_ARG
        assert args(31, 64, 32, 0) == SC.INVALID_ARG and args(32, 96, 32) == SC.INVALID_ARG
        assert args(1 << 60, 64, 32) == SC.INVALID_ARG and args(32, 64, 32, 2) == SC.INVALID_ARG
        assert args(32, 64, 32) == SC.INVALID_ARG and b"null" in L.sim_comm_last_error()
        assert L.coll_linear_w4(c._h, None, None, None, 1 << 31, 32, 64, 32, 1, 2, None, None) == SC.INVALID_ARG
        assert b"int32" in L.sim_comm_last_error()
        n = c.launch_count()
        c.linear_w4([x[:0] for x in xs], w, s, [v[:0] for v in o])
        assert c.launch_count() == n
