"""The operators of a model's step on rank views, every rank its own process with its own CUDA context on one GPU: the
row-parallel 4-bit linear, the expert layer and the log probabilities with their gradient read the peers' weights and
scores through IPC mappings. Every rank regenerates every rank's inputs from seeds and runs the whole communicator on its
own copies; its view's outputs are the same bits. No kernel waits on another process: the ranks meet only at host
barriers between calls."""
import pytest

from test_gpu_rank_views import _setup, _spawn

pytestmark = pytest.mark.gpu


class Shared:
    """This rank's tensor in registered memory: `all` has the peers' pointers and this rank's tensor."""

    def __init__(self, comm, ranks, t):
        self.buf = ranks.SharedBuffer(max(4, -(-t.numel() * t.element_size() // 4) * 4))
        raw = self.buf.view("int32").view(t.dtype)
        self.mine = raw[:t.numel()].view(t.shape)
        self.mine.copy_(t)
        self.all = comm.register(self.buf)
        self.all[comm.rank] = self.mine


def _ops(rank, world, port, case, q):
    try:
        _setup(rank, world, port, 60)
        import torch
        import torch.distributed as dist

        from collective_communication_primitives_b200 import ranks
        from collective_communication_primitives_b200 import simcomm as SC
        from test_gpu_linear_w4 import make
        from test_gpu_moe_layer import Layer
        p = world
        comm, whole = ranks.RankComm(), SC.SimComm(p)
        kept = []

        def shared(ts):
            kept.append(Shared(comm, ranks, ts[rank]))
            return kept[-1].all

        def own(ts):
            return None if ts is None else [t if r == rank else None for r, t in enumerate(ts)]

        def fresh(ts):
            return [torch.full_like(t, 3) if r == rank else None for r, t in enumerate(ts)]

        def same(name, got, want):
            torch.cuda.synchronize()
            assert torch.equal(got[rank].view(torch.uint8), want[rank].view(torch.uint8)), f"{name}: rank {rank} differs"

        if case == "linear":
            for T, N, K, group, out in ((1, 200, 64 * p, 32, "bf16"), (5, 4096, 256 * p, 64, "fp32"),
                                        (40, 333, 128 * p, 128, "fp32")):
                xs, w, s, _, o = make(p, T, N, K, group, "row", out, seed=T)
                whole.linear_w4(xs, w, s, o, parallel="row")
                got = fresh(o)
                comm.linear_w4(shared(xs), shared(w), shared(s), got, parallel="row")
                same("row", got, o)
                xs, w, s, _, o = make(p, T, 64 * p, K, group, "column", out, seed=T)
                whole.linear_w4(xs, w, s, o, parallel="column")
                got = fresh(o)
                comm.linear_w4(own(xs), own(w), own(s), got, parallel="column")
                same("column", got, o)
        elif case == "layer":
            # few k's: no sum is split, whatever the number of assignments
            for T, k, H, F, group, tensor in ((1, 2, 32, 32, 0, 0), (9, 3, 32, 24, 0, 0), (20, 2, 64, 64, 0, 1),
                                              (7, 2, 128, 64, 32, -1), (30, 1, 128, 128, 128, -1)):
                a = Layer(p, T, 4 * p, k, H, F, group, seed=T)
                whole.set_option("moe_layer_tensor", tensor)
                comm.set_option("moe_layer_tensor", tensor)
                a.run(whole)
                got = fresh(a.out)
                sc = {"up_scale": shared(a.us), "down_scale": shared(a.ds)} if group else {}
                s = torch.cuda.Stream()  # a stream of the caller's
                s.wait_stream(torch.cuda.current_stream())
                comm.moe_layer(own(a.x), own(a.idx), own(a.w), a.E, shared(a.up), shared(a.down), got,
                               residual=own(a.res), stream=s, **sc)
                same("expert layer", got, a.out)
                a.check()
        else:
            for R, V, dt, n in ((3, 1000 * p + 1, torch.float32, 4), (40, 777, torch.bfloat16, 0),
                                (700, 129, torch.float32, 1)):
                g = torch.Generator("cuda").manual_seed(R)
                m = -(-V // p)
                logits = [3 * torch.randn(R, m, generator=g, device="cuda") for _ in range(p)]
                logits = [x.to(dt) for x in logits]
                tokens = torch.randint(-1, V, (R,), generator=g, device="cuda", dtype=torch.int32)
                f = [[torch.empty(R, device="cuda") for _ in range(p)] for _ in range(3)]
                ti = [torch.empty(R, n, dtype=torch.int32, device="cuda") for _ in range(p)] if n else None
                tl = [torch.empty(R, n, device="cuda") for _ in range(p)] if n else None
                whole.logprobs(logits, tokens, V, *f, ti, tl)
                all_ = shared(logits)
                got = [fresh(x) for x in f]
                gi, gl = (fresh(ti), fresh(tl)) if n else (None, None)
                comm.logprobs(all_, tokens, V, *got, gi, gl)
                for x, y in zip(got + ([gi, gl] if n else []), f + ([ti, tl] if n else [])):
                    same("log probabilities", x, y)
                gp, ge = torch.randn(R, generator=g, device="cuda"), torch.randn(R, generator=g, device="cuda")
                dx = [torch.empty_like(x) for x in logits]
                whole.logprobs_backward(logits, tokens, V, f[2], gp, dx, entropy=f[1], grad_entropy=ge)
                gx = fresh(dx)
                comm.logprobs_backward(all_, tokens, V, got[2], gp, gx, entropy=got[1], grad_entropy=ge)
                same("gradient", gx, dx)
        assert comm.async_error() == 0 and whole.async_error() == 0
        whole.close()
        comm.sync()
        comm.close()
        dist.barrier()
        for b in kept:
            b.buf.close()
        dist.destroy_process_group()
        q.put((rank, "ok"))
    except Exception as e:  # reported to the parent
        import traceback
        q.put((rank, f"{type(e).__name__}: {e}\n{traceback.format_exc()}"))


@pytest.mark.parametrize("case", ["linear", "layer", "log probabilities"])
@pytest.mark.parametrize("world", [2, 3])
def test_operators_match_the_whole_communicator(world, case):
    res, codes = _spawn(_ops, world, case)
    assert all(v == "ok" for v in res.values()), res
    assert codes == [0] * world
