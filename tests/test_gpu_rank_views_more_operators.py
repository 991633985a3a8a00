"""The norm, the adapters, the score adjustment and the distillation on rank views, every rank its own process with its own
CUDA context on one GPU: what they read of the peers' rows, tokens, adapters and scores comes through IPC mappings. Every
rank regenerates every rank's inputs from seeds and runs the whole communicator on its own copies; its view's outputs are
the same bits. No kernel waits on another process: the ranks meet only at host barriers between calls."""
import pytest

from test_gpu_rank_views import _setup, _spawn

pytestmark = pytest.mark.gpu


def _ops(rank, world, port, case, q):
    try:
        _setup(rank, world, port, 60)
        import torch
        import torch.distributed as dist

        from collective_communication_primitives_b200 import ranks
        from collective_communication_primitives_b200 import simcomm as SC
        from test_gpu_adapters import Adapted
        from test_gpu_adjust_logits import Adjust
        from test_gpu_distill import Distill, make
        from test_gpu_rank_views_operators import Shared
        from test_gpu_rmsnorm import Back, EPS, Norm
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
            assert torch.equal(got[rank].contiguous().view(torch.uint8), want[rank].contiguous().view(torch.uint8)), \
                f"{name}: rank {rank} differs"

        if case == "norm":
            for T, H, dt, group in ((1, 4096, "bf16", 0), (9, 1001, "fp32", 1001), (5, 512, "bf16", 128), (2, 20000, "fp32", 32)):
                a = Norm(p, T, H, dt, True, group, seed=T)
                a.run(whole)
                total, y = fresh(a.total), fresh(a.y)
                qs = {"q": fresh(a.q), "scale": fresh(a.scale)} if group else {}
                comm.rmsnorm(shared(a.x), a.w, EPS, out=y, residual=a.res, total=total, **qs)
                same("total", total, a.total)
                same("norm", y, a.y)
                if group:
                    same("8-bit rows", qs["q"], a.q)
                    same("scales", qs["scale"], a.scale)
                b = Back(p, T, H, dt, seed=T)
                b.run(whole)
                gx, gw = fresh(b.gx), fresh(b.gw)
                s = torch.cuda.Stream()  # a stream of the caller's
                s.wait_stream(torch.cuda.current_stream())
                comm.rmsnorm_backward(shared(b.gy), b.h, b.w, EPS, gx, grad_total=b.past, grad_weight=gw, stream=s)
                same("gradient", gx, b.gx)
                same("weight's gradient", gw, b.gw)
        elif case == "adapters":
            for T, N, K, R, par in ((3, 8 * p, 32 * p, 16, "row"), (70, 10 * p, 24 * p, 20, "row"), (5, 6 * p, 64 * p, 8, "column"),
                                    (600, 16 * p, 8 * p, 64, "row")):
                a = Adapted(p, T, N, K, 4, R, par, "fp32", "bf16", seed=T, whole=False)
                a.run(whole)
                got = fresh(a.out)
                read = shared if par == "row" else own
                comm.adapters(read(a.x), a.ad, read(a.a), own(a.b), got, base=own(a.base), scale=a.sc, parallel=par)
                same(par, got, a.out)
        elif case == "adjust":
            for R, V, dt in ((3, 1000 * p + 1, "fp32"), (7, 333, "bf16")):
                a = Adjust(p, R, V, dt, 40, 6, True, seed=R)
                a.run(whole)
                got = [o.clone().fill_(11) if r == rank else None for r, o in enumerate(a.out)]
                comm.adjust_logits(own(a.logits), V, got, **a.kw)
                same("scores", got, a.out)
        else:
            for R, V, n, dt, tail in ((3, 20000 * p + 1, 32, "fp32", True), (40, 777, 5, "bf16", False)):
                x, idx, val = make(R, V, n, dt, R, tail)
                a = Distill(x, idx, val, p, 1.0, tail)
                g = torch.rand(R, device="cuda", generator=torch.Generator("cuda").manual_seed(R))
                a.run(whole)
                a.grad(whole, g)
                loss, st, gx = fresh(a.loss), fresh(a.stats), fresh(a.gx)
                comm.distill(shared(a.logits), V, a.idx, a.val, loss, stats=st, tail=tail)
                same("loss", loss, a.loss)
                same("stats", st, a.stats)
                comm.distill_backward(own(a.logits), V, a.idx, a.val, st, g, gx, tail=tail)
                same("gradient", gx, a.gx)
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


@pytest.mark.parametrize("case", ["norm", "adapters", "adjust", "distill"])
@pytest.mark.parametrize("world", [2, 3])
def test_operators_match_the_whole_communicator(world, case):
    res, codes = _spawn(_ops, world, case)
    assert all(v == "ok" for v in res.values()), res
    assert codes == [0] * world
