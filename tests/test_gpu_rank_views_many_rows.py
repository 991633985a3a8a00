"""The norm of many long rows on rank views: rows of all ranks come through the ring of bulk copies, the peers' from their
mappings. Outputs are the whole communicator's bits."""
import pytest

from test_gpu_rank_views import _setup, _spawn

pytestmark = pytest.mark.gpu


def _norm(rank, world, port, case, q):
    try:
        _setup(rank, world, port, 60)
        import torch
        import torch.distributed as dist

        from collective_communication_primitives_b200 import ranks
        from collective_communication_primitives_b200 import simcomm as SC
        from test_gpu_rank_views_operators import Shared
        from test_gpu_rmsnorm import Back, EPS, Norm
        T, H, dt, group = case
        comm, whole = ranks.RankComm(), SC.SimComm(world)
        kept = []

        def shared(ts):
            kept.append(Shared(comm, ranks, ts[rank]))
            return kept[-1].all

        def fresh(ts):
            return [torch.full_like(t, 3) if r == rank else None for r, t in enumerate(ts)]

        a, b = Norm(world, T, H, dt, True, group, seed=T), Back(world, T, H, dt, seed=T)
        a.run(whole)
        b.run(whole)
        total, y, gx, gw = fresh(a.total), fresh(a.y), fresh(b.gx), fresh(b.gw)
        qs = {"q": fresh(a.q), "scale": fresh(a.scale)} if group else {}
        comm.rmsnorm(shared(a.x), a.w, EPS, out=y, residual=a.res, total=total, **qs)
        comm.rmsnorm_backward(shared(b.gy), b.h, b.w, EPS, gx, grad_total=b.past, grad_weight=gw)
        torch.cuda.synchronize()
        for got, want in [(total, a.total), (y, a.y), (gx, b.gx), (gw, b.gw)] + ([(qs["q"], a.q), (qs["scale"], a.scale)] if group else []):
            assert torch.equal(got[rank].view(torch.uint8), want[rank].view(torch.uint8)), f"rank {rank} differs"
        assert comm.async_error() == 0 and whole.async_error() == 0
        whole.close()
        comm.sync()
        comm.close()
        dist.barrier()
        for s in kept:
            s.buf.close()
        dist.destroy_process_group()
        q.put((rank, "ok"))
    except Exception as e:  # reported to the parent
        import traceback
        q.put((rank, f"{type(e).__name__}: {e}\n{traceback.format_exc()}"))


@pytest.mark.parametrize("case", [(700, 4096, "bf16", 128), (601, 4100, "fp32", 0), (597, 8192, "bf16", 8192)])
def test_many_rows(case):
    res, codes = _spawn(_norm, 2, case)
    assert [res.get(r) for r in range(2)] == ["ok", "ok"], res
    assert codes == [0, 0]
