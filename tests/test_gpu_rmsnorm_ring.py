"""The norm's ring in shared memory in the cases where it could go wrong: the residual in place, where the copying warp reads
later rows of the buffer that other rows of the same launch are written to, and rows whose squares pass fp32 between others. Rows
are long and many enough for the ring (16-byte vectors, 512 of them or more, twice as many rows as CTAs), with a vector, two and
four to a thread, and each CTA has several."""
import pytest
import torch

from collective_communication_primitives_b200 import simcomm as SC
from test_gpu_rmsnorm import Norm

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("p,T,H,dtype", [(2, 900, 4096, "bf16"), (2, 2100, 2048, "fp32"), (3, 700, 8192, "bf16"), (1, 1500, 16384, "bf16"),
                                         (2, 1000, 5120, "bf16"), (8, 1201, 4096, "bf16")])
@pytest.mark.parametrize("q", [False, True])
def test_residual_in_place(p, T, H, dtype, q):
    with SC.SimComm(p) as c:
        for rank in {0, p - 1}:
            a = Norm(p, T, H, dtype, True, 128 if q else 0, seed=2)
            res = a.res.clone()
            a.total[rank].copy_(a.res)
            kw = {"q": a.q, "scale": a.scale} if q else {}
            c.rmsnorm(a.x, a.w, 1e-5, out=a.y, residual=a.total[rank], total=a.total, **kw)
            torch.cuda.synchronize()
            assert c.async_error() == SC.OK
            a.check(res)
            first = [v.clone() for v in a.total + a.y]
            a.total[rank].copy_(res)
            c.rmsnorm(a.x, a.w, 1e-5, out=a.y, residual=a.total[rank], total=a.total, **kw)
            torch.cuda.synchronize()
            assert all(torch.equal(u, v) for u, v in zip(first, a.total + a.y))


@pytest.mark.parametrize("H", [2048, 4096, 8192])
def test_huge_rows_among_others(H):
    """Every third row times 2^70, whose squares pass fp32: scaled by 2^-80 they are the same rows times 2^-10. With an eps that both
    lose beside mean h^2 every step is the same but for powers of two, so all bits are: of the norm, of the gradient, 2^-70 of the other
    one's, and of the weight's gradient."""
    T, eps = 1200, 1e-37
    g = torch.Generator("cuda").manual_seed(H)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x, w, gy = rn(T, H), 1 + 0.3 * rn(H), rn(T, H)
    scale = torch.where(torch.arange(T, device="cuda") % 3 == 1, 2.0 ** 70, 1.0)[:, None]
    got = []
    with SC.SimComm(1) as c:
        for h in (x, x * scale):
            y, gx, gw = torch.empty_like(x), torch.empty_like(x), torch.empty(H, device="cuda")
            c.rmsnorm([h], w, eps, out=[y])
            c.rmsnorm_backward([gy], h, w, eps, [gx], grad_weight=[gw])
            torch.cuda.synchronize()
            assert c.async_error() == SC.OK
            got.append((y, gx, gw))
    (y0, gx0, gw0), (y1, gx1, gw1) = got
    assert torch.equal(y0, y1)
    assert torch.equal(gx0, gx1 * scale)
    assert torch.equal(gw0, gw1)
