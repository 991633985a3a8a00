"""GPU tests of what the expert layer keeps of the values between its two products, h = silu(g) u.

h goes into the second product in two bf16 parts: its rounding (half a step: 2^-8 of it) and the rounding of what that
left out (2^-8 of the first error), so 2^-16 of h is lost; the exponential, quotient and product take 2^-20 of it. The
first sum's error is H 2^-23 of its terms' magnitudes, passed on with |silu'| <= 1.1; the second has 2 F terms. Sizes
are small, so that these bounds stay far below the 2^-8 of h that one part would lose: where a row's terms cancel,
h in one part is out of bounds.
"""
import pytest
import torch

from collective_communication_primitives_b200 import simcomm as SC
from test_gpu_moe_layer import Layer

pytestmark = pytest.mark.gpu


def bounds(a, lost_of_h):
    """Expected output in 64 bits and its bound, with h off by lost_of_h of itself."""
    p, T, k, H, F = a.p, a.T, a.k, a.H, a.F
    x, idx, w = torch.cat(a.x).double(), torch.cat(a.idx).long(), torch.cat(a.w).double()
    want = torch.zeros(p * T, H, dtype=torch.float64, device="cuda")
    mag, slack = torch.zeros_like(want), torch.zeros_like(want)
    for e in torch.unique(idx).tolist():
        t, s = torch.nonzero(idx == e, as_tuple=True)
        up, down = a.upd[e], a.downd[e]
        v, vm = x[t] @ up.t(), x[t].abs() @ up.abs().t()
        gate, u = v[:, :F], v[:, F:]
        silu = gate * torch.sigmoid(gate)
        h = silu * u
        dh = H * 2.0 ** -23 * (1.1 * u.abs() * vm[:, :F] + silu.abs() * vm[:, F:]) + h.abs() * (lost_of_h + 2.0 ** -20)
        y, ws = h @ down.t(), w[t, s][:, None]
        want.index_add_(0, t, ws * y)
        mag.index_add_(0, t, ws.abs() * y.abs())
        slack.index_add_(0, t, ws.abs() * ((dh + 2 * F * 2.0 ** -23 * h.abs()) @ down.abs().t()))
    bound = slack + (k + 2) * 2.0 ** -24 * mag
    return want, bound + 2.0 ** -8 * (want.abs() + bound)


@pytest.mark.parametrize("p,T,E,k,H,F,group,tensor", [
    (1, 7, 4, 2, 64, 32, 0, 0), (1, 7, 4, 2, 64, 32, 0, 1), (2, 20, 4, 1, 64, 96, 0, 0), (2, 20, 4, 1, 64, 96, 0, 1),
    (2, 64, 4, 2, 40, 200, 0, 1), (1, 5, 4, 2, 33, 17, 0, 0), (1, 70, 4, 1, 31, 45, 0, 0), (1, 300, 2, 1, 32, 64, 0, 1),
    (1, 7, 4, 2, 64, 32, 32, -1), (2, 20, 4, 1, 64, 96, 32, -1), (2, 40, 8, 3, 64, 128, 64, -1),
    (1, 90, 4, 2, 128, 128, 128, -1)])
def test_h_keeps_sixteen_bits(p, T, E, k, H, F, group, tensor):
    a = Layer(p, T, E, k, H, F, group, residual=False, seed=T + H)
    with SC.SimComm(p) as c:
        c.set_option("moe_layer_tensor", tensor)
        a.run(c)
        torch.cuda.synchronize()
        assert c.async_error() == SC.OK
    want, bound = bounds(a, 2.0 ** -16)
    off = (torch.cat(a.out).double() - want).abs()
    assert bool((off <= bound).all()), float((off / bound).max())


def test_infinite_h_stays_infinite():
    """A second part of infinity minus infinity would turn it into NaN."""
    a = Layer(1, 3, 2, 1, 8, 8, residual=False, idx=torch.zeros(1, 3, 1, device="cuda"))
    for tensor in (0, 1):
        a.x[0][1] = 3e38
        a.up[0][0].fill_(1.0)
        a.down[0][0].fill_(1.0)
        a.w[0].fill_(1.0)
        with SC.SimComm(1) as c:
            c.set_option("moe_layer_tensor", tensor)
            a.run(c)
            torch.cuda.synchronize()
        assert bool((a.out[0][1] == float("inf")).all()) and bool(a.out[0][[0, 2]].isfinite().all())
