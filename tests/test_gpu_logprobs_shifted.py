"""GPU test of the scores' gradient in rows that lie far from 0: adding a number to every score of a row changes no
probability, and none may be lost to the rounding of the row's lse.

Scores are multiples of 2^-6 within 8 of the shift, so that they stay the same numbers after it. With gl = 1 and no
token in reach the gradient is -P. P's relative error: an fp32 lse within 128 of 0 is off by at most 2^-18; where the
sum is taken again, ln of it (at most 16) by 2^-21 + 2^-22, the sum itself by 2^-22 + (V / 256 + 32) 2^-24, the
exponent's argument (at most 32 in powers of two) by 2^-20 ln 2 and the exponential by 2^-22.
"""
import pytest
import torch

from collective_communication_primitives_b200 import simcomm as SC
from test_gpu_logprobs import Call

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("p,V,offset", [(1, 1000, 0), (2, 5001, 0), (4, 50257, 3), (8, 131072, 0)])
def test_the_gradient_of_a_shifted_row_is_the_gradient_of_the_row(p, V, offset):
    shifts = [0.0, 90.0, -100.0, 127.0, 130.0, -140.0, 1000.0, -5000.0, 30000.0, -50000.0, 90000.0, 99990.0, -99990.0,
              110000.0]
    g = torch.Generator("cuda").manual_seed(V)
    base = torch.randint(-512, 513, (1, V), generator=g, device="cuda").float() / 64
    x = base + torch.tensor(shifts, device="cuda")[:, None]
    assert torch.equal(x.double() - torch.tensor(shifts, device="cuda").double()[:, None],
                       base.double().expand(len(shifts), V))
    R = len(shifts)
    ids = torch.zeros(R, dtype=torch.int32, device="cuda")
    a = Call(x, ids, p, offset=offset)
    with SC.SimComm(p) as c:
        a.run(c)
        gx = a.grad(c, torch.ones(R, device="cuda"))
        ge = a.grad(c, torch.zeros(R, device="cuda"), torch.ones(R, device="cuda"))
        torch.cuda.synchronize()
        assert c.async_error() == SC.OK
    prob = torch.softmax(base.double(), 1)
    got = torch.cat(gx, 1)[:, :V].double()
    assert bool((torch.cat(gx, 1)[:, V:] == 0).all())
    again = 2.0 ** -21 + 2.0 ** -22 + 2.0 ** -22 + (V / 256 + 32) * 2.0 ** -24 + 2.0 ** -20 * 0.7 + 2.0 ** -22
    for t, s in enumerate(shifts):
        bound = again + (2.0 ** -18 if abs(float(a.lse[0][t])) <= 128 else 0.0)
        off = ((got[t, 1:] + prob[0, 1:]).abs() / prob[0, 1:]).max()
        assert float(off) <= bound, (s, float(off), bound)
    # the entropy's gradient -P (ln P + H): ln P and H are off by the same absolute errors, H by its own sum's as well
    logp = prob.log()
    h = -(prob * logp).sum()
    want = -prob * (logp + h)
    got = torch.cat(ge, 1)[:, :V].double()
    for t, s in enumerate(shifts):
        rel = again + (2.0 ** -18 if abs(float(a.lse[0][t])) <= 128 else 0.0)
        bound = rel * want[0].abs() + prob[0] * (2 * rel + (logp[0].abs() + h) * 2.0 ** -21)
        assert bool(((got[t] - want[0]).abs() <= bound).all()), s


def test_bf16_rows_that_lie_far_out():
    """Multiples of 4 up to 32 below the shift 512 (of 16 below 2160) stay the same numbers in bf16; the gradient is
    rounded to it, and P may be off by 2^-14 within 2048."""
    V = 3001
    g = torch.Generator("cuda").manual_seed(1)
    small = -4.0 * torch.randint(0, 9, (1, V), generator=g, device="cuda").float()
    large = -16.0 * torch.randint(0, 4, (1, V), generator=g, device="cuda").float()
    base = torch.cat([small, small, small, large, large])
    shift = torch.tensor([0.0, 512.0, -256.0, 2160.0, 1100.0 // 16 * 16], device="cuda")[:, None]
    x = (base + shift).bfloat16()
    assert torch.equal(x.float() - shift, base)
    R = len(x)
    a = Call(x, torch.full((R,), -1, dtype=torch.int32, device="cuda"), 3)
    with SC.SimComm(3) as c:
        a.run(c)
        gx = a.grad(c, torch.zeros(R, device="cuda"), torch.ones(R, device="cuda"))
        torch.cuda.synchronize()
    got = torch.cat(gx, 1)[:, :V].double()
    prob = torch.softmax(base.double(), 1)
    logp = prob.log()
    h = -(prob * logp).sum(1, keepdim=True)
    want = -prob * (logp + h)
    for t in range(R):
        lost = 2.0 ** -17 + (2.0 ** -24 * abs(float(a.lse[0][t])) if abs(float(a.lse[0][t])) <= 2048 else 0.0)
        bound = 2.0 ** -8 * want[t].abs() + 1.01 * lost * prob[t] * (1 + logp[t].abs() + h[t])
        assert bool(((got[t] - want[t]).abs() <= bound).all()), t
