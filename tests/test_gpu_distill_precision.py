"""The distillation's loss with the class of the rest, where the teacher's probabilities are the student's in another order: the
loss is a small difference of large terms, and an error of the scores' sum must not show in it.

Tolerance: the sum over the columns that are not listed is off by less than 2^-16 of it (an exponential by 2^-22 and its
argument, at most 32, by 2^-24 of it, and a thread's chain of at most 256 additions by 2^-24 each). All other arithmetic is in
64 bits, so that this error enters ln P of the listed columns times P_rest and the rest's class times Q with the other sign:
2^-16 |P_rest - Q|, which is 2^-20 or less here but for the values' rounding; the result is rounded by 2^-24 of it."""
import pytest
import torch

from collective_communication_primitives_b200 import simcomm as SC

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("R,V,n,spread", [(64, 32374, 6, 2.5), (5, 131072, 32, 1.0), (700, 5000, 100, 2.0), (3, 1001, 2, 5.0)])
def test_a_permuted_teacher(R, V, n, spread, dtype):
    p = 2
    g = torch.Generator("cuda").manual_seed(V + n)
    x = (spread * torch.randn(R, p * -(-V // p), generator=g, device="cuda")).to(dtype)
    logits = [c.contiguous() for c in x.chunk(p, 1)]
    X = x[:, :V].double()
    lse = torch.logsumexp(X, 1, keepdim=True)
    best = torch.topk(X, n, 1)
    idx, value = best.indices.int(), (best.values - lse).roll(1, 1).float().contiguous()
    loss = [torch.empty(R, device="cuda") for _ in range(p)]
    with SC.SimComm(p) as c:
        c.distill(logits, V, idx, value, loss, tail=True)
        torch.cuda.synchronize()
        assert c.async_error() == 0
    v = value.double()
    q = v.exp()
    Q = 1 - q.sum(1)
    rest = torch.logsumexp(X.scatter(1, idx.long(), float("-inf")), 1, keepdim=True) - lse
    want = (q * (v - (best.values - lse))).sum(1) + Q * (Q.log() - rest[:, 0])
    bound = 2 ** -16 * (rest[:, 0].exp() - Q).abs() + 2 ** -23 * want.abs() + 2 ** -40
    off = (loss[0].double() - want).abs()
    assert (off <= bound).all(), (off / bound).max().item()
