"""The adapters' fp32 results against float64, beside those of fp32 sums: A x goes into the second product in three bf16 parts
(2^-24 of it is lost), and no warp's chain of matrix instructions is longer than 4,096 k's.

Tolerance: an addition of the matrix instruction cuts less than 2^-23 of the largest number in it. A chain over K / 128 k's of a
warp, at most 32 additions, and one over 3 R / 16 each cut that much of their sums at most, always to the same side; the
results add up to numbers as large as their parts, so that the relative error of all results together is at most the sum of the cuts,
(32 + 3 R / 16) 2^-23, and a few roundings of 2^-24. In two parts the loss alone is up to 2^-17 of every term."""
import pytest
import torch

from collective_communication_primitives_b200 import simcomm as SC

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.mark.parametrize("parallel", ["row", "column"])
@pytest.mark.parametrize("T,K,R", [(1, 8192, 16), (40, 4096, 64), (300, 8192, 16), (300, 8192, 64), (300, 512, 256), (600, 8196, 40),
                                   (2000, 2048, 64)])
def test_fp32_results_are_as_exact_as_fp32_sums(T, K, R, parallel):
    p, S, N = 2, 3, 128
    g = torch.Generator("cuda").manual_seed(T + K + R)
    rand = lambda *s: (torch.rand(*s, generator=g, device="cuda") + 0.5).to(BF)  # noqa: E731  (of one sign: nothing cancels)
    X, A, B = rand(T, K), rand(S, R, K), rand(S, N, R)
    if parallel == "row":
        cut = lambda t, d: [c.contiguous() for c in t.chunk(p, d)]  # noqa: E731
        x, a, b = cut(X, 1), cut(A, 2), [B] * p
        out = [torch.empty(T, N, device="cuda") for _ in range(p)]
    else:
        x, a, b = [X] * p, [A] * p, [c.contiguous() for c in B.chunk(p, 1)]
        out = [torch.empty(T, N // p, device="cuda") for _ in range(p)]
    ad = torch.randint(0, S, (T,), generator=g, dtype=torch.int32, device="cuda")
    with SC.SimComm(p) as c:
        c.adapters(x, ad, a, b, out, parallel=parallel)
        torch.cuda.synchronize()
        assert c.async_error() == 0
    got = out[0] if parallel == "row" else torch.cat(out, 1)
    want = torch.empty(T, N, dtype=torch.float64, device="cuda")
    for e in range(S):
        m = ad == e
        want[m] = X[m].double() @ A[e].double().T @ B[e].double().T
    off = ((got.double() - want).norm() / want.norm()).item()
    assert off <= (32 + 3 * R / 16) * 2 ** -23 + 8 * 2 ** -24, off
