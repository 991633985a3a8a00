"""The adapters' fp32 results where k is far beyond 65,536: a warp's chain of matrix instructions ends as soon as for shorter
rows, and its sums are added up.

Tolerance: as for shorter rows, an addition of the matrix instruction cuts less than 2^-23 of the largest number in it,
and the numbers are of one sign: (32 + 3 R / 16) 2^-23 for a chain over 4,096 k's of a part (8 warps, 16 k's to an instruction) and the
second product. The K / 4096 parts are joined one after the other, or in groups: each addition rounds to nearest, by at most 2^-24 of
the sum so far, which is i / n of the whole after i of n equal parts. Roundings of one kind to either side add up as their squares:
2^-24 sqrt(n / 3) for one result, and the norm of all results' errors over the results' norm is as large; four times that is granted, and
eight roundings of 2^-24 for the rest. A chain over K / 16 k's would cut up to K / 65536 32 2^-23."""
import math

import pytest
import torch

from collective_communication_primitives_b200 import simcomm as SC

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.mark.parametrize("parallel", ["row", "column"])
@pytest.mark.parametrize("T,K,R", [(2, 1 << 22, 16), (3, (1 << 21) + 2 * 5, 16), (70, 1 << 21, 16), (5, 1 << 17, 40), (530, 1 << 17, 64)])
def test_fp32_results_of_long_rows(T, K, R, parallel):
    p, N = 2, 64
    g = torch.Generator("cuda").manual_seed(T + K + R)
    rand = lambda *s: (torch.rand(*s, generator=g, device="cuda") + 0.5).to(BF)  # noqa: E731  (of one sign: nothing cancels)
    X, A, B = rand(T, K), rand(1, R, K), rand(1, N, R)
    if parallel == "row":
        cut = lambda t, d: [c.contiguous() for c in t.chunk(p, d)]  # noqa: E731
        x, a, b = cut(X, 1), cut(A, 2), [B] * p
        out = [torch.empty(T, N, device="cuda") for _ in range(p)]
    else:
        x, a, b = [X] * p, [A] * p, [c.contiguous() for c in B.chunk(p, 1)]
        out = [torch.empty(T, N // p, device="cuda") for _ in range(p)]
    ad = torch.zeros(T, dtype=torch.int32, device="cuda")
    with SC.SimComm(p) as c:
        c.adapters(x, ad, a, b, out, parallel=parallel)
        torch.cuda.synchronize()
        assert c.async_error() == 0
    got = out[0] if parallel == "row" else torch.cat(out, 1)
    u = sum(X[:, k:k + (1 << 18)].double() @ A[0, :, k:k + (1 << 18)].double().T for k in range(0, K, 1 << 18))
    want = u @ B[0].double().T
    off = ((got.double() - want).norm() / want.norm()).item()
    assert off <= (32 + 3 * R / 16) * 2 ** -23 + (4 * math.sqrt(K / 4096 / 3) + 8) * 2 ** -24, off
