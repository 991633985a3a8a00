"""GPU tests of the expert layer where experts with few and with many assignments meet in one call, so that a CTA has
units of 8, 16 and 32 tokens one after the other, in both products, at row lengths whose panels do not come out even
(the bounds are those of test_gpu_moe_layer)."""
import pytest
import torch

from collective_communication_primitives_b200 import simcomm as SC
from test_gpu_moe_layer import Layer

pytestmark = pytest.mark.gpu

COUNTS = [9, 1, 17, 8, 2, 33, 7, 16, 65, 3, 32, 5]


def _mixed(p, E, H, F, group, back=False, seed=0):
    """One slot per token; expert e has COUNTS[e % 12] assignments (from the last expert on with `back`), their tokens in
    no order over the ranks."""
    counts = [COUNTS[e % len(COUNTS)] for e in range(E)]
    ids = torch.repeat_interleave(torch.arange(E), torch.tensor(counts[::-1] if back else counts))
    ids = ids[:len(ids) // p * p]
    ids = ids[torch.randperm(len(ids), generator=torch.Generator().manual_seed(seed))].cuda()
    return Layer(p, len(ids) // p, E, 1, H, F, group, seed=seed + H + F, idx=ids.view(p, -1, 1))


# (H, F): panels of 1024, 512 and 256 k's in numbers that are no multiple of 4, or are in one product only. With 36 or
# more experts each product has several units to a CTA.
SHAPES = [(1024, 1536, 0), (1024, 1536, 32), (1536, 1024, 64), (1024, 1024, 128), (2880, 1024, 64), (2560, 1536, 128),
          (5120, 1024, 128), (1024, 7168, 64), (2048, 1024, 32), (1024, 2048, 128), (512, 640, 128), (352, 416, 32)]


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("H,F,group", SHAPES)
def test_few_and_many_assignments_in_one_call(H, F, group, back):
    a = _mixed(2, 36, H, F, group, back)
    with SC.SimComm(2) as c:
        c.set_option("moe_layer_tensor", 0)
        a.run(c)
        torch.cuda.synchronize()
        assert c.async_error() == SC.OK
        a.check()
        first = [o.clone() for o in a.out]
        for _ in range(8):
            for o in a.out:
                o.fill_(3.0)
            a.run(c)
            torch.cuda.synchronize()
            assert all(torch.equal(x, y) for x, y in zip(first, a.out))


@pytest.mark.parametrize("group", [0, 32, 64, 128])
def test_counts_around_the_token_tiles_in_four_bits(group):
    """Experts with 1, 8, 9, 16, 17, 32, 33 and 65 assignments in one call, in no order."""
    counts = [1, 8, 9, 16, 17, 32, 33, 65]
    ids = torch.repeat_interleave(torch.arange(8), torch.tensor(counts))
    ids = ids[torch.randperm(len(ids), generator=torch.Generator().manual_seed(1))].cuda()
    a = Layer(1, len(ids), 8, 1, 1024, 640, group, seed=5, idx=ids.view(1, -1, 1))
    with SC.SimComm(1) as c:
        for _ in range(3):
            a.run(c)
            torch.cuda.synchronize()
            a.check()


@pytest.mark.parametrize("group", [0, 64])
def test_skewed_picks(group):
    """Tokens that pick by Zipf's law: one expert with hundreds of assignments, many with one or none."""
    p, T, E, k = 4, 96, 64, 4
    share = 1.0 / torch.arange(1, E + 1, dtype=torch.float64) ** 1.1
    g = torch.Generator().manual_seed(3)
    idx = torch.multinomial(share.expand(p * T, E), k, generator=g).view(p, T, k).cuda()
    a = Layer(p, T, E, k, 1024, 1536, group, seed=12, idx=idx)
    with SC.SimComm(p) as c:
        for _ in range(2):
            a.run(c)
            torch.cuda.synchronize()
            assert c.async_error() == SC.OK
            a.check()
