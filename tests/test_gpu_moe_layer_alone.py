"""GPU test that a token's result in the expert layer does not depend on the other tokens of the call: the same bits
whatever experts they pick, how many of them pick its own, and where in the call it stands."""
import pytest
import torch

from collective_communication_primitives_b200 import simcomm as SC
from test_gpu_moe_layer import Layer

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("group,tensor", [(0, 0), (0, 1), (32, -1), (64, -1), (128, -1)])
@pytest.mark.parametrize("T,E,k,H,F", [(8, 16, 2, 1024, 640), (40, 8, 2, 640, 1024), (70, 40, 3, 512, 384),
                                       (200, 4, 2, 384, 512)])
def test_other_tokens_do_not_matter(T, E, k, H, F, group, tensor):
    a = Layer(1, T, E, k, H, F, group, seed=T)
    g = torch.Generator().manual_seed(2)
    results = []
    with SC.SimComm(1) as c:
        c.set_option("moe_layer_tensor", tensor)
        x, ids, w, res = a.x[0][0].clone(), a.idx[0][0].clone(), a.w[0][0].clone(), a.res[0][0].clone()
        mine = set(ids.tolist())
        apart = [e for e in range(E) if e not in mine]
        for others in ("as they are", "all on the token's experts", "none of them there", "one expert", "any"):
            for t in range(T):
                if others == "all on the token's experts":
                    a.idx[0][t] = ids
                elif others == "none of them there":
                    a.idx[0][t] = torch.tensor([apart[i % len(apart)] for i in range(t, t + k)])
                elif others == "one expert":
                    a.idx[0][t] = apart[0]
                elif others == "any":
                    a.idx[0][t] = torch.randperm(E, generator=g)[:k]
            at = {"as they are": 0, "any": T // 2}.get(others, T - 1)
            a.x[0][at], a.idx[0][at], a.w[0][at], a.res[0][at] = x, ids, w, res
            a.run(c)
            torch.cuda.synchronize()
            assert c.async_error() == SC.OK
            results.append(a.out[0][at].clone())
    assert all(torch.equal(r, results[0]) for r in results), [torch.equal(r, results[0]) for r in results]
