"""The distillation's loss at temperatures that are no power of two. With one place the teacher has q = 1, and a row whose second
score lies D below the first has loss D / temperature + ln(1 + e^(-D / temperature)); from D / temperature = 64 on the second
term is below 2^-92 and the loss is D / temperature.

Tolerance: places are done in 64 bits (a reciprocal, a product, a logarithm of a sum that is 1 and differences: 8 steps of 2^-53
of the result), and the result is rounded once, by half a step of fp32: 2^-24 of it. 1 / temperature in fp32 alone would be off by as much again."""
import pytest
import torch

from collective_communication_primitives_b200 import simcomm as SC

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("p", [1, 2])
@pytest.mark.parametrize("temperature", [0.1, 0.3, 0.7, 1.0, 1.1, 1.7, 2.0, 3.0, 4.7, 0.0123, 47.3, 6.1e5, 3.3e-20])
def test_distance_over_temperature(temperature, p):
    g = torch.Generator("cuda").manual_seed(3)
    R = 500
    D = ((64 + 64 * torch.rand(R, generator=g, device="cuda")) * temperature).float()
    x = torch.zeros(R, 2, device="cuda")
    x[:, 1] = -D
    idx = torch.ones(R, 1, dtype=torch.int32, device="cuda")
    value = torch.randn(R, 1, generator=g, device="cuda")
    loss = [torch.empty(R, device="cuda") for _ in range(p)]
    with SC.SimComm(p) as c:
        c.distill([v.contiguous() for v in x.chunk(p, 1)], 2, idx, value, loss, temperature=temperature)
        torch.cuda.synchronize()
        assert c.async_error() == 0
    want = D.double() / torch.tensor(temperature, dtype=torch.float32).double().item()
    off = ((loss[0].double() - want).abs() / want).max().item()
    assert off <= 2 ** -24 + 2 ** -49, off * 2 ** 24
