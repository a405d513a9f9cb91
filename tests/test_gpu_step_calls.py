"""Calls of the training step's operators that a program makes around them: sums of
balance losses in place."""
import pytest
import torch

from mxcheck import ensure_built

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def mx():
    ensure_built()
    import mxfp8_block_scaled_mx_gb300 as mx
    return mx


def randn(*shape, seed, dtype=FP32):
    return torch.randn(shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda").to(dtype)


@pytest.mark.parametrize("tokens", [40, 3000])
def test_balance_losses_added_in_place(mx, tokens):
    layers = [randn(tokens, 24, seed=s).requires_grad_() for s in range(3)]
    routings = [mx.route(z, 4) for z in layers]
    total = routings[0].balance
    for r in routings[1:]:
        total += r.balance
    got = torch.autograd.grad(total, layers)
    one = torch.ones((), device="cuda")
    for z, g in zip(layers, got):
        assert torch.equal(g, mx.route_backward(None, one, z.detach(), mx.route(z.detach(), 4)))
