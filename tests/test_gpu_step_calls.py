"""What a program does around the training step's operators: sums of balance losses in
place, outputs of which it keeps some."""
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


def test_a_kept_output_keeps_no_large_one(mx):
    """Small outputs share an allocation, at most 1 MB of them; of many tokens those
    that have their size stand alone."""
    kept = 2 ** 20 + 200
    for tokens, experts, k in ((50, 64, 8), (10000, 64, 8), (12000, 64, 8), (65536, 8, 2), (30000, 512, 32)):
        r = mx.route(randn(tokens, experts, seed=1), k)
        for name in ("counts", "offsets", "balance"):
            assert getattr(r, name).untyped_storage().nbytes() <= kept, (tokens, name)
        for name in ("ids", "weights", "order", "lse"):
            t = getattr(r, name)
            assert t.untyped_storage().nbytes() <= max(kept, t.numel() * 4), (tokens, name)
    w = randn(16, 8, seed=2, dtype=BF16)
    for tokens in (1, 131072, 200000):
        labels = torch.zeros(tokens, dtype=torch.int32, device="cuda")
        for t in mx.linear_cross_entropy(torch.zeros(tokens, 8, dtype=BF16, device="cuda"), w, labels):
            assert t.untyped_storage().nbytes() <= max(kept, tokens * 4)
    # the winners are those of a call whose outputs share one
    z = randn(20000, 32, seed=3)
    assert torch.equal(mx.route(z, 4).ids[:2000], mx.route(z[:2000], 4).ids) and mx.device_status() == 0
