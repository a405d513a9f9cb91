"""What a program does around the training step's operators: sums of balance losses in
place, outputs of which it keeps some, modes of torch's that watch or fill new tensors, one
workspace for batches of any size."""
import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

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


class Seen(TorchDispatchMode):
    """The sizes and types that are asked of torch's allocating operator."""

    def __init__(self):
        super().__init__()
        self.made = []

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        out = func(*args, **(kwargs or {}))
        if func is torch.ops.aten.empty.memory_format:
            self.made.append((tuple(out.shape), out.dtype))
        return out


def calls_of_every_kind(mx):
    heads, w = randn(30, 6, 64, seed=1, dtype=BF16), randn(64, seed=2, dtype=BF16)
    args = (heads[:, :4], heads[:, 4:], w, w, torch.arange(30, device="cuda"), mx.rotary_frequencies(64))
    z = {n: randn(n, 16, seed=3) for n in (20, 20000)}
    r = mx.route(z[20], 2)
    x, v, labels = randn(30, 64, seed=4, dtype=BF16), randn(100, 64, seed=5, dtype=BF16), torch.arange(30, device="cuda")
    lse = mx.linear_cross_entropy(x, v, labels)[1]
    return [lambda: mx.norm_rotate(*args), lambda: vars(mx.norm_rotate_backward(*args[:2], *args)).values(),
            lambda: vars(mx.route(z[20], 2)).values(), lambda: vars(mx.route(z[20000], 2)).values(),
            lambda: [mx.route_backward(r.weights, None, z[20], r)], lambda: mx.linear_cross_entropy(x, v, labels),
            lambda: mx.linear_cross_entropy_backward(lse, None, x, v, labels, lse),
            lambda: mx.norm_residual(x, x, x[0].contiguous()),
            lambda: [t for t in vars(mx.norm_residual_backward(x, x, x, x, x[0].contiguous())).values() if t is not None]]


def test_new_tensors_are_seen_by_dispatch_modes(mx):
    for call in calls_of_every_kind(mx):
        want = list(call())
        with Seen() as seen:
            got = list(call())
        for a, b in zip(want, got):
            assert torch.equal(a, b) and (tuple(b.shape), b.dtype) in seen.made


def test_new_tensors_are_filled_where_algorithms_are_deterministic(mx):
    calls = calls_of_every_kind(mx)
    want = [list(c()) for c in calls]
    before = torch.are_deterministic_algorithms_enabled()
    torch.use_deterministic_algorithms(True)
    try:
        for call, ref in zip(calls, want):
            with torch.autograd.profiler.profile() as p:
                got = list(call())
            assert all(torch.equal(a, b) for a, b in zip(ref, got))
            names = [e.name for e in p.function_events]
            assert names.count("aten::fill_") >= len(got), names
    finally:
        torch.use_deterministic_algorithms(before)
    assert mx.device_status() == 0


def test_one_workspace_for_batches_of_any_size(mx):
    """A workspace for the largest, full of NaN, gives what a call's own gives."""
    dirty = lambda n: torch.full((n,), 255, dtype=torch.uint8, device="cuda")  # noqa: E731
    z = randn(10000, 64, seed=1)
    ws = dirty(mx.mx_route_workspace(10000, 64))
    for tokens in (10000, 9729, 9728, 8192, 8191, 300, 64):
        a, b = mx.route(z[:tokens], 8), mx.route(z[:tokens], 8, workspace=ws)
        assert all(torch.equal(u, v) for u, v in zip(vars(a).values(), vars(b).values())), tokens
    x, w, labels = randn(400, 72, seed=2, dtype=BF16), randn(1000, 72, seed=3, dtype=BF16), torch.arange(400, device="cuda")
    ws = dirty(mx.mx_linear_cross_entropy_workspace(400, 72, 1000))
    back = dirty(mx.mx_linear_cross_entropy_backward_workspace(400, 72, 1000))
    for tokens in (400, 65, 64, 33, 1):
        xs, ls, d = x[:tokens], labels[:tokens], torch.ones(tokens, device="cuda")
        a, b = mx.linear_cross_entropy(xs, w, ls), mx.linear_cross_entropy(xs, w, ls, workspace=ws)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]), tokens
        a, b = (mx.linear_cross_entropy_backward(d, None, xs, w, ls, b[1], workspace=s) for s in (None, back))
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]), tokens
    assert mx.device_status() == 0


def test_heads_in_place_where_autograd_records(mx):
    """The backward pass needs q and k: it says that they were overwritten."""
    heads = randn(20, 4, 32, seed=1, dtype=BF16)
    w = torch.ones(32, device="cuda").requires_grad_()
    q, k = heads[:, :3].clone(), heads[:, 3:].clone()
    args = (w, w, torch.arange(20, device="cuda"), mx.rotary_frequencies(32))
    want = mx.norm_rotate(q, k, *args)
    a, _ = mx.norm_rotate(q, k, *args, out_q=q)
    assert a is q and torch.equal(q, want[0])
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        a.float().sum().backward()
