"""norm_rotate, route and linear_cross_entropy where autograd records: what they
keep for the backward pass, and what a caller may do with their outputs before
it.  The built module is replaced by the formulas in float64 on the CPU (and is
itself asked what it refuses before it looks for a device)."""
import pytest
import torch
from torch.autograd import forward_ad

from mxcheck import ensure_built

import mxfp8_block_scaled_mx_gb300 as mx


def routing(z, top_k, renormalize, mask):
    """ids, weights, counts, offsets, order, balance, lse."""
    experts = z.shape[1]
    p = torch.softmax(z, 1)
    ids = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :top_k]
    w = p.gather(1, ids)
    if renormalize:
        w = w / w.sum(1, keepdim=True)
    valid = torch.ones(len(z), dtype=torch.bool) if mask is None else mask.bool()
    n = int(valid.sum())
    counts = torch.bincount(ids[valid].flatten(), minlength=experts)
    load = torch.bincount(ids.flatten(), minlength=experts)
    offsets = torch.cat([load.new_zeros(1), load.cumsum(0)])
    order = torch.sort(ids.flatten(), stable=True).indices
    balance = experts * (counts / (n * top_k) * p[valid].mean(0)).sum()
    return (ids.int(), w, counts.int(), offsets.int(), order.int(), balance, torch.logsumexp(z, 1))


class Module:
    """What the built module does, None where a call is to be recorded among it."""

    def route(self, z, top_k, renormalize, mask, *_):
        if torch.is_grad_enabled() and z.requires_grad:
            return None
        return tuple(t.detach() for t in routing(z, top_k, renormalize, mask))

    def route_backward(self, d_weights, d_balance, d_lse, z, ids, weights, counts, lse, renormalize, mask, _):
        # what the gradient is computed from has the forward pass's values
        assert all(torch.is_tensor(t) for t in (ids, weights, counts, lse))
        with torch.enable_grad():
            v = z.detach().clone().requires_grad_()
            r = routing(v, ids.shape[1], renormalize, mask)
            assert torch.equal(r[0], ids) and torch.equal(r[1], weights) and torch.equal(r[2], counts)
            total = 0
            for d, t in ((d_weights, r[1]), (d_balance, r[5]), (d_lse, r[6])):
                total = total if d is None else total + (d * t).sum()
            return torch.autograd.grad(total, v)[0]


@pytest.fixture
def module(monkeypatch):
    m = Module()
    monkeypatch.setattr(mx, "_native", lambda: m)
    return m


def logits(seed):
    return torch.randn(7, 5, generator=torch.Generator().manual_seed(seed), dtype=torch.float64).requires_grad_()


def test_balance_losses_added_in_place(module):
    """The balance loss of several layers, summed into the first one's."""
    layers = [logits(s) for s in range(3)]
    total = None
    for z in layers:
        r = mx.route(z, 2)
        if total is None:
            total = r.balance
        else:
            total += r.balance
    got = torch.autograd.grad(total, layers)
    want = torch.autograd.grad(sum(routing(z, 2, True, None)[5] for z in layers), layers)
    assert all(torch.allclose(a, b, rtol=1e-12, atol=0) for a, b in zip(got, want))


def test_outputs_that_the_gradient_does_not_need_are_the_callers(module):
    """Offsets and order may be overwritten before the backward pass; what it reads
    (ids, weights, counts, lse) may not, and says so."""
    z = logits(4)
    r = mx.route(z, 2)
    r.offsets.zero_()
    r.order.zero_()
    got, = torch.autograd.grad((r.weights ** 2).sum() + r.balance, z)
    want, = torch.autograd.grad((routing(z, 2, True, None)[1] ** 2).sum() + routing(z, 2, True, None)[5], z)
    assert torch.allclose(got, want, rtol=1e-12, atol=1e-15)
    for name in ("ids", "weights", "counts", "lse"):
        r = mx.route(z, 2)
        with torch.no_grad():
            getattr(r, name).zero_()
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            torch.autograd.grad(r.balance, z)


def test_dual_tensors_are_refused():
    """A tangent of forward-mode differentiation is not dropped silently, whether
    backward-mode differentiation is on or off: by no operator of the module, for no argument."""
    ensure_built()
    x, w, z = torch.zeros(4, 2, 64), torch.ones(64), torch.zeros(4, 8)
    pos, f = torch.arange(4), torch.ones(8, dtype=torch.float64)
    h, v, lse = torch.zeros(4, 64), torch.zeros(9, 64), torch.zeros(4)
    r = mx.Routing(torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2), torch.zeros(8, dtype=torch.int32),
                   None, None, None, lse)
    e = mx.MxTensor(torch.zeros(9, 64, 64, dtype=torch.uint8), torch.zeros(4, dtype=torch.uint8), "e4m3")
    calls = {
        "norm_rotate": (mx.norm_rotate, dict(q=x, k=x, w_q=w, w_k=w, positions=pos, frequencies=f),
                        ("q", "k", "w_q", "w_k", "frequencies")),
        "norm_rotate_backward": (mx.norm_rotate_backward,
                                 dict(d_q=x, d_k=x, q=x, k=x, w_q=w, w_k=w, positions=pos, frequencies=f),
                                 ("d_q", "k")),
        "route": (mx.route, dict(logits=z, top_k=2), ("logits",)),
        "route_backward": (mx.route_backward, dict(d_weights=r.weights, d_balance=None, logits=z, routing=r),
                           ("d_weights", "logits")),
        "linear_cross_entropy": (mx.linear_cross_entropy, dict(x=h, weight=v, labels=pos), ("x", "weight")),
        "linear_cross_entropy_backward": (mx.linear_cross_entropy_backward,
                                          dict(d_loss=lse, d_lse=None, x=h, weight=v, labels=pos, lse=lse),
                                          ("d_loss", "weight")),
        "norm_residual": (mx.norm_residual, dict(block=h, residual=h, w_pre=w), ("block", "w_pre")),
        "moe_few_tokens": (mx.moe_few_tokens, dict(x=h, router=v, gate=e, up=e, down=e, top_k=2), ("x", "router")),
    }
    for name, (call, args, duals) in calls.items():
        for grad in (False, True):
            for dual in duals:
                with torch.set_grad_enabled(grad), forward_ad.dual_level():
                    t = args[dual].detach().requires_grad_(grad)
                    with pytest.raises(ValueError, match="forward-mode"):
                        call(**{**args, dual: forward_ad.make_dual(t, torch.ones_like(t))})
        with pytest.raises(ValueError) as plain:
            call(**args)
        assert "forward-mode" not in str(plain.value), name


def test_frequencies_that_ask_for_a_gradient_are_refused():
    """norm_rotate has none for them, and does not give them none silently; where
    autograd is off they are numbers like any others."""
    ensure_built()
    x, w, pos = torch.zeros(4, 2, 64), torch.ones(64), torch.arange(4)
    f = torch.ones(8, dtype=torch.float64, requires_grad=True)
    for q in (x, x.clone().requires_grad_()):
        with pytest.raises(ValueError, match="frequencies"):
            mx.norm_rotate(q, x, w, w, pos, f)
    with torch.no_grad(), pytest.raises(ValueError) as plain:
        mx.norm_rotate(x, x, w, w, pos, f)   # (host tensors)
    assert "frequencies" not in str(plain.value)
