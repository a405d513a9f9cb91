"""norm_residual and moe_few_tokens where autograd records: the gradients that
arrive at each input, given outputs and their histories.  The built module
is replaced by the formulas in float64 on the CPU."""
import pytest
import torch

import mxfp8_block_scaled_mx_gb300 as mx


def rms(v, w, eps):
    return v * torch.rsqrt(v.square().mean(1, keepdim=True) + eps) * w


def formula(block, residual, w_pre, w_post, gate, alpha, eps):
    n = block if w_post is None else rms(block, w_post, eps)
    if gate is not None:
        g = gate.reshape(-1, block.shape[1])
        n = n * g.repeat_interleave(len(block) // len(g), 0)
    stored = alpha * residual + n
    return stored, rms(stored, w_pre, eps)


class Module:
    """What the built module does, None where a call is to be recorded among it."""

    def __init__(self):
        self.backward_calls = 0

    def norm_residual(self, block, residual, w_pre, w_post, gate, alpha, eps, out_residual, out, _):
        given = [t for t in (block, residual, w_pre, w_post, gate, out_residual, out) if t is not None]
        if torch.is_grad_enabled() and any(t.requires_grad for t in given):
            return None
        r = formula(block, residual, w_pre, w_post, gate, alpha, eps)
        return tuple(v if o is None else o.copy_(v) for v, o in zip(r, (out_residual, out)))

    def norm_residual_backward(self, d_res, d_y, block, stored, w_pre, w_post, gate, alpha, eps, *_):
        self.backward_calls += 1
        assert d_y.is_contiguous() and (d_res is None or d_res.is_contiguous())
        with torch.enable_grad():
            # the residual that gives this stream
            n = formula(block, torch.zeros_like(block), w_pre, w_post, gate, alpha, eps)[0]
            ins = [t if t is None else t.detach().clone().requires_grad_()
                   for t in (block, (stored - n) / alpha, w_pre, w_post, gate)]
            s, y = formula(*ins, alpha, eps)
            loss = (y * d_y).sum() + (0 if d_res is None else (s * d_res).sum())
            grads = iter(torch.autograd.grad(loss, [t for t in ins if t is not None]))
        return [None if t is None else next(grads) for t in ins]

    def moe_few_tokens(self, x, router, *args):
        if torch.is_grad_enabled() and (x.requires_grad or router.requires_grad):
            return None
        z = x @ router.T
        y = x * 2
        if args[-3] is not None:
            y = args[-3].copy_(y)
        return y, z.argmax(1, keepdim=True).int(), z.amax(1, keepdim=True)


@pytest.fixture
def module(monkeypatch):
    m = Module()
    monkeypatch.setattr(mx, "_native", lambda: m)
    return m


def inputs(post=True, gates=1, rows=4, cols=6):
    g = torch.Generator().manual_seed(1)
    n = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    return dict(block=n(rows, cols), residual=n(rows, cols), w_pre=n(cols) + 2,
                w_post=n(cols) + 2 if post else None,
                gate=None if not gates else n(cols) if gates == 1 else n(gates, cols))


def leaves(d):
    return {k: None if t is None else t.clone().requires_grad_() for k, t in d.items()}


def compare(mine, ref):
    for k, t in ref.items():
        if t is not None:
            assert torch.allclose(mine[k].grad, t.grad, rtol=1e-9, atol=1e-12), k


@pytest.mark.parametrize("post,gates", [(True, 1), (False, 0), (True, 2), (False, 4)])
@pytest.mark.parametrize("use", ["both", "stream", "normed", "sums"])
def test_gradients_reach_their_inputs(module, post, gates, use):
    d = inputs(post, gates)
    mine, ref = leaves(d), leaves(d)

    def loss(s, y):
        a = torch.linspace(-1, 1, s.numel(), dtype=s.dtype).view(s.shape)
        return {"both": (s * a).sum() + (y * a.flip(0)).sum(), "stream": (s * a).sum(),
                "normed": (y * a).sum(), "sums": s.sum() + y.sum()}[use]

    loss(*mx.norm_residual(**mine, alpha=0.5, eps=1e-3)).backward()
    s, y = formula(*ref.values(), 0.5, 1e-3)
    loss(s, y).backward()
    assert module.backward_calls == 1
    if use == "stream":
        ref["w_pre"].grad = torch.zeros_like(ref["w_pre"])
    compare(mine, ref)


def test_only_wanted_gradients(module):
    d = inputs()
    w = d["w_pre"].clone().requires_grad_()
    s, y = mx.norm_residual(**{**d, "w_pre": w})
    assert s.requires_grad and y.requires_grad
    y.sum().backward()
    assert w.grad is not None
    with torch.no_grad():
        s, y = mx.norm_residual(**{**d, "w_pre": w})
    assert not s.requires_grad and not y.requires_grad
    s, y = mx.norm_residual(**d)
    assert not s.requires_grad and not y.requires_grad


def test_given_outputs(module):
    """A stream that is added to in place, and outputs that are views: the
    same gradients as without."""
    d = inputs()
    ref, mine = leaves(d), leaves(d)

    def two(p, buffers):
        stream = p["residual"] * 1.0
        x = p["block"] * 1.0
        for i in range(2):
            kw = dict(out_residual=stream, out=buffers[i][:, :6]) if buffers else {}
            s, y = mx.norm_residual(x, stream, p["w_pre"], p["w_post"], p["gate"], **kw)
            if buffers:
                assert s is stream and y.data_ptr() == buffers[i].data_ptr()
            stream, x = s, y
        return (stream * x).sum()

    two(ref, None).backward()
    two(mine, [torch.zeros(4, 8, dtype=torch.float64) for _ in range(2)]).backward()
    compare(mine, ref)
    for bad in (dict(out=torch.zeros(4, 5)), dict(out_residual=torch.zeros(4, 6)), dict(out=3)):
        with pytest.raises(ValueError):
            mx.norm_residual(**leaves(d), **bad)


def test_a_stream_changed_behind_the_back_is_reported(module):
    d = leaves(inputs())
    s, y = mx.norm_residual(**d)
    with torch.no_grad():
        s.add_(1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


def test_the_layer_has_no_gradient(module):
    codes = mx.MxTensor(torch.zeros(2, 4, 4, dtype=torch.uint8), torch.zeros(8), "e4m3")
    x, router = torch.ones(3, 4), torch.ones(2, 4, requires_grad=True)
    for kw in (dict(), dict(out=torch.zeros(3, 6)[:, :4])):
        y = mx.moe_few_tokens(x, router, codes, codes, codes, 1, **kw)
        assert torch.equal(y, 2 * x) and y.requires_grad
        with pytest.raises(RuntimeError, match="moe_few_tokens has no gradient"):
            y.sum().backward()
    y, ids, w = mx.moe_few_tokens(x, router, codes, codes, codes, 1, return_routing=True)
    assert not ids.requires_grad and ids.shape == w.shape == (3, 1)
    with torch.no_grad():
        assert not mx.moe_few_tokens(x, router, codes, codes, codes, 1).requires_grad
    assert not mx.moe_few_tokens(x, router.detach(), codes, codes, codes, 1).requires_grad
