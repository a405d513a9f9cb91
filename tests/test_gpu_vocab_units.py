"""The units that the vocabulary gradient holds its logits' gradient in, for more than
64 tokens: the label's entry of a mean is exact but for the label's probability.

Tolerances, against products in 64 bits.  In units of d_loss, the same for all tokens that
count, an entry of dz is p, rounded by half a step of bf16, 2^-8 p, or at the label p - 1,
which is rounded to -1 or to its other neighbour: by no more than p, nor more than 2^-9.
The softmax's own error and the products' sums are those of test_gpu_vocab_loss; division
by the unit and multiplication with it add two half steps of FP32."""
import pytest
import torch

import test_gpu_vocab_loss as loss
from mxcheck import ensure_built

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def mx():
    ensure_built()
    import mxfp8_block_scaled_mx_gb300 as mx
    return mx


# (1 / 255 = 2^-8 x 1.0039 lies in the middle between two values of bf16)
SHAPES = [(255, 64, 5000), (255, 1032, 700), (510, 200, 3001), (510, 2056, 300), (1020, 72, 20001)]


@pytest.mark.parametrize("weight_dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("ignored", [0.0, 0.3])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_gradient_of_a_mean(mx, shape, ignored, weight_dtype):
    tokens, hidden, vocab = shape
    x, w, labels = loss.inputs(*shape, ignored=ignored, seed=tokens)
    w = (w.float() * 0.25).to(BF16)
    share = 1.0 / tokens
    _, lse = mx.linear_cross_entropy(x, w, labels)
    dx, dw = mx.linear_cross_entropy_backward(torch.full((tokens,), share, device="cuda"), None, x, w, labels, lse,
                                              weight_dtype=weight_dtype)
    share = torch.tensor(share, dtype=FP32).double().item()
    xd, wd = x.double(), w.double()
    z = xd @ wd.T
    mag = (xd.abs() @ wd.abs().T).max().item()
    soft = 2 * (loss.z_error(hidden, mag) + 2.0 ** -20 + 2.0 ** -22 * torch.logsumexp(z, 1).abs().max().item())
    p = torch.softmax(z, 1)
    valid = labels != -100
    p[~valid] = 0
    off = p * (2.0 ** -8 + soft)
    rows = valid.nonzero()[:, 0]
    at = labels[rows]
    off[rows, at] = p[rows, at].clamp(max=2.0 ** -9) + p[rows, at] * soft
    dz = p.clone()
    dz[rows, at] -= 1
    for got, ref, tol, m, length in ((dx, dz @ wd, off @ wd.abs(), dz.abs() @ wd.abs(), vocab),
                                     (dw, dz.T @ xd, off.T @ xd.abs(), dz.abs().T @ xd.abs(), tokens)):
        bound = share * (1.01 * tol + (length / 16 + 3) * 2.0 ** -22 * m)
        half = torch.finfo(got.dtype).eps / 2
        err = (got.double() - share * ref).abs()
        assert (err <= bound + half * (share * ref.abs() + bound)).all(), (err / bound).max().item()
    assert mx.device_status() == 0


@pytest.mark.parametrize("hidden", [64, 1032])
def test_units_of_any_size(mx, hidden):
    """Powers of two change nothing but the gradients' exponents; what stands in d_loss where
    no label counts is not looked at; a token with an infinite one touches no other row."""
    x, w, labels = loss.inputs(200, hidden, 700)
    _, lse = mx.linear_cross_entropy(x, w, labels)
    g = torch.Generator("cuda").manual_seed(1)
    d = torch.rand(200, generator=g, device="cuda") + 0.5
    odd = (labels != -100) & (torch.arange(200, device="cuda") % 2 == 1)
    d[odd.nonzero()[0]] = 2.0   # the largest, and so the unit
    back = lambda d, e=None: mx.linear_cross_entropy_backward(d, e, x, w, labels, lse, weight_dtype="fp32")  # noqa: E731
    dx, dw = back(d)
    for k in (-60, -8, 1, 50):
        a, b = back(d * 2.0 ** k)
        assert torch.equal(a, dx * 2.0 ** k) and torch.equal(b, dw * 2.0 ** k), k
    for junk in (float("nan"), float("inf"), -float("inf"), 1e30):
        a, b = back(torch.where(labels == -100, junk, d))
        assert torch.equal(a, dx) and torch.equal(b, dw), junk
    assert all((t == 0).all() for t in back(torch.zeros_like(d)))
    first = int((labels != -100).nonzero()[0])
    a, _ = back(torch.where(torch.arange(200, device="cuda") == first, float("inf"), d))
    keep = torch.arange(200, device="cuda") != first
    # (in units of 1 the entries of dz round otherwise, by half a step each way; then dx does)
    p = torch.softmax(x.double() @ w.double().T, 1)
    rows = (labels != -100).nonzero()[:, 0]
    p[labels == -100] = 0
    p[rows, labels[rows]] -= 1
    m = (p.abs() * d.double()[:, None]) @ w.double().abs()
    off = 2 * 1.05 * 2.0 ** -8 * (m + dx.double().abs())
    assert ((a.double() - dx.double()).abs() <= off)[keep].all() and not torch.isfinite(a[first]).all()
    # only the normalizer's gradient: as for a loss of nothing
    e = torch.randn(200, generator=g, device="cuda")
    assert all(torch.equal(u, v) for u, v in zip(back(None, e), back(torch.zeros_like(d), e)))
    # small and large ones side by side: a token's row of dx has its own scale
    wide = d * torch.where(torch.arange(200, device="cuda") % 2 == 0, 2.0 ** -40, 1.0)
    a, _ = back(wide)
    even = torch.arange(0, 200, 2, device="cuda")
    assert torch.equal(a[even], dx[even] * 2.0 ** -40) and torch.equal(a[1::2], dx[1::2])
    assert mx.device_status() == 0
