"""The cross entropy over a vocabulary, and its gradients, on the GPU against the
oracle.

Tolerances: the tensor core adds 16 exact products of bf16 values to an FP32
accumulator at a time, and may cut each sum off at 24 bits: a logit is off by at
most (hidden / 16 + 2) 2^-22 of the magnitudes behind it, Z below.  The sum of
exponentials adds 2^-20 (its terms' 2^-22 each, chains of 32 and of the parts), so
lse is off by Z + 2^-20 + 2^-22 |lse|, the loss by twice Z.  dz has that relative
error of its softmax part and is rounded to bf16, half a step, 2^-8 (for up to 64
tokens to two bf16 terms, 2^-16); the products add (length / 16 + 2) 2^-22 of their
magnitudes, the output its half step."""
import numpy as np
import pytest
import torch

from mxcheck import ensure_built, to_f64
from oracle import step_oracle as S

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32
HALF = {BF16: 2.0 ** -8, FP32: 2.0 ** -24}


@pytest.fixture(scope="module")
def mx():
    ensure_built()
    import mxfp8_block_scaled_mx_gb300 as mx
    return mx


def inputs(tokens, hidden, vocab, ignored=0.2, seed=0, dtype=torch.int64):
    g = torch.Generator("cuda").manual_seed(seed)
    w = (torch.randn((vocab, hidden), generator=g, device="cuda") * 2 / hidden ** 0.5).to(BF16)
    labels = torch.randint(0, vocab, (tokens,), generator=g, device="cuda")
    x = (torch.randn((tokens, hidden), generator=g, device="cuda") + w[labels].float()).to(BF16)
    drop = torch.rand((tokens,), generator=g, device="cuda") < ignored
    return x, w, torch.where(drop, -100, labels).to(dtype)


def z_error(hidden, magnitude):
    return (hidden / 16 + 2) * 2.0 ** -22 * magnitude


def check(mx, x, w, labels, ignore=-100, **kw):
    loss, lse = mx.linear_cross_entropy(x, w, labels, ignore, **kw)
    ref_loss, ref_lse, z, mag = S.cross_entropy(to_f64(x), to_f64(w), labels.cpu().numpy(), ignore)
    err = z_error(x.shape[1], mag) + 2.0 ** -20 + 2.0 ** -22 * np.abs(ref_lse)
    assert loss.dtype == lse.dtype == FP32 and loss.shape == lse.shape == labels.shape
    assert (np.abs(to_f64(lse) - ref_lse) <= err).all(), np.max(np.abs(to_f64(lse) - ref_lse) / err)
    off = np.abs(to_f64(loss) - ref_loss)
    assert (off <= 2 * err + 2.0 ** -24 * np.abs(ref_loss)).all(), np.max(off / err)
    assert (loss[labels == ignore] == 0).all()
    return lse, ref_lse, z, mag


def check_backward(mx, x, w, labels, ignore=-100, weight_dtype="bf16", use=(True, True), **kw):
    lse, ref_lse, z, mag = check(mx, x, w, labels, ignore)
    g = torch.Generator("cuda").manual_seed(9)
    d_loss = torch.rand(len(x), generator=g, device="cuda") / len(x) if use[0] else None
    d_lse = torch.randn(len(x), generator=g, device="cuda") / len(x) * 0.1 if use[1] else None
    dx, dw = mx.linear_cross_entropy_backward(d_loss, d_lse, x, w, labels, lse, ignore, weight_dtype, **kw)
    zero = np.zeros(len(x))
    d = S.cross_entropy_backward(to_f64(x), to_f64(w), labels.cpu().numpy(), ignore,
                                 zero if d_loss is None else to_f64(d_loss), zero if d_lse is None else to_f64(d_lse),
                                 z, ref_lse)
    soft = 2 * (z_error(x.shape[1], mag) + 2.0 ** -20 + 2.0 ** -22 * np.abs(ref_lse))  # of exp(z - lse)
    for name, got, length, row_soft in (("dx", dx, w.shape[0], soft[:, None]), ("dw", dw, len(x), soft.max())):
        half = HALF[got.dtype]
        ref, m = d[name], d[name + "_mag"]
        tol = ((2.0 ** (-16 if len(x) <= 64 else -8) + (length / 16 + 2) * 2.0 ** -22) * m
               + row_soft * d["p_" + name[1]]) * 1.01
        err = np.abs(to_f64(got) - ref)
        assert (err <= tol + half * (np.abs(ref) + tol) + 1e-37).all(), (name, np.max(err / (tol + 1e-37)))
    assert dw.dtype == (FP32 if weight_dtype == "fp32" else BF16)
    return dx, dw


# tiles that end inside: rows and columns around 128 and 256, a vocabulary of
# one; contractions of one element run up to several stages' rounds
SHAPES = [(1, 64, 1000), (2, 8, 1), (5, 16, 2), (127, 72, 255), (128, 64, 256), (129, 200, 257), (256, 64, 31),
          (257, 136, 513), (600, 520, 1100), (33, 1000, 2000), (1, 2048, 300), (300, 24, 5000),
          # few tokens: boxes of 16, 32 and 64, the first count that is not few; more tiles than
          # blocks, a hidden length of several tiles
          (16, 72, 700), (17, 64, 129), (32, 136, 1500), (64, 320, 33000), (65, 64, 300), (3, 64, 20001)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_losses(mx, shape):
    check(mx, *inputs(*shape, seed=sum(shape)))


@pytest.mark.parametrize("weight_dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_gradients(mx, shape, weight_dtype):
    check_backward(mx, *inputs(*shape, seed=sum(shape)), weight_dtype=weight_dtype)


@pytest.mark.parametrize("use", [(True, False), (False, True), (False, False)])
def test_gradients_one_by_one(mx, use):
    check_backward(mx, *inputs(100, 64, 700), use=use)


@pytest.mark.parametrize("tokens", [20, 300])
def test_only_one_gradient(mx, tokens):
    x, w, labels = inputs(tokens, 64, 700)
    _, lse = mx.linear_cross_entropy(x, w, labels)
    ones = torch.ones(tokens, device="cuda")
    dx, dw = mx.linear_cross_entropy_backward(ones, None, x, w, labels, lse)
    a, none = mx.linear_cross_entropy_backward(ones, None, x, w, labels, lse, need_weight=False)
    assert none is None and torch.equal(a, dx)
    none, b = mx.linear_cross_entropy_backward(ones, None, x, w, labels, lse, need_x=False)
    assert none is None and torch.equal(b, dw)
    assert mx.linear_cross_entropy_backward(ones, None, x, w, labels, lse, need_x=False,
                                            need_weight=False) == (None, None)
    none, b = mx.linear_cross_entropy_backward(None, None, x[:0], w, labels[:0], lse[:0], need_x=False)
    assert none is None and (b == 0).all()


def test_labels(mx):
    x, w, labels = inputs(70, 64, 300, dtype=torch.int32)
    check_backward(mx, x, w, labels)
    check_backward(mx, x, w, torch.full_like(labels, -100))     # none counts
    check_backward(mx, x, w, torch.where(labels == -100, 7, labels), ignore=7)   # an index of the vocabulary
    for t in (torch.int32, torch.int64):
        bad = labels.to(t)
        bad[3], bad[5], bad[6] = 300, -1, -100
        loss, lse = mx.linear_cross_entropy(x, w, bad)
        assert mx.device_status() == 6 and mx.device_status() == 0
        assert loss[[3, 5]].isnan().all() and loss[6].item() == 0 and torch.isfinite(lse).all()
        # no gradient through them
        ones = torch.ones(70, device="cuda")
        dx, dw = mx.linear_cross_entropy_backward(ones, None, x, w, bad, lse)
        good = bad.clone()
        good[[3, 5]] = -100
        a, b = mx.linear_cross_entropy_backward(ones, None, x, w, good, lse)
        assert torch.equal(dx, a) and torch.equal(dw, b) and (dx[[3, 5]] == 0).all()


def test_large_and_equal_logits(mx):
    x, w, labels = inputs(40, 64, 500, ignored=0.0)
    check(mx, x * 64, w, labels)                     # one logit holds all
    check_backward(mx, torch.zeros_like(x), w, labels)   # all alike
    lse, *_ = check(mx, x, torch.zeros_like(w), labels)
    assert np.allclose(to_f64(lse), np.log(500), rtol=2.0 ** -22)
    # a token with NaN or infinity touches no other
    y = x.clone()
    y[3, 5], y[7, 9] = float("nan"), float("inf")
    loss, lse = mx.linear_cross_entropy(y, w, labels)
    clean, _ = mx.linear_cross_entropy(x, w, labels)
    keep = torch.ones(40, dtype=torch.bool, device="cuda")
    keep[[3, 7]] = False
    assert not torch.isfinite(loss[[3, 7]]).any() and torch.equal(loss[keep], clean[keep])
    dx, _ = mx.linear_cross_entropy_backward(torch.ones(40, device="cuda"), None, y, w, labels, lse)
    assert torch.isfinite(dx[keep]).all()


def test_strided_operands(mx):
    x, w, labels = inputs(150, 64, 400)
    wide_x = torch.full((150, 96), float("nan"), dtype=BF16, device="cuda")
    wide_w = torch.full((400, 80), float("nan"), dtype=BF16, device="cuda")
    wide_x[:, 8:72], wide_w[:, 16:] = x, w
    a = mx.linear_cross_entropy(x, w, labels)
    b = mx.linear_cross_entropy(wide_x[:, 8:72], wide_w[:, 16:], labels)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    ones = torch.ones(150, device="cuda")
    a = mx.linear_cross_entropy_backward(ones, None, x, w, labels, a[1])
    b = mx.linear_cross_entropy_backward(ones, None, wide_x[:, 8:72], wide_w[:, 16:], labels, b[1])
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("tokens,hidden,vocab,chunk", [(8192, 64, 70001, 1024), (64, 8, 4200001, 8)])
def test_pieces_of_the_vocabulary(mx, tokens, hidden, vocab, chunk):
    """More than one piece, a last one that is not whole: gradients against products
    of the softmax in 64 bits, whose terms are bounded as above."""
    x, w, labels = inputs(tokens, hidden, vocab)
    assert mx.mx_linear_cross_entropy_backward_workspace(tokens, hidden, vocab) < 2 * tokens * vocab
    loss, lse = mx.linear_cross_entropy(x, w, labels)
    d_loss = torch.full((tokens,), 1.0 / tokens, device="cuda")
    dx, dw = mx.linear_cross_entropy_backward(d_loss, None, x, w, labels, lse)
    dx2, dw2 = mx.linear_cross_entropy_backward(d_loss, None, x, w, labels, lse)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)
    rx = torch.zeros(tokens, hidden, dtype=torch.float64, device="cuda")
    rw = torch.zeros(vocab, hidden, dtype=torch.float64, device="cuda")
    mag_x, mag_w = torch.zeros_like(rx), torch.zeros_like(rw)
    for t in range(0, tokens, chunk):
        xs, ls = x[t:t + chunk].double(), labels[t:t + chunk]
        p = torch.softmax(xs @ w.double().T, 1)
        valid = ls != -100
        p[~valid] = 0
        p[valid, ls[valid]] -= 1
        p /= tokens
        rx[t:t + chunk], mag_x[t:t + chunk] = p @ w.double(), p.abs() @ w.double().abs()
        rw += p.T @ xs
        mag_w += p.abs().T @ xs.abs()
    for got, ref, mag in ((dx, rx, mag_x), (dw, rw, mag_w)):
        assert ((got.double() - ref).abs() <= 1.05 * 2.0 ** -8 * mag + 2.0 ** -8 * ref.abs() + 1e-37).all()


def test_without_tokens(mx):
    x, w, labels = inputs(0, 64, 100)
    loss, lse = mx.linear_cross_entropy(x, w, labels)
    assert loss.shape == lse.shape == (0,)
    dx, dw = mx.linear_cross_entropy_backward(loss, None, x, w, labels, lse)
    assert dx.shape == (0, 64) and (dw == 0).all()


def test_same_bits_again_and_a_workspace(mx):
    x, w, labels = inputs(700, 256, 3000)
    a = mx.linear_cross_entropy(x, w, labels)
    ws = torch.full((mx.mx_linear_cross_entropy_workspace(700, 256, 3000),), 255, dtype=torch.uint8, device="cuda")
    b = mx.linear_cross_entropy(x, w, labels, workspace=ws)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    with pytest.raises(ValueError):
        mx.linear_cross_entropy(x, w, labels, workspace=ws[:-1])
    ones = torch.ones(700, device="cuda")
    ws = torch.full((mx.mx_linear_cross_entropy_backward_workspace(700, 256, 3000),), 255, dtype=torch.uint8, device="cuda")
    a = mx.linear_cross_entropy_backward(ones, None, x, w, labels, a[1])
    b = mx.linear_cross_entropy_backward(ones, None, x, w, labels, b[1], workspace=ws)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


# vocabularies whose last 256 columns end before the last part of dx begins, with few
# tokens and with many
ENDS = [(16, 8, 2817), (5, 264, 1537), (64, 1000, 5377), (65, 1000, 5633), (300, 520, 3329), (777, 520, 1793)]


@pytest.mark.parametrize("shape", SHAPES + ENDS, ids=str)
def test_nothing_is_read_from_a_workspace_that_was_not_written(mx, shape):
    """A workspace full of NaN."""
    x, w, labels = inputs(*shape, seed=3)
    dirty = lambda n: torch.full((n,), 255, dtype=torch.uint8, device="cuda")  # noqa: E731
    check(mx, x, w, labels, workspace=dirty(mx.mx_linear_cross_entropy_workspace(*shape)))
    check_backward(mx, x, w, labels, workspace=dirty(mx.mx_linear_cross_entropy_backward_workspace(*shape)))


def test_refusals(mx):
    x, w, labels = inputs(20, 64, 100)
    lse = torch.zeros(20, device="cuda")
    for bad in (dict(x=x.float()), dict(weight=w.float()), dict(labels=labels[:19]), dict(labels=labels.float()),
                dict(x=x[:, :60], weight=w[:, :60]), dict(weight=w[:, :56]), dict(x=x.t()), dict(x=x.cpu()), dict(x=x[0]),
                dict(weight=w[:0])):
        args = {**dict(x=x, weight=w, labels=labels), **bad}
        with pytest.raises(ValueError):
            mx.linear_cross_entropy(**args)
        with pytest.raises(ValueError):
            mx.linear_cross_entropy_backward(None, None, lse=lse, **args)
    with pytest.raises(ValueError):
        mx.linear_cross_entropy_backward(lse[:3], None, x, w, labels, lse)
    with pytest.raises(ValueError):
        mx.linear_cross_entropy_backward(None, None, x, w, labels, lse[:3])
    with pytest.raises(mx.MxError):     # rows off 16 bytes
        wide = torch.zeros(20, 65, dtype=BF16, device="cuda")
        mx.linear_cross_entropy(wide[:, 1:], w, labels)


def test_autograd(mx):
    x, w, labels = inputs(90, 64, 500)
    a, b = x.clone().requires_grad_(), w.clone().requires_grad_()
    loss, lse = mx.linear_cross_entropy(a, b, labels)
    gx, gw = torch.autograd.grad(loss.sum() / 64 + (lse * 0.25).sum(), (a, b))
    dx, dw = mx.linear_cross_entropy_backward(torch.full((90,), 1 / 64, device="cuda"), torch.full((90,), 0.25, device="cuda"),
                                              x, w, labels, lse.detach())
    assert torch.equal(gx, dx) and torch.equal(gw, dw)
    loss, _ = mx.linear_cross_entropy(x, b, labels)      # one input alone, an expanded gradient
    gw, = torch.autograd.grad(loss.sum(), b)
    assert torch.equal(gw, mx.linear_cross_entropy_backward(torch.ones(90, device="cuda"), None, x, w, labels, lse.detach())[1])
    loss, _ = mx.linear_cross_entropy(a, w, labels)
    gx, = torch.autograd.grad(loss.sum(), a)
    assert torch.equal(gx, mx.linear_cross_entropy_backward(torch.ones(90, device="cuda"), None, x, w, labels, lse.detach())[0])


def test_gradient_against_differences(mx):
    """Differences of the kernel's own losses along random directions: steps of bf16
    values (2^-4 of a row), so that x + h d is exact; second-order terms stay below a
    hundredth, dz's rounding below 2^-8."""
    x, w, labels = inputs(8, 64, 200, ignored=0.0)
    x = (x.float() * 4).round().div(4).to(BF16)          # multiples of 1/4
    ones = torch.ones(8, device="cuda")
    _, lse = mx.linear_cross_entropy(x, w, labels)
    dx, _ = mx.linear_cross_entropy_backward(ones, None, x, w, labels, lse)
    g = torch.Generator("cuda").manual_seed(4)
    for _ in range(4):
        d = torch.randint(-1, 2, x.shape, generator=g, device="cuda").to(BF16) / 32
        up, down = (mx.linear_cross_entropy(x + s * d, w, labels)[0].double().sum().item() for s in (1, -1))
        slope = (dx.double() * d.double()).sum().item()
        scale = (dx.double().abs() * d.double().abs()).sum().item()
        assert torch.equal((x + d) - x, d) and abs((up - down) / 2 - slope) < 0.01 * scale
