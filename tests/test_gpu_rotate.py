"""The norms of query and key heads with their rotation, and their gradient, on
the GPU against the oracle.

Tolerances, in half steps of FP32 (u = 2^-24): a sum of up to 512 squares in
chains of at most 16 and five exchanges is off by 21 u, so the root by 11 u, plus
4 u of the reciprocal root; the angle's fraction of a turn is rounded to 2^-25
half turns, 3.2 u of the rotated value, and sine and cosine add 4 u; five
roundings follow.  Together less than 2^-19 of the magnitudes behind a value;
the gradient takes the sums twice: 2^-18.  Sums over rows add a chain of at most
64 rows a thread and ten exchanges: 2^-17.  Outputs are rounded once more, by half
a step of their type."""
import numpy as np
import pytest
import torch

from mxcheck import ensure_built, to_f64
from oracle import step_oracle as S

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32
EPS = 1e-6


@pytest.fixture(scope="module")
def mx():
    ensure_built()
    import mxfp8_block_scaled_mx_gb300 as mx
    return mx


def inputs(tokens, hq, hk, dim, rotary, x, w, seed=0, start=1000):
    """q, k, their outputs' gradients (parts of wider rows), weights, positions, frequencies."""
    g = torch.Generator("cuda").manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    rows, grads = (n(tokens, hq + 2 * hk, dim) * 1.5).to(x), n(tokens, hq + hk, dim).to(x)
    w_q, w_k = ((n(dim) * 0.1 + 1).to(w) for _ in range(2))
    pos = torch.arange(tokens, device="cuda") * 3 + start
    f = torch.pow(500000.0, torch.arange(rotary // 2, dtype=torch.float64, device="cuda") * (-2.0 / rotary))
    return (rows[:, :hq], rows[:, hq:hq + hk], w_q, w_k, pos, f), (grads[:, :hq], grads[:, hq:])


def close(got, ref, mag, rel, what):
    got = to_f64(got)
    assert got.shape == ref.shape, what
    half = rel[1]
    bad = np.abs(got - ref) > rel[0] * mag + half * np.abs(ref) + 1e-37
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size}, worst {np.max(np.abs(got - ref) / (mag + 1e-37))}"


def half_step(t):
    return torch.finfo(t).eps / 2


def check_forward(mx, args, interleaved=False, scale=1.0, **kw):
    q, k, w_q, w_k, pos, f = args
    want = [S.norm_rotate(to_f64(x), to_f64(w), pos.cpu().numpy(), f.cpu().numpy(), interleaved, scale, EPS)
            for x, w in ((q, w_q), (k, w_k))]
    got = mx.norm_rotate(*args, interleaved=interleaved, scale=scale, eps=EPS, **kw)
    for name, y, (ref, mag) in zip("qk", got, want):
        assert y.dtype == q.dtype
        close(y, ref, mag, (2.0 ** -19, half_step(q.dtype)), name)
    return got


def check_backward(mx, args, grads, interleaved=False, scale=1.0):
    q, k, w_q, w_k, pos, f = args
    d = mx.norm_rotate_backward(*grads, *args, interleaved=interleaved, scale=scale, eps=EPS)
    for name, x, w, dy, dx, dw in (("q", q, w_q, grads[0], d.q, d.w_q), ("k", k, w_k, grads[1], d.k, d.w_k)):
        ref, mag, wref, wmag = S.norm_rotate_backward(to_f64(dy), to_f64(x), to_f64(w), pos.cpu().numpy(),
                                                      f.cpu().numpy(), interleaved, scale, EPS)
        assert dx.dtype == q.dtype and dw.dtype == FP32 and dx.is_contiguous()
        close(dx, ref, mag, (2.0 ** -18, half_step(q.dtype)), "d" + name)
        close(dw, wref, wmag, (2.0 ** -17, half_step(FP32)), "dw_" + name)
    return d


# every form of a row: 8, 16, 32 lanes of one slot, two slots; single channels
# in one, two, four and eight slots; odd lengths; one token, tokens that end
# inside a block, more tokens than blocks
SHAPES = [(1, 32, 8, 128, 128), (5, 3, 1, 64, 64), (7, 2, 2, 80, 32), (33, 1, 1, 128, 64),
          (9, 4, 2, 192, 192), (3, 5, 3, 256, 128), (6, 2, 1, 512, 256), (4, 2, 1, 50, 50),
          (11, 3, 2, 101, 100), (5, 1, 2, 200, 18), (2, 2, 2, 511, 510), (3, 1, 1, 2, 2),
          (2, 40, 24, 7, 4), (700, 2, 1, 16, 8),
          # full rows in part rotated, lanes of three slots, short single channels
          (9, 3, 2, 128, 64), (6, 3, 2, 96, 96), (5, 2, 1, 96, 32), (4, 2, 1, 192, 64), (7, 2, 1, 14, 6),
          (9, 3, 2, 30, 20)]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("x,w", [(BF16, BF16), (BF16, FP32), (FP32, FP32), (FP32, BF16)])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_both_directions(mx, shape, x, w, interleaved):
    args, grads = inputs(*shape, x, w, seed=sum(shape))
    check_forward(mx, args, interleaved, 1.0 if interleaved else 0.75)
    check_backward(mx, args, grads, interleaved, 1.0 if interleaved else 0.75)


def test_many_tokens(mx):
    """More tokens than the gradient has blocks, several of them a block."""
    for shape in ((1500, 3, 1, 64, 32), (20000, 1, 1, 8, 8)):
        args, grads = inputs(*shape, BF16, BF16)
        check_forward(mx, args)
        check_backward(mx, args, grads)


@pytest.mark.parametrize("start", [0, -100, 2 ** 20, 2 ** 31 - 10, -(2 ** 33)])
def test_positions_far_from_zero(mx, start):
    args, grads = inputs(6, 2, 1, 64, 64, FP32, FP32, start=start)
    check_forward(mx, args)
    if -(2 ** 31) <= start and start + 20 < 2 ** 31:
        args32 = (*args[:4], args[4].int(), args[5])
        a, b = mx.norm_rotate(*args), mx.norm_rotate(*args32)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        check_backward(mx, args32, grads)


def test_frequencies_of_any_size(mx):
    args, _ = inputs(6, 2, 1, 32, 12, FP32, FP32, start=17)
    f = torch.tensor([100.0, 1.0, 0.0, -0.5, 1e-30, 2.0 ** 40], dtype=torch.float64, device="cuda")
    # (2^40 radians a position times 17: the oracle is exact, the kernel's fraction of
    # a turn keeps the 64 bits of 2^66 / (2 pi): its error there is 2^-65 x 2^40 x 32)
    check_forward(mx, (*args[:5], f))


@pytest.mark.parametrize("x", [BF16, FP32])
@pytest.mark.parametrize("layout", ["heads first", "gaps", "off by one", "inputs of one head for all"])
def test_strides(mx, layout, x):
    (q, k, w_q, w_k, pos, f), (dq, dk) = inputs(9, 4, 2, 64, 32, x, x)
    if layout == "heads first":
        q, k, dq, dk = (t.transpose(0, 1).contiguous().transpose(0, 1) for t in (q, k, dq, dk))
    elif layout == "gaps":
        q, k = (torch.nn.functional.pad(t, (3, 6)) [:, :, 3:-6] for t in (q, k))
    elif layout == "off by one":
        def shift(t):
            flat = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
            flat[1:] = t.reshape(-1)
            return flat[1:].view(t.shape)
        q, k, dq, dk, w_q, w_k = map(shift, (q, k, dq, dk, w_q, w_k))
    else:
        q, dq = q[:, :1].expand(9, 4, 64), dq[:1].expand(9, 4, 64)
    args = (q, k, w_q, w_k, pos, f)
    check_forward(mx, args)
    check_backward(mx, args, (dq, dk))


@pytest.mark.parametrize("dim", [64, 30])
def test_in_place_in_a_products_rows(mx, dim):
    (q, k, w_q, w_k, pos, f), _ = inputs(40, 4, 2, dim, dim // 2 // 2 * 2, BF16, BF16)
    want = mx.norm_rotate(q, k, w_q, w_k, pos, f)
    rows = torch.cat([q, k, torch.full_like(k, 7.0)], 1)
    a, b = rows[:, :4], rows[:, 4:6]
    got = mx.norm_rotate(a, b, w_q, w_k, pos, f, out_q=a, out_k=b)
    assert got[0] is a and got[1] is b
    assert torch.equal(a, want[0]) and torch.equal(b, want[1]) and (rows[:, 6:] == 7).all()


def test_rows_of_zeros_infinities_and_nan(mx):
    args, grads = inputs(6, 2, 1, 64, 32, FP32, FP32)
    clean = mx.norm_rotate(*args)
    q = args[0].clone()
    q[1, 0], q[2, 1, 5], q[3, 0, 63] = 0.0, float("inf"), float("nan")
    args = (q, *args[1:])
    y, _ = mx.norm_rotate(*args)
    assert (y[1, 0] == 0).all() and y[2, 1].isnan().any() and y[3, 0].isnan().all()
    keep = torch.ones(6, 2, dtype=torch.bool, device="cuda")
    keep[1, 0] = keep[2, 1] = keep[3, 0] = False
    assert torch.equal(y[keep], clean[0][keep])
    d = mx.norm_rotate_backward(*grads, *args)
    assert torch.isfinite(d.q[keep]).all() and torch.isfinite(d.k).all() and torch.isfinite(d.w_k).all()
    assert torch.isfinite(d.q[1, 0]).all()


def test_without_tokens(mx):
    args, grads = inputs(0, 2, 1, 64, 32, BF16, FP32)
    q, k = mx.norm_rotate(*args)
    assert q.shape == (0, 2, 64) and k.shape == (0, 1, 64)
    d = mx.norm_rotate_backward(*grads, *args)
    assert d.q.shape == (0, 2, 64) and (d.w_q == 0).all() and (d.w_k == 0).all()


@pytest.mark.parametrize("tokens", [1, 5, 153, 777, 5000])
@pytest.mark.parametrize("dim,rotary", [(80, 32), (128, 128), (256, 64), (34, 34)])
def test_nothing_is_read_from_a_workspace_that_was_not_written(mx, tokens, dim, rotary):
    args, grads = inputs(tokens, 3, 1, dim, rotary, BF16, FP32)
    need = mx.mx_norm_rotate_backward_workspace(tokens, dim)
    a, b = (mx.norm_rotate_backward(*grads, *args, workspace=torch.full((need,), fill, dtype=torch.uint8, device="cuda"))
            for fill in (0, 255))
    assert all(torch.equal(u, v) for u, v in zip(vars(a).values(), vars(b).values()))


def test_same_bits_again_and_a_workspace(mx):
    args, grads = inputs(3000, 4, 2, 128, 128, BF16, BF16)
    a = mx.norm_rotate_backward(*grads, *args)
    need = mx.mx_norm_rotate_backward_workspace(3000, 128)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    b = mx.norm_rotate_backward(*grads, *args, workspace=ws)
    assert all(torch.equal(u, v) for u, v in zip(vars(a).values(), vars(b).values()))
    with pytest.raises(ValueError):
        mx.norm_rotate_backward(*grads, *args, workspace=ws[:-1])


def test_refusals(mx):
    (q, k, w_q, w_k, pos, f), (dq, dk) = inputs(4, 2, 1, 64, 32, BF16, BF16)
    bad = [dict(q=q.float()), dict(k=k[:3]), dict(w_q=w_q[:63]), dict(w_k=w_k.float()), dict(positions=pos.float()),
           dict(positions=pos[:3]), dict(positions=pos[:, None]), dict(frequencies=f.float()), dict(frequencies=f[:0]),
           dict(frequencies=torch.cat([f, f, f])), dict(q=q.transpose(1, 2)), dict(q=q[0]), dict(k=k.cpu()),
           dict(positions=torch.arange(8, device="cuda")[::2])]
    good = dict(q=q, k=k, w_q=w_q, w_k=w_k, positions=pos, frequencies=f)
    for b in bad:
        with pytest.raises(ValueError):
            mx.norm_rotate(**{**good, **b})
        with pytest.raises(ValueError):
            mx.norm_rotate_backward(dq, dk, **{**good, **b})
    for d in ((dq[:3], dk), (dq, dk.float()), (dq.cpu(), dk)):
        with pytest.raises(ValueError):
            mx.norm_rotate_backward(*d, **good)
    with pytest.raises(ValueError):
        mx.norm_rotate(**good, out_q=q[:, :1])
    with pytest.raises(mx.MxError):     # rows of an output that overlap
        mx.norm_rotate(**good, out_q=torch.empty_like(q[:, :1]).expand(4, 2, 64))
    with pytest.raises(mx.MxError):
        mx.norm_rotate(**good, eps=-1.0)


@pytest.mark.parametrize("x", [BF16, FP32])
def test_autograd(mx, x):
    args, grads = inputs(20, 3, 2, 64, 32, x, FP32)
    leaves = [t.detach().clone().requires_grad_() for t in args[:4]]
    q, k = mx.norm_rotate(*leaves, *args[4:], interleaved=True, scale=1.25)
    got = torch.autograd.grad([q, k], leaves, grads)
    d = mx.norm_rotate_backward(*grads, *args, interleaved=True, scale=1.25)
    for a, b, t in zip(got, (d.q, d.k, d.w_q, d.w_k), leaves):
        assert a.dtype == t.dtype and torch.equal(a, b.to(t.dtype))
    # one output alone, with an expanded gradient; only one input that asks
    q, k = mx.norm_rotate(*leaves, *args[4:])
    g, = torch.autograd.grad(k.sum(), leaves[1:2])
    assert torch.equal(g, mx.norm_rotate_backward(torch.zeros_like(args[0]), torch.ones_like(args[1]), *args).k)
    out = torch.empty_like(args[0])
    q, _ = mx.norm_rotate(*leaves, *args[4:], out_q=out)
    assert q is out and q.requires_grad


def test_gradient_against_differences(mx):
    """Central differences of the kernel's own FP32 forward pass: with a step of 2^-7
    the third-order term and the rounding of the differences stay below 2^-9 of the
    largest gradient."""
    args, grads = inputs(2, 1, 1, 16, 8, FP32, FP32)
    d = mx.norm_rotate_backward(*grads, *args)

    def total(q, w_q):
        y, _ = mx.norm_rotate(q, args[1], w_q, *args[3:])
        return (y.double() * grads[0].double()).sum().item()

    h = 2.0 ** -7
    for t, got, f in ((args[0], d.q, lambda v: total(v, args[2])), (args[2], d.w_q, lambda v: total(args[0], v))):
        big = got.abs().max().item()
        for i in range(t.numel()):
            step = torch.zeros(t.numel(), device="cuda")
            step[i] = h
            diff = (f(t + step.view(t.shape)) - f(t - step.view(t.shape))) / (2 * h)
            assert abs(diff - got.reshape(-1)[i].item()) < 2.0 ** -9 * big
