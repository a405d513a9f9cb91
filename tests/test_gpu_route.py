"""Routing with its balance loss, and its gradient, on the GPU against the
oracle.

Whole numbers are equal.  Tolerances (u = 2^-24): an exponential is off by 2 u and by
its argument's rounding, at most 32 u here (logits within 32 of a row's largest
that matter); a sum of up to 512 exponentials in chains of 16 and five exchanges by
21 u; quotients add 4 u: less than 2^-18 of a weight or a probability.  The sums
over tokens run in chains of at most 64 tokens, eight warps and 304 blocks: 400 u
more, 2^-15 of the balance loss.  Its gradient and the weights' are differences of
such terms: 2^-17 of the magnitudes behind them, then the output's half step."""
import numpy as np
import pytest
import torch

from mxcheck import ensure_built, to_f64
from oracle import step_oracle as S

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def mx():
    ensure_built()
    import mxfp8_block_scaled_mx_gb300 as mx
    return mx


def logits(tokens, experts, dtype, seed=0):
    g = torch.Generator("cuda").manual_seed(seed)
    z = torch.randn((tokens, experts), generator=g, device="cuda")
    return (z + torch.randn(experts, generator=g, device="cuda") * 0.5).to(dtype)


def check(mx, z, k, renormalize=True, mask=None, finite=True):
    r = mx.route(z, k, renormalize, mask)
    ref = S.route(to_f64(z), k, renormalize, None if mask is None else mask.cpu().numpy())
    for name in ("ids", "counts", "offsets", "order"):
        got = getattr(r, name)
        assert got.dtype == torch.int32
        assert np.array_equal(got.cpu().numpy(), ref[name]), name
    assert r.balance.shape == () and r.weights.dtype == FP32
    if finite:
        assert np.allclose(to_f64(r.weights), ref["weights"], rtol=2.0 ** -18, atol=1e-37)
        assert abs(r.balance.item() - ref["balance"]) <= 2.0 ** -15 * ref["balance"]
        assert (np.abs(to_f64(r.lse) - ref["lse"]) <= 2.0 ** -18 + 2.0 ** -22 * np.abs(ref["lse"])).all()
    return r, ref


def check_backward(mx, z, k, renormalize=True, mask=None, use=(True, True, True), seed=5):
    r, ref = check(mx, z, k, renormalize, mask)
    g = torch.Generator("cuda").manual_seed(seed)
    dw = torch.randn(r.weights.shape, generator=g, device="cuda") if use[0] else None
    db = torch.tensor(3.0, device="cuda") if use[1] else None
    dl = torch.randn(len(z), generator=g, device="cuda") if use[2] else None
    d = mx.route_backward(dw, db, z, r, renormalize, mask, dl)
    zero = np.zeros(ref["weights"].shape)
    want, mag = S.route_backward(ref, k, renormalize, zero if dw is None else to_f64(dw), 3.0 if use[1] else 0.0,
                                 zero[:, 0] if dl is None else to_f64(dl))
    assert d.dtype == z.dtype and d.shape == z.shape
    err = np.abs(to_f64(d) - want)
    half = torch.finfo(z.dtype).eps / 2
    assert (err <= 2.0 ** -17 * mag + half * np.abs(want) + 1e-37).all(), np.max(err / (mag + 1e-37))
    return r


SHAPES = [(1, 128, 8), (1, 1, 1), (2, 2, 2), (63, 20, 3), (64, 64, 8), (65, 64, 8), (33, 33, 5), (300, 8, 2),
          (1000, 32, 32), (129, 65, 6), (200, 200, 7), (77, 257, 9), (40, 512, 32), (5000, 64, 8), (9731, 5, 4)]


@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_both_directions(mx, shape, dtype, masked, renormalize):
    tokens, experts, k = shape
    z = logits(tokens, experts, dtype, seed=tokens)
    mask = torch.arange(tokens, device="cuda") % 3 != 1 if masked else None
    check_backward(mx, z, k, renormalize, mask)


@pytest.mark.parametrize("tokens", [5, 500])
def test_masks(mx, tokens):
    z = logits(tokens, 16, FP32)
    for mask in (torch.zeros(tokens, dtype=torch.bool, device="cuda"),
                 torch.ones(tokens, dtype=torch.uint8, device="cuda") * 255):
        r = check_backward(mx, z, 4, True, mask)
    none = check_backward(mx, z, 4, True, torch.zeros(tokens, dtype=torch.uint8, device="cuda"))
    assert none.balance.item() == 0 and (none.counts == 0).all() and none.offsets[-1].item() == tokens * 4
    assert r.counts.sum().item() == tokens * 4


@pytest.mark.parametrize("use", [(True, False, False), (False, True, False), (False, False, True),
                                 (False, False, False)])
@pytest.mark.parametrize("renormalize", [True, False])
def test_gradients_one_by_one(mx, use, renormalize):
    check_backward(mx, logits(90, 40, FP32), 6, renormalize, None, use)


@pytest.mark.parametrize("experts", [24, 64, 130])
def test_ties(mx, experts):
    """Equal logits, among them +0 and -0: the lowest index first."""
    for tokens in (200, 16389):
        for z in (torch.zeros(tokens, experts), torch.randint(-2, 3, (tokens, experts)).float(),
                  torch.where(torch.rand(tokens, experts) < 0.5, 0.0, -0.0)):
            for dtype in (BF16, FP32):
                check(mx, z.to(dtype).cuda(), 8)


@pytest.mark.parametrize("tokens", [3, 200, 16500])
@pytest.mark.parametrize("experts", [8, 48, 300])
def test_special_logits(mx, tokens, experts):
    z = logits(tokens, experts, FP32)
    z[0, ::2] = float("-inf")
    z[1, 3], z[1, 1] = float("nan"), float("-inf")
    z[2, 4] = float("-inf")
    r, ref = check(mx, z, 6, finite=False)
    assert r.weights[1].isnan().all() and r.lse[1].isnan()
    ok = torch.arange(tokens, device="cuda") != 1
    assert np.allclose(to_f64(r.weights[ok]), ref["weights"][ok.cpu().numpy()], rtol=2.0 ** -18, atol=1e-37)
    assert r.balance.isnan()
    # a token that does not count touches nothing
    r, ref = check(mx, z, 6, True, ok, finite=False)
    assert abs(r.balance.item() - ref["balance"]) <= 2.0 ** -15 * ref["balance"]
    d = mx.route_backward(None, torch.tensor(1.0, device="cuda"), z, r, True, ok)
    assert torch.isfinite(d[ok]).all()
    # nothing but the lowest, +infinity, NaN throughout
    z[0], z[1], z[2, 5] = float("-inf"), float("nan"), float("inf")
    r, _ = check(mx, z, 6, finite=False)
    assert r.weights[:3].isnan().all() and r.ids[0].tolist() == r.ids[1].tolist() == list(range(6))
    # the lowest finite value as a mask
    z = logits(tokens, experts, FP32)
    z[:, experts // 2:] = torch.finfo(FP32).min
    check(mx, z, experts // 2 if experts < 60 else 20)


def test_strided_logits(mx):
    for dtype in (BF16, FP32):
        for tokens in (300, 33000):
            wide = logits(tokens, 80, dtype)
            for z in (wide[:, :64], wide[:, 1:62], wide[::2, 4:36]):
                check_backward(mx, z, 4)


@pytest.mark.parametrize("tokens,experts,top_k", [(80000, 512, 2), (200000, 64, 8), (300000, 130, 1), (120000, 33, 32)])
def test_more_tokens_of_a_block_than_it_places_at_a_time(mx, tokens, experts, top_k):
    check(mx, logits(tokens, experts, FP32), top_k)


def test_without_tokens(mx):
    z = torch.zeros(0, 8, device="cuda")
    r = mx.route(z, 2)
    assert r.ids.shape == (0, 2) and (r.counts == 0).all() and (r.offsets == 0).all() and r.balance.item() == 0
    assert mx.route_backward(None, r.balance, z, r).shape == (0, 8)


def test_same_bits_again_and_a_workspace(mx):
    for tokens in (3000, 20000):
        z = logits(tokens, 64, FP32)
        a = mx.route(z, 8)
        ws = torch.full((mx.mx_route_workspace(tokens, 64),), 255, dtype=torch.uint8, device="cuda")
        b = mx.route(z, 8, workspace=ws)
        assert all(torch.equal(u, v) for u, v in zip(vars(a).values(), vars(b).values()))
        with pytest.raises(ValueError):
            mx.route(z, 8, workspace=ws[:-1])


@pytest.mark.parametrize("tokens,experts,top_k", [(1, 1, 1), (1, 128, 8), (33, 20, 3), (1025, 7, 7), (4097, 20, 3),
                                                  (16384, 33, 4), (16385, 512, 8), (40001, 64, 8)])
def test_nothing_is_read_from_a_workspace_that_was_not_written(mx, tokens, experts, top_k):
    z = logits(tokens, experts, FP32)
    need = mx.mx_route_workspace(tokens, experts)
    a, b = (mx.route(z, top_k, workspace=torch.full((need,), fill, dtype=torch.uint8, device="cuda"))
            for fill in (0, 255))
    assert all(torch.equal(u, v) for u, v in zip(vars(a).values(), vars(b).values()))


def test_refusals(mx):
    z = logits(10, 8, FP32)
    r = mx.route(z, 2)
    mask = torch.ones(10, dtype=torch.bool, device="cuda")
    for bad in (lambda: mx.route(z, 0), lambda: mx.route(z, 9), lambda: mx.route(z.double(), 2), lambda: mx.route(z[0], 2),
                lambda: mx.route(z.t(), 2), lambda: mx.route(z, 2, mask=mask[:9]), lambda: mx.route(z, 2, mask=mask.float()),
                lambda: mx.route(z, 2, mask=mask.cpu()), lambda: mx.route(logits(4, 600, FP32), 2),
                lambda: mx.route(logits(4, 64, FP32), 33),
                lambda: mx.route_backward(r.weights[:9], None, z, r), lambda: mx.route_backward(None, r.weights, z, r),
                lambda: mx.route_backward(None, None, z[:9], r), lambda: mx.route_backward(None, None, z, r, d_lse=r.lse[:9])):
        with pytest.raises(ValueError):
            bad()


def test_ids_out_of_range_are_passed_over(mx):
    z = logits(50, 24, FP32)
    r = mx.route(z, 4)
    dw = torch.randn_like(r.weights)
    r.ids[3, 1], r.ids[4, 2], r.ids[5, 0] = -1, 24, 2 ** 30
    d = mx.route_backward(dw, None, z, r)
    assert torch.isfinite(d).all() and mx.device_status() == 0


def test_autograd(mx):
    for dtype in (BF16, FP32):
        z = logits(200, 24, dtype).requires_grad_()
        mask = torch.arange(200, device="cuda") < 150
        r = mx.route(z, 4, False, mask)
        assert not r.ids.requires_grad and not r.order.requires_grad and r.weights.requires_grad
        dw = torch.randn_like(r.weights)
        g, = torch.autograd.grad((r.weights * dw).sum() + 2 * r.balance + (r.lse ** 2).mean(), z)
        q = mx.route(z.detach(), 4, False, mask)
        want = mx.route_backward(dw, torch.tensor(2.0, device="cuda"), z.detach(), q, False, mask, 2 * q.lse / 200)
        assert g.dtype == dtype
        if dtype == FP32:   # (the gradient of the mean of squares may be rounded otherwise)
            assert torch.allclose(g, want, rtol=1e-5, atol=1e-7)
        r = mx.route(z, 4, False, mask)
        g, = torch.autograd.grad(r.balance, z)
        assert torch.equal(g, mx.route_backward(None, torch.ones((), device="cuda"), z.detach(), q, False, mask))


def test_gradient_against_differences(mx):
    """Central differences of the balance loss and the weights: steps of 2^-6, whose
    third-order term and the FP32 values' rounding stay below 2^-8 of the largest."""
    z = logits(12, 6, FP32)
    # apart, so that a step changes no winner
    z = (torch.argsort(torch.argsort(z, 1), 1) * 0.3).float()
    r = mx.route(z, 2, True)
    dw = torch.randn(12, 2, generator=torch.Generator("cuda").manual_seed(1), device="cuda")
    d = mx.route_backward(dw, torch.tensor(5.0, device="cuda"), z, r)

    def total(v):
        q = mx.route(v, 2, True)
        return ((q.weights.double() * dw.double()).sum() + 5 * q.balance.double()).item()

    h, big = 2.0 ** -6, d.abs().max().item()
    for i in range(z.numel()):
        step = torch.zeros(z.numel(), device="cuda")
        step[i] = h
        step = step.view(z.shape)
        diff = (total(z + step) - total(z - step)) / (2 * h)
        assert abs(diff - d.reshape(-1)[i].item()) < 2.0 ** -8 * big


def test_feeds_the_grouped_products(mx):
    """offsets and order as the grouped quantization and product take them."""
    tokens, experts, k, hidden, n = 300, 12, 3, 128, 128
    z = logits(tokens, experts, FP32)
    x = torch.randn(tokens, hidden, device="cuda").bfloat16()
    w = (torch.randn(experts, n, hidden, device="cuda") * 0.05).bfloat16()
    r = mx.route(z, k)
    rows = x[torch.div(r.order, k, rounding_mode="floor").long()]
    qx = mx.quantize_grouped(rows, r.offsets, "e4m3")
    qw = mx.quantize(w.view(-1, hidden), "e4m3", "row")
    y = mx.grouped_gemm(qx, r.offsets, mx.MxTensor(qw.codes.view(experts, n, hidden), qw.scales, "e4m3"), "fp32")
    assert mx.device_status() == 0
    pairs = torch.empty_like(y)
    pairs[r.order.long()] = y
    got = (pairs.view(tokens, k, n) * r.weights[..., None]).sum(1)
    want = torch.einsum("tk,tkn->tn", r.weights.double(),
                        torch.einsum("th,tknh->tkn", x.double(), w.double()[r.ids.long()]))
    # two E4M3 roundings, of 2^-4 each, and a scale's: their sum of 128 terms stays
    # within a quarter of the norm
    assert (got - want).norm() < 0.25 * want.norm()
