"""Sizes at which the training step's operators take a path of their own, against the
oracle: contractions of several runs in the vocabulary loss, routing of many tokens
over 65 to 128 experts and around the rules that choose a kernel, more heads than a
block takes at a time, elements further apart than 32 bits count.

Tolerances are those of the operators' own tests (their checks are used here); the
sums over tokens of the routing below run in chains of at most 96 rows a lane, 27 warps,
5 blocks a thread and 32 threads, which is less than the 400 half steps allowed."""
import pytest
import torch

import test_gpu_rotate as rotate
import test_gpu_route as routing
import test_gpu_vocab_loss as loss
from mxcheck import ensure_built

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def mx():
    ensure_built()
    import mxfp8_block_scaled_mx_gb300 as mx
    return mx


# ------------------------------------------------------------------ vocabulary loss

# (runs of at most 16 steps of 64: two, three and four of them, the last short or as
# long as the others; more tiles than pairs of blocks, or than blocks where tokens are
# few, in boxes of 16, 32 and 64)
RUNS = [(130, 1032, 20000), (300, 2056, 10300), (257, 4096, 700), (66, 1088, 40), (70, 2048, 513),
        (1, 4096, 20001), (20, 1032, 20001), (32, 2056, 300), (40, 1088, 20001), (64, 4096, 2000)]


@pytest.mark.parametrize("shape", RUNS, ids=str)
def test_loss_of_several_runs(mx, shape):
    x, w, labels = loss.inputs(*shape, seed=sum(shape))
    loss.check(mx, x, w, labels)
    loss.check_backward(mx, x, w, labels)
    assert mx.device_status() == 0


@pytest.mark.parametrize("tokens", [1, 17, 64, 130, 300])
def test_runs_keep_what_one_accumulator_would_cut_off(mx, tokens):
    """The first 1024 terms of a logit make 2^20, the other 3072 are 2^-8 each, 12
    together (or nothing, in every other column).  In a single FP32 accumulator, whose
    step at 2^20 is 2^-3, sixteen of them at a time are lost; in runs of 1024 all sums
    are exact, the last ones in FP32 too.

    lse is 2^20 + 12 + log(columns) of a logit of such size: its product with log2 e is
    rounded by 2^-4 and by the constant's 2^-25, that with ln 2 by as much and its sum by
    2^-4: together less than 1/4."""
    hidden, vocab = 4096, 520
    x = torch.ones(tokens, hidden, dtype=BF16, device="cuda")
    w = torch.zeros(vocab, hidden, dtype=BF16, device="cuda")
    w[:, :1024] = 2.0 ** 10
    w[::2, 1024:] = 2.0 ** -8
    labels = torch.arange(tokens, device="cuda")
    value, lse = mx.linear_cross_entropy(x, w, labels)
    want = 2.0 ** 20 + 12 + torch.tensor(260 + 260 * 2.718281828459045 ** -12, dtype=torch.float64).log()
    z = 2.0 ** 20 + 12 * (labels % 2 == 0).double()
    assert ((lse.double() - want.item()).abs() < 0.25).all()
    assert ((value.double() - (want.item() - z)).abs() < 0.25).all()
    assert mx.device_status() == 0


@pytest.mark.parametrize("tokens", [1, 17, 64, 130, 300])
def test_the_gradient_exponentiates_the_logits_of_the_losses(mx, tokens):
    """Logits of 2^15, every other one with 3072 terms of 2^-13 more, 3/8 together, of
    which a single accumulator (step 2^-8) would lose all: a gradient whose logits were
    summed in another way than those of lse would give these columns two thirds of
    their probability.

    Exponents are off by 2^-9 each of lse's last rounding and of log2 e and ln 2 and, in the
    gradient, of lse's product with log2 e and the logit's: less than 2^-7; dz is rounded
    by 2^-8 at most, sums of 300 equal terms by less than 2^-16."""
    hidden, vocab = 4096, 520
    x = torch.ones(tokens, hidden, dtype=BF16, device="cuda")
    w = torch.zeros(vocab, hidden, dtype=BF16, device="cuda")
    w[:, :1024] = 2.0 ** 5
    w[::2, 1024:] = 2.0 ** -13
    labels = torch.full((tokens,), -100, device="cuda")
    _, lse = mx.linear_cross_entropy(x, w, labels)
    ones = torch.ones(tokens, device="cuda")
    _, dw = mx.linear_cross_entropy_backward(None, ones, x, w, labels, lse, weight_dtype="fp32")
    z = torch.zeros(vocab, dtype=torch.float64)
    z[::2] = 0.375
    want = tokens * torch.softmax(z, 0)[:, None].cuda()
    assert ((dw.double() - want).abs() <= (2.0 ** -7 + 2.0 ** -8 + 2.0 ** -16) * 1.01 * want).all()
    assert mx.device_status() == 0


# ------------------------------------------------------------------ routing

# (a lane a token from 8192 tokens and 128 an expert on, up to 128 experts and 8
# winners: the form of 65 to 128 experts, in one round of warps and in several; each rule
# from both sides)
WIDE = [(16389, 128, 8), (8321, 65, 8), (14001, 100, 3), (100003, 128, 8), (50001, 97, 1),
        (16383, 128, 8), (16384, 128, 8), (8319, 65, 8), (8320, 65, 8), (8191, 64, 8), (8192, 64, 8),
        (20000, 128, 9), (20000, 129, 8)]


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("shape", WIDE, ids=str)
def test_routing_of_many_tokens(mx, shape, dtype, masked):
    tokens, experts, k = shape
    z = routing.logits(tokens, experts, dtype, seed=experts)
    mask = torch.arange(tokens, device="cuda") % 5 != 2 if masked else None
    routing.check_backward(mx, z, k, not masked, mask)


@pytest.mark.parametrize("experts", [65, 72, 100, 128])
def test_special_logits_of_many_tokens(mx, experts):
    routing.test_special_logits(mx, 16500, experts)


@pytest.mark.parametrize("experts", [70, 96, 128])
def test_ties_of_many_tokens(mx, experts):
    """16389 tokens, equal logits (among them +0 and -0): the lowest index first."""
    routing.test_ties(mx, experts)


def test_strided_logits_of_many_tokens(mx):
    for dtype in (BF16, FP32):
        wide = routing.logits(33000, 140, dtype)
        for z in (wide[:, :128], wide[:, 1:101], wide[::2, 4:104]):
            routing.check_backward(mx, z, 6)


# ------------------------------------------------------------------ heads' norms

# (more heads than the places of an item's rows, and tokens for every block: a block
# goes from part to part of a token's heads, queries and keys in one part, the last short)
MANY_HEADS = [(400, 64, 17, 256, 128, BF16), (500, 9, 4, 512, 512, FP32), (400, 70, 9, 101, 100, BF16),
              (333, 60, 60, 64, 64, FP32), (200, 300, 5, 96, 96, BF16)]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("shape", MANY_HEADS, ids=str)
def test_many_heads_of_many_tokens(mx, shape, interleaved):
    *sizes, x = shape
    args, grads = rotate.inputs(*sizes, x, FP32, seed=1)
    want = rotate.check_forward(mx, args, interleaved)
    rotate.check_backward(mx, args, grads, interleaved)
    q, k = (t.clone(memory_format=torch.contiguous_format) for t in args[:2])
    got = mx.norm_rotate(q, k, *args[2:], interleaved=interleaved, eps=rotate.EPS, out_q=q, out_k=k)
    assert got[0] is q and torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert mx.device_status() == 0


# ------------------------------------------------------------------ beyond 32 bits

def apart(t, stride, offset=0):
    """A copy of t whose rows lie `stride` elements apart, `offset` into a buffer."""
    rows = t.reshape(len(t), -1)
    buf = torch.empty(offset + (len(t) - 1) * stride + rows.shape[1], dtype=t.dtype, device="cuda")
    far = buf[offset:].as_strided(rows.shape, (stride, 1))
    far.copy_(rows)
    return buf[offset:].as_strided(t.shape, (stride, *t.stride()[1:]))


def test_heads_far_apart(mx):
    args, grads = rotate.inputs(17, 3, 1, 64, 32, BF16, BF16)
    near = [t.contiguous() for t in (*args[:2], *grads)]
    q, k, dq, dk = (apart(t, 2 ** 28 - 64, 8) for t in near)
    a = mx.norm_rotate(*near[:2], *args[2:])
    b = mx.norm_rotate(q, k, *args[2:])
    assert all(torch.equal(u, v) for u, v in zip(a, b))
    a = mx.norm_rotate_backward(*near[2:], *near[:2], *args[2:])
    b = mx.norm_rotate_backward(dq, dk, q, k, *args[2:])
    assert all(torch.equal(u, v) for u, v in zip(vars(a).values(), vars(b).values()))
    got = mx.norm_rotate(q, k, *args[2:], out_q=q, out_k=k)
    want = mx.norm_rotate(*near[:2], *args[2:])
    assert got[0] is q and torch.equal(q, want[0]) and torch.equal(k, want[1])


@pytest.mark.parametrize("tokens,experts,stride", [(40, 64, 2 ** 27), (3000, 200, 2 ** 21), (9000, 64, 2 ** 19)])
def test_logits_far_apart(mx, tokens, experts, stride):
    z = routing.logits(tokens, experts, BF16)
    far = apart(z, stride)
    a, b = mx.route(z, 4), mx.route(far, 4)
    assert all(torch.equal(u, v) for u, v in zip(vars(a).values(), vars(b).values()))
    one = torch.ones((), device="cuda")
    assert torch.equal(mx.route_backward(a.weights, one, z, a), mx.route_backward(a.weights, one, far, a))


def test_as_many_tokens_and_experts_as_routing_takes(mx):
    """2^31 logits less a few: every token's own outputs are those of a smaller call;
    offsets, order and counts belong together."""
    tokens, experts, k = 4194303, 512, 2
    z = torch.randn(1 << 16, experts, device="cuda").bfloat16().repeat(64, 1)[:tokens]
    r, few = mx.route(z, k), mx.route(z[:1 << 16], k)
    for name in ("ids", "weights", "lse"):
        got, want = getattr(r, name), getattr(few, name)
        for at in range(0, tokens, 1 << 16):
            part = got[at:at + (1 << 16)]
            assert torch.equal(part, want[:len(part)]), (name, at)
    flat = r.ids.flatten()
    counts = torch.bincount(flat, minlength=experts)
    assert torch.equal(r.counts.long(), counts)
    assert torch.equal(r.offsets[1:].long(), counts.cumsum(0)) and r.offsets[0].item() == 0
    assert torch.equal(r.order.long(), torch.sort(flat, stable=True).indices)
    d = torch.randn(1 << 16, k, device="cuda").repeat(64, 1)[:tokens].contiguous()
    got, want = mx.route_backward(d, None, z, r), mx.route_backward(d[:1 << 16], None, z[:1 << 16], few)
    for at in range(0, tokens, 1 << 16):
        part = got[at:at + (1 << 16)]
        assert torch.equal(part, want[:len(part)]), at
    assert mx.device_status() == 0


@pytest.mark.parametrize("tokens", [5, 130])
def test_rows_of_the_loss_far_apart(mx, tokens):
    x, w, labels = loss.inputs(tokens, 72, 130)
    far_x, far_w = apart(x, 2 ** 32 // (tokens - 1) // 8 * 8 + 8), apart(w, 2 ** 25 + 8)
    a, b = mx.linear_cross_entropy(x, w, labels), mx.linear_cross_entropy(far_x, far_w, labels)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    ones = torch.ones(tokens, device="cuda")
    a = mx.linear_cross_entropy_backward(ones, None, x, w, labels, a[1])
    b = mx.linear_cross_entropy_backward(ones, None, far_x, far_w, labels, b[1])
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("tokens", [3, 70])
def test_weights_of_more_than_two_to_the_31_elements(mx, tokens):
    """Losses against a softmax in 64 bits, a piece of the vocabulary at a time; rows of
    the weights' gradient from its start, its middle and its end."""
    hidden, vocab = 2056, (1 << 20) + 5
    g = torch.Generator("cuda").manual_seed(tokens)
    w = torch.empty(vocab, hidden, dtype=BF16, device="cuda")
    for v in range(0, vocab, 1 << 17):
        part = w[v:v + (1 << 17)]
        part.copy_(torch.randn(part.shape, generator=g, device="cuda") * 2 / hidden ** 0.5)
    x = torch.randn(tokens, hidden, generator=g, device="cuda").to(BF16)
    labels = vocab - 1 - 7 * torch.arange(tokens, device="cuda")
    z = torch.cat([x.double() @ w[v:v + (1 << 17)].double().T for v in range(0, vocab, 1 << 17)], 1)
    want = torch.logsumexp(z, 1)
    value, lse = mx.linear_cross_entropy(x, w, labels)
    mag = max((x.double().abs() @ w[v:v + (1 << 17)].double().abs().T).max().item() for v in range(0, vocab, 1 << 17))
    tol = loss.z_error(hidden, mag) + 2.0 ** -20 + 2.0 ** -22 * want.abs().max().item()
    assert ((lse.double() - want).abs() <= tol).all()
    assert ((value.double() - (want - z.gather(1, labels[:, None])[:, 0])).abs() <= 2 * tol).all()
    d = torch.full((tokens,), 1.0 / tokens, device="cuda")
    _, dw = mx.linear_cross_entropy_backward(d, None, x, w, labels, lse, need_x=False)
    for lo in (0, vocab // 2, vocab - 600):
        p = torch.exp(z[:, lo:lo + 600] - want[:, None]) / tokens
        for t in range(tokens):
            at = int(labels[t]) - lo
            if 0 <= at < 600:
                p[t, at] -= 1.0 / tokens
        ref, m = p.T @ x.double(), p.abs().T @ x.double().abs()
        # dz: half a step of bf16 and the softmax's relative error; sums; the output's half step
        bound = (2.0 ** -8 + 2 * tol + 2.0 ** -18) * 1.01 * m
        assert ((dw[lo:lo + 600].double() - ref).abs() <= bound + 2.0 ** -8 * (ref.abs() + bound) + 1e-37).all(), lo
    assert mx.device_status() == 0
