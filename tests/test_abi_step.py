"""Host-only checks of the C entries of the operators between the products:
sizes of workspaces, and refusal of invalid arguments before a device is
touched; and of the helper that makes their frequencies."""
import math

import pytest

from mxcheck import ensure_built

FAKE = 0x10000


@pytest.fixture(scope="module")
def mx():
    ensure_built()
    import mxfp8_block_scaled_mx_gb300 as mx
    return mx


SIZES = dict(tokens=4, q_heads=3, k_heads=2, dim=64, rotary=32)
HEADS = dict(q=FAKE, q_st=320, q_sh=64, k=FAKE, k_st=320, k_sh=64, x=0, w_q=FAKE, w_k=FAKE, w=0,
             positions=FAKE, position_bits=64, frequencies=FAKE, interleaved=0, scale=1.0, eps=1e-6)
ROTATE = dict(**SIZES, **HEADS, out_q=FAKE, oq_st=192, oq_sh=64, out_k=FAKE, ok_st=128, ok_sh=64,
              stream=0)
ROTATE_BACK = dict(**SIZES, d_q=FAKE, dq_st=192, dq_sh=64, d_k=FAKE, dk_st=128, dk_sh=64, **HEADS,
                   dx_q=FAKE, dx_k=FAKE, dw_q=FAKE, dw_k=FAKE, workspace=FAKE,
                   workspace_bytes=1 << 40, stream=0)
ROUTE = dict(tokens=100, experts=8, top_k=2, logits=FAKE, ld=8, dtype=0, mask=None, renormalize=1,
             ids=FAKE, weights=FAKE, lse=FAKE, counts=FAKE, offsets=FAKE, order=FAKE, balance=FAKE,
             workspace=FAKE, workspace_bytes=1 << 40, stream=0)
ROUTE_BACK = dict(tokens=100, experts=8, top_k=2, d_weights=FAKE, d_balance=FAKE, d_lse=FAKE,
                  logits=FAKE, ld=8, dtype=0, mask=None, renormalize=1, ids=FAKE, weights=FAKE,
                  lse=FAKE, counts=FAKE, d_logits=FAKE, stream=0)
LOSS = dict(tokens=4, hidden=64, vocab=100, x=FAKE, ldx=64, w=FAKE, ldw=64, labels=FAKE,
            label_bits=64, ignore_index=-100, loss=FAKE, lse=FAKE, workspace=FAKE,
            workspace_bytes=1 << 40, stream=0)
LOSS_BACK = dict(tokens=4, hidden=64, vocab=100, d_loss=FAKE, d_lse=FAKE, x=FAKE, ldx=64, w=FAKE,
                 ldw=64, labels=FAKE, label_bits=64, ignore_index=-100, lse=FAKE, dx=FAKE, dw=FAKE,
                 dw_dtype=0, workspace=FAKE, workspace_bytes=1 << 40, stream=0)


def rotate_refusals(call, outputs, pointers):
    for name in pointers:
        assert call(**{name: None}) == 1, name
    for name in ("q_heads", "k_heads"):
        assert call(**{name: 0}) == 1
    assert call(tokens=-1) == 1 and call(dim=1, rotary=2) == 1
    assert call(rotary=0) == 1 and call(rotary=31) == 1 and call(rotary=66) == 1
    assert call(x=2) == 1 and call(w=2) == 1 and call(position_bits=16) == 1
    assert call(eps=-1.0) == 1 and call(eps=float("nan")) == 1
    assert call(q_st=-1) == 1 and call(k_sh=-64) == 1
    assert call(dim=514, **{n: 514 * 8 for n in outputs}) == 3
    assert call(tokens=1 << 30) == 3
    assert call(q=FAKE + 1) == 2 and call(x=1, k=FAKE + 2) == 2 and call(w=1, w_k=FAKE + 2) == 2
    assert call(frequencies=FAKE + 4) == 2 and call(positions=FAKE + 4) == 2


def test_rotated_norm_rejects_bad_arguments_on_the_host(mx):
    call = lambda **kw: mx.mx_norm_rotate(*{**ROTATE, **kw}.values())  # noqa: E731
    rotate_refusals(call, ("oq_st", "oq_sh", "ok_st", "ok_sh"),
                    ("q", "k", "w_q", "w_k", "positions", "frequencies", "out_q", "out_k"))
    # rows of outputs that overlap
    assert call(oq_sh=63) == 1 and call(oq_st=191) == 1 and call(ok_st=0) == 1


def test_rotated_norm_gradient_rejects_bad_arguments_on_the_host(mx):
    call = lambda **kw: mx.mx_norm_rotate_backward(*{**ROTATE_BACK, **kw}.values())  # noqa: E731
    rotate_refusals(call, (), ("d_q", "d_k", "q", "k", "w_q", "w_k", "positions", "frequencies",
                               "dx_q", "dx_k", "dw_q", "dw_k", "workspace"))
    assert call(dq_st=-1) == 1 and call(workspace_bytes=0) == 1
    assert call(workspace=FAKE + 8) == 2 and call(dw_q=FAKE + 2) == 2
    size = mx.mx_norm_rotate_backward_workspace
    assert size(4, 64) > 0 and size(0, 64) == 0 and size(-1, 64) == 0 and size(4, 514) == 0
    assert size(1 << 29, 64) == size(1 << 20, 64)   # blocks, not tokens


def test_routing_rejects_bad_arguments_on_the_host(mx):
    call = lambda **kw: mx.mx_route(*{**ROUTE, **kw}.values())  # noqa: E731
    back = lambda **kw: mx.mx_route_backward(*{**ROUTE_BACK, **kw}.values())  # noqa: E731
    for name in ("logits", "ids", "weights", "lse", "counts", "offsets", "order", "balance",
                 "workspace"):
        assert call(**{name: None}) == 1, name
    for name in ("logits", "ids", "weights", "lse", "counts", "d_logits"):
        assert back(**{name: None}) == 1, name
    for f in (call, back):
        assert f(tokens=-1) == 1 and f(experts=0) == 1 and f(top_k=0) == 1 and f(top_k=9) == 1
        assert f(experts=64, ld=64, top_k=33) == 1 and f(ld=7) == 1 and f(dtype=2) == 1
        assert f(experts=513, ld=513) == 3 and f(tokens=4194304) == 3
        assert f(logits=FAKE + 1) == 2 and f(ids=FAKE + 2) == 2 and f(dtype=1, logits=FAKE + 2) == 2
    assert call(workspace_bytes=0) == 1 and call(workspace=FAKE + 8) == 2
    assert call(order=FAKE + 2) == 2 and call(balance=FAKE + 2) == 2
    assert back(d_weights=FAKE + 2) == 2 and back(d_logits=FAKE + 1) == 2
    size = mx.mx_route_workspace
    assert size(1, 8) == 0 and size(100000, 8) > 0
    assert size(-1, 8) == 0 and size(100, 513) == 0 and size(100, 0) == 0


def test_loss_rejects_bad_arguments_on_the_host(mx):
    call = lambda **kw: mx.mx_linear_cross_entropy(*{**LOSS, **kw}.values())  # noqa: E731
    back = lambda **kw: mx.mx_linear_cross_entropy_backward(*{**LOSS_BACK, **kw}.values())  # noqa: E731
    for name in ("x", "w", "labels", "loss", "lse", "workspace"):
        assert call(**{name: None}) == 1, name
    for name in ("x", "w", "labels", "lse", "workspace"):
        assert back(**{name: None}) == 1, name
    assert back(dx=None, dw=None) == 1
    for f in (call, back):
        assert f(tokens=-1) == 1 and f(vocab=0) == 1 and f(hidden=0) == 1 and f(hidden=60) == 1
        assert f(ldx=56) == 1 and f(ldw=56) == 1 and f(label_bits=8) == 1
        assert f(tokens=(1 << 24) + 1) == 3 and f(vocab=(1 << 24) + 1) == 3
        assert f(workspace_bytes=16) == 1 and f(workspace=FAKE + 8) == 2
        assert f(x=FAKE + 8) == 2 and f(w=FAKE + 8) == 2 and f(ldx=68) == 2 and f(ldw=68) == 2
        assert f(labels=FAKE + 4) == 2 and f(lse=FAKE + 2) == 2
    assert back(dw_dtype=2) == 1 and back(dx=FAKE + 8) == 2 and back(d_loss=FAKE + 2) == 2
    size, size_back = mx.mx_linear_cross_entropy_workspace, mx.mx_linear_cross_entropy_backward_workspace
    for f in (size, size_back):
        assert f(4, 64, 100) > 0
        assert f(-1, 64, 100) == 0 and f(4, 60, 100) == 0 and f(4, 64, 0) == 0
    # a piece of the vocabulary and not all of it; several parts of dx at most
    assert size_back(16384, 64, 1 << 20) <= (1 << 29) + 76 * 16384 * 64 * 4


def test_tensor_api_refuses_host_tensors(mx):
    import torch
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    w, pos, f = torch.ones(64), torch.arange(4), torch.ones(8, dtype=torch.float64)
    z = torch.zeros(4, 8)
    h, v = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(9, 64, dtype=torch.bfloat16)
    r = mx.Routing(*(torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2),
                     torch.zeros(8, dtype=torch.int32), None, None, None, torch.zeros(4)))
    calls = (lambda: mx.norm_rotate(x, x, w, w, pos, f),
             lambda: mx.norm_rotate_backward(x, x, x, x, w, w, pos, f), lambda: mx.route(z, 2),
             lambda: mx.route_backward(None, None, z, r), lambda: mx.linear_cross_entropy(h, v, pos),
             lambda: mx.linear_cross_entropy_backward(None, None, h, v, pos, torch.zeros(4)))
    for call in calls:
        with pytest.raises(ValueError):
            call()
    for bad in (None, 3, [z], torch.zeros(4)):
        for call in (lambda: mx.route(bad, 2), lambda: mx.norm_rotate(bad, x, w, w, pos, f),
                     lambda: mx.linear_cross_entropy(bad, v, pos)):
            with pytest.raises(ValueError):
                call()
    with pytest.raises(ValueError):
        mx.linear_cross_entropy_backward(None, None, h, v, pos, torch.zeros(4), weight_dtype="fp16")


def test_frequencies(mx):
    import torch
    f = mx.rotary_frequencies(8, 100.0, device="cpu")
    assert f.dtype == torch.float64
    assert torch.allclose(f, torch.tensor([1, 100 ** -0.25, 0.1, 100 ** -0.75], dtype=torch.float64))
    assert torch.allclose(mx.rotary_frequencies(8, 100.0, factor=4.0, device="cpu"), f / 4)
    # within 200 positions the pairs turn 31.8, 10.1, 3.2 and 1.007 times
    g = mx.rotary_frequencies(8, 100.0, factor=4.0, trained_length=200, fast=10, slow=2, device="cpu")
    keep = [1, 1, (20 / (2 * math.pi) - 2) / 8, 0]
    want = [v * (c + (1 - c) / 4) for v, c in zip(f.tolist(), keep)]
    assert torch.allclose(g, torch.tensor(want, dtype=torch.float64))
    for bad in (dict(rotary=7), dict(rotary=0), dict(rotary=8, base=0.0), dict(rotary=8, factor=-1.0),
                dict(rotary=8, fast=1.0, slow=1.0)):
        with pytest.raises(ValueError):
            mx.rotary_frequencies(device="cpu", **bad)


def test_a_workspace_for_more_tokens_suffices_for_fewer(mx):
    """Sizes do not fall as tokens grow: around every count where a kernel, its blocks or
    its pieces change, and over counts of all magnitudes."""
    counts = sorted({t for b in (1, 16, 32, 64, 128, 256, 1024, 2048, 4096, 4864, 8192, 9728, 16384, 19456, 65536,
                                 131072, 262144, 1 << 20, (1 << 22) - 64) for t in range(b, b + 34)}
                    | {int(1.07 ** i) for i in range(1, 220)})
    for experts in (1, 5, 64, 65, 128, 129, 512):
        sizes = [mx.mx_route_workspace(t, experts) for t in counts]
        assert sizes == sorted(sizes) and sizes[-1] > 0, experts
    for hidden, vocab in ((8, 1), (64, 300), (1000, 1000), (1000, 18433), (2048, 32768), (4096, 131072),
                          (7168, 131072), (128, 1 << 22), (32768, 5000)):
        for size in (mx.mx_linear_cross_entropy_workspace, mx.mx_linear_cross_entropy_backward_workspace):
            sizes = [size(t, hidden, vocab) for t in counts]
            assert sizes == sorted(sizes) and sizes[0] > 0, (hidden, vocab)
    # and stay in proportion: dz of one piece and a few MB beside it
    assert mx.mx_linear_cross_entropy_backward_workspace(2048, 2048, 32768) <= 2 * 2048 * 32768 + (32 << 20)
    assert mx.mx_linear_cross_entropy_backward_workspace(1, 4096, 131072) <= 2 << 20


def test_limits_of_sizes(mx):
    """What the header states, each just above."""
    rotate = lambda **kw: mx.mx_norm_rotate(*{**ROTATE, **kw}.values())  # noqa: E731
    back = lambda **kw: mx.mx_norm_rotate_backward(*{**ROTATE_BACK, **kw}.values())  # noqa: E731
    for call in (rotate, back):
        assert call(q_heads=65537) == 3 and call(k_heads=65537) == 3 and call(tokens=(1 << 30) + 1) == 3
        assert call(tokens=1 << 29, q_heads=2, k_heads=2) == 3
        for huge in (1 << 29, 1 << 61, (1 << 63) - 1):
            assert call(q_st=huge) == 3 and call(k_sh=huge) == 3
    for name in ("oq_st", "oq_sh", "ok_st", "ok_sh"):
        for huge in (1 << 29, 1 << 61, (1 << 63) - 1):
            assert rotate(**{name: huge}) == 3, name
    for size in (mx.mx_linear_cross_entropy_workspace, mx.mx_linear_cross_entropy_backward_workspace):
        assert size(1 << 24, 8, 256) > 0 and size((1 << 24) + 1, 8, 256) == 0
        assert size(1, 8, 1 << 24) > 0 and size(1, 8, (1 << 24) + 1) == 0
        assert size(1, 1 << 20, 8) > 0 and size(1, (1 << 20) + 8, 8) == 0
        assert size(1 << 24, 8, 1 << 23) == 0 and size(1 << 24, 8, (1 << 23) - 256) > 0
    assert mx.mx_route_workspace(4194303, 512) > 0 and mx.mx_route_workspace(4194304, 512) == 0
