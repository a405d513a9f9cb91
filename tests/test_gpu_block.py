"""The block operators together, as a serving loop and a training step run
them: a mixture-of-experts block of the cases module against the oracle, and
a training step's norms around the grouped GEMMs."""
from types import SimpleNamespace

import numpy as np
import pytest
import torch

from mxcheck import ensure_built, to_f64
from oracle import block_oracle as B

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mx():
    ensure_built()
    import mxfp8_block_scaled_mx_gb300 as mx
    return mx


@pytest.mark.parametrize("tokens,fmt", [(1, "e4m3"), (5, "e2m1_packed"), (20, "e5m2")])
def test_serving_step(mx, tokens, fmt):
    from mxfp8_block_scaled_mx_gb300 import cases, workloads as W
    dev = torch.device("cuda")
    a = SimpleNamespace(k=256, inter=128, experts=6, top_k=2, fmt=fmt)
    step, p = cases.moe_block(a, dev)
    stream = W.synth_matrix((tokens, a.k), 2.0, seed=1, device=dev)
    attention = W.synth_matrix((tokens, a.k), 0.5, seed=2, device=dev)
    got_stream, got = step(stream, attention)
    assert mx.device_status() == 0
    # the same step by the oracle, from the values that each operator stored
    s1, x = mx.norm_residual(attention, stream, p["w_in"])
    y, ids, w = mx.moe_few_tokens(x, p["router"], p["gate"], p["up"], p["down"], a.top_k,
                                  return_routing=True)
    mats = []
    for n, rows, k in (("gate", a.inter, a.k), ("up", a.inter, a.k), ("down", a.k, a.inter)):
        t = p[n]
        size = t.scales.numel() // a.experts
        mats.append([B.expert_weight(t.codes[e].cpu().numpy(),
                                     t.scales[e * size:(e + 1) * size].cpu().numpy(), rows, k, fmt)
                     for e in range(a.experts)])
    ref, tol = B.moe_layer(to_f64(x), ids.cpu().numpy(), to_f64(w), *mats, 1e-4, 2.0 ** -8)
    assert (np.abs(to_f64(y) - ref) <= tol + 2.0 ** -8 * np.abs(ref) + 1e-30).all()
    ref, mag = B.norm_residual_stream(to_f64(y), to_f64(s1), to_f64(p["w_post"]),
                                      to_f64(p["scale"]), 1.0, 1e-6)
    assert (np.abs(to_f64(got_stream) - ref) <= 2.0 ** -16 * mag + 2.0 ** -8 * np.abs(ref)).all()
    ref = B.norm_rows(to_f64(got_stream), to_f64(p["w_next"]), 1e-6)
    assert (np.abs(to_f64(got) - ref) <= (2.0 ** -16 + 2.0 ** -8) * np.abs(ref)).all()
    # the step in a CUDA graph, as a serving loop replays it
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again = step(stream, attention)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(again[0], got_stream) and torch.equal(again[1], got)


def test_few_tokens_agree_with_the_grouped_path(mx):
    """The layer for a few tokens against the same layer by the training
    operators (rows sorted by expert, grouped quantization, grouped GEMMs),
    whose activations are rounded to MXFP8: 2^-4 of each value, so within
    2^-4 / sqrt(3) in the 2-norm for either product, 6e-2 together."""
    g = torch.Generator().manual_seed(9)
    tokens, h, inter, experts, k = 48, 512, 256, 4, 2
    x = torch.randn(tokens, h, generator=g).to(torch.bfloat16).cuda()
    router = (torch.randn(experts, h, generator=g) * 0.05).to(torch.bfloat16).cuda()
    ws = {n: (torch.randn(experts * r, c, generator=g) * 0.05).to(torch.bfloat16).cuda()
          for n, r, c in (("gate", inter, h), ("up", inter, h), ("down", h, inter))}
    q = {}
    for n, w in ws.items():
        t = mx.quantize(w, "e4m3", "row")
        q[n] = mx.MxTensor(t.codes.view(experts, -1, t.codes.shape[1]), t.scales, "e4m3")
    y, ids, w = mx.moe_few_tokens(x, router, q["gate"], q["up"], q["down"], k, return_routing=True)
    flat = ids.flatten().long()
    order = torch.argsort(flat, stable=True)
    counts = torch.bincount(flat, minlength=experts)
    off = torch.cat([torch.zeros(1, dtype=torch.long, device="cuda"), counts.cumsum(0)]).int()
    xs = x[order // k].contiguous()
    qx = mx.quantize_grouped(xs, off, "e4m3")
    a = mx.grouped_gemm(qx, off, q["gate"], "fp32")
    b = mx.grouped_gemm(qx, off, q["up"], "fp32")
    act = torch.nn.functional.silu(a) * b
    o = mx.grouped_gemm(mx.quantize_grouped(act, off, "e4m3"), off, q["down"], "fp32")
    ref = torch.zeros(tokens, h, device="cuda").index_add_(0, order // k,
                                                            o * w.flatten()[order][:, None])
    assert mx.device_status() == 0
    assert (y.float() - ref).norm() <= 6e-2 * ref.norm()


def test_training_step_of_a_residual_block(mx):
    """Norm, MX product, norm with gate and residual, forward and backward,
    against torch's gradients in float64 of the same computation on the
    quantized operands.  The products' bf16 outputs (2^-9 of the norm each
    way) and E5M2 gradients are shared, so what is left is FP32 rounding and
    one bf16 rounding per stored tensor: 1e-2 in the 2-norm."""
    g = torch.Generator().manual_seed(4)
    t, h = 64, 256
    x = torch.randn(t, h, generator=g).to(torch.bfloat16).cuda()
    w = (torch.randn(h, h, generator=g) * 0.06).to(torch.bfloat16).cuda()
    stream = torch.randn(t, h, generator=g).cuda()
    w_pre, w_post = (torch.randn(2, h, generator=g) * 0.1 + 1).cuda()
    gate = (torch.randn(h, generator=g) * 0.3).cuda()
    d_res, d_y = torch.randn(t, h, generator=g).cuda(), torch.randn(t, h, generator=g).to(torch.bfloat16).cuda()
    b = mx.gemm(mx.quantize(x, "e4m3", "row"), mx.quantize(w, "e4m3", "col"), "bf16")
    s, y = mx.norm_residual(b, stream, w_pre, w_post=w_post, gate=gate, alpha=0.5)
    d = mx.norm_residual_backward(d_res, d_y, b, s, w_pre, w_post=w_post, gate=gate, alpha=0.5)
    dx = mx.gemm(mx.quantize(d.block, "e5m2", "row"), mx.quantize(w, "e4m3", "row"), "fp32")
    assert dx.shape == (t, h) and dx.isfinite().all()
    p = {n: v.double().requires_grad_() for n, v in
         (("block", b), ("residual", stream), ("w_pre", w_pre), ("w_post", w_post), ("gate", gate))}

    def rms(v, u):
        return v * torch.rsqrt(v.square().mean(1, keepdim=True) + 1e-6) * u

    r = 0.5 * p["residual"] + p["gate"] * rms(p["block"], p["w_post"])
    out = rms(r, p["w_pre"])
    ((r * d_res.double()).sum() + (out * d_y.double()).sum()).backward()
    for n, v in p.items():
        mine = getattr(d, n).double()
        assert (mine - v.grad).norm() <= 1e-2 * v.grad.norm(), n
    assert mx.device_status() == 0
