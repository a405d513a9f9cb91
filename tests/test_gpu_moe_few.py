"""moe_few_tokens against the float64 oracle.

Tolerances.  Products: 1e-4 of their sum of magnitudes, as for every GEMM
of the library.  The weighted activation is rounded to 8 significant bits
(2^-8 of itself, and 2^-24 of its block's largest value where small values
lose bits); both are carried through the down product by the oracle.  y is
rounded to bf16, 2^-8 of itself.  Those bounds hold for any signs; as the
signs are random, the whole y is also held to 5e-3 in the 2-norm, twice the
2^-8 / sqrt(3) of one rounding.  Routing weights: the logits are FP32 sums of
`hidden` products (2^-19 of their magnitudes) through exp, so 2^-18 times the
magnitudes' sum, and 2^-20 for exp and division."""
import numpy as np
import pytest
import torch

from mxcheck import ensure_built, to_f64
from oracle import block_oracle as B
from oracle import mx_oracle as O

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def mx():
    ensure_built()
    import mxfp8_block_scaled_mx_gb300 as mx
    return mx


def weights(rng, experts, rows, k, fmt, spread=1):
    """MX weights from quantized normals, each block moved by a power of two;
    padding scale bytes hold NaN, which must not matter.  Returns the device
    operand and the experts' float64 matrices."""
    from mxfp8_block_scaled_mx_gb300 import MxTensor
    name = fmt.replace("_packed", "")
    codes, scales, values = [], [], []
    for _ in range(experts):
        q = O.quantize(rng.normal(0, 0.05, (rows, k)), name, "row")
        move = rng.integers(-spread, spread + 1, q.scales.shape)
        s = (q.scales.astype(np.int64) + move).astype(np.uint8)
        c = O.pack_dense(q.codes, name) if fmt.endswith("packed") else q.codes
        buf = O.swizzle_scales(s)
        used = np.zeros(buf.shape, dtype=bool)
        r, j = np.meshgrid(np.arange(rows), np.arange(s.shape[1]), indexing="ij")
        used[O.swizzle_offset(r, j, s.shape[1])] = True
        buf[~used] = 0xFF
        codes.append(c)
        scales.append(buf)
        values.append(B.expert_weight(c, buf, rows, k, fmt))
    t = MxTensor(torch.from_numpy(np.stack(codes)).cuda(),
                 torch.from_numpy(np.concatenate(scales)).cuda(), fmt)
    return t, values


def layer(seed, tokens, hidden, inter, experts, fmt="e4m3", fmt_d=None, router=BF16, spread=1):
    rng = np.random.default_rng(seed)
    d = dict(x=torch.from_numpy(rng.normal(size=(tokens, hidden))).to(BF16).cuda(),
             router=torch.from_numpy(rng.normal(0, 0.05, (experts, hidden))).to(router).cuda())
    d["gate"], g = weights(rng, experts, inter, hidden, fmt, spread)
    d["up"], u = weights(rng, experts, inter, hidden, fmt, spread)
    d["down"], n = weights(rng, experts, hidden, inter, fmt_d or fmt, spread)
    return d, (g, u, n)


def check(mx, d, mats, top_k, renormalize=True, **kw):
    y, ids, w = mx.moe_few_tokens(d["x"], d["router"], d["gate"], d["up"], d["down"], top_k,
                                  renormalize=renormalize, return_routing=True, **kw)
    assert mx.device_status() == 0
    x, r = to_f64(d["x"]), to_f64(d["router"])
    z = x @ r.T
    rid, rw = B.route(z, top_k, renormalize)
    assert np.array_equal(ids.cpu().numpy(), rid)
    off = 2.0 ** -18 * (np.abs(x) @ np.abs(r).T).max(1, keepdims=True) + 2.0 ** -20
    assert (np.abs(to_f64(w) - rw) <= 4 * off * rw).all()
    ref, tol = B.moe_layer(x, rid, to_f64(w), *mats, 1e-4, 2.0 ** -8)
    got = to_f64(y)
    assert np.isfinite(got).all()
    err = np.abs(got - ref)
    tol = tol + 2.0 ** -8 * np.abs(ref) + 1e-30
    assert (err <= tol).all(), f"{float((err / tol).max()):.3g} x the tolerance"
    norm = np.linalg.norm(ref)
    assert np.linalg.norm(err) <= 5e-3 * norm
    return y, ids, w


@pytest.mark.parametrize("tokens", [1, 2, 7, 8, 9, 16, 17, 33, 48, 64])
def test_token_counts(mx, tokens):
    d, mats = layer(tokens, tokens, 256, 128, 8)
    check(mx, d, mats, 2)


@pytest.mark.parametrize("hidden,inter", [(16, 16), (32, 48), (144, 16), (16, 272), (128, 128),
                                          (400, 304), (1040, 144), (256, 1168)])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_odd_sizes(mx, hidden, inter, fmt):
    """Partial final blocks along either contraction, partial row tiles."""
    d, mats = layer(hidden + inter, 5, hidden, inter, 4, fmt)
    check(mx, d, mats, 2)


@pytest.mark.parametrize("hidden,inter", [(128, 128), (384, 256), (256, 640)])
def test_packed_4_bit_weights(mx, hidden, inter):
    d, mats = layer(hidden, 6, hidden, inter, 5, "e2m1_packed")
    check(mx, d, mats, 3)


@pytest.mark.parametrize("fmt,fmt_d", [("e2m1_packed", "e4m3"), ("e4m3", "e2m1_packed"),
                                       ("e5m2", "e4m3")])
def test_formats_of_their_own(mx, fmt, fmt_d):
    d, mats = layer(3, 4, 256, 128, 6, fmt, fmt_d)
    check(mx, d, mats, 2)


@pytest.mark.parametrize("experts,top_k", [(1, 1), (2, 2), (3, 1), (7, 5), (33, 32), (130, 8),
                                           (512, 6)])
@pytest.mark.parametrize("renormalize", [False, True])
def test_experts_and_choices(mx, experts, top_k, renormalize):
    d, mats = layer(experts, 3, 64, 32, experts, router=FP32)
    check(mx, d, mats, top_k, renormalize)


def test_many_partial_tiles(mx):
    """Long contractions over few tiles: many parts of one sum."""
    d, mats = layer(21, 3, 4096, 64, 2)
    check(mx, d, mats, 1)
    d, mats = layer(22, 2, 64, 4096, 2)
    check(mx, d, mats, 2)


def test_block_scales_over_a_wide_range(mx):
    d, mats = layer(11, 4, 256, 256, 3, spread=12)
    check(mx, d, mats, 2)


def test_small_and_large_tokens(mx):
    """x over many binades, within a block and between tokens."""
    d, mats = layer(12, 6, 256, 128, 3)
    lift = torch.tensor([1e-6, 1e-3, 1.0, 4.0, 1.0, 0.0], device="cuda")[:, None]
    tilt = 2.0 ** -torch.arange(256, device="cuda").remainder(13)
    x = d["x"].float() * lift
    x[4] *= tilt
    d["x"] = x.to(BF16)
    d["router"] = (d["router"].float() / 4).to(BF16)
    y, ids, w = mx.moe_few_tokens(d["x"], d["router"], d["gate"], d["up"], d["down"], 2,
                                  return_routing=True)
    assert (y[5] == 0).all()                            # an empty token: silu(0) * 0
    assert ids[5].tolist() == [0, 1] and (w[5] == 0.5).all()
    d["x"] = d["x"][:5].contiguous()
    check(mx, d, mats, 2)


def test_equal_logits_go_to_the_lowest_expert(mx):
    d, mats = layer(13, 4, 128, 64, 12)
    d["router"][7] = d["router"][2]
    d["router"][9] = d["router"][2]
    d["router"][2:10:5] = d["router"][2]
    x = d["x"].float()
    x[0] = d["router"][2].float() * 20                  # experts 2, 7 and 9 tie in front
    d["x"] = x.to(BF16)
    y, ids, w = check(mx, d, mats, 3)
    assert ids[0].tolist() == [2, 7, 9]


def test_a_bad_token_touches_no_other(mx):
    d, mats = layer(14, 9, 256, 128, 6)
    clean = mx.moe_few_tokens(d["x"], d["router"], d["gate"], d["up"], d["down"], 2)
    x = d["x"].clone()
    x[3, 40] = float("nan")
    x[6, 0] = float("inf")
    y, ids, w = mx.moe_few_tokens(x, d["router"], d["gate"], d["up"], d["down"], 2,
                                  return_routing=True)
    keep = [0, 1, 2, 4, 5, 7, 8]
    # (which experts are read may change, and with it the order of the sums)
    assert (y[keep].double() - clean[keep].double()).norm() <= 5e-3 * clean[keep].double().norm()
    assert y[3].isnan().all() and y[6].isnan().all()
    for row in ids.tolist():                            # still two experts of the six
        assert len(set(row)) == 2 and all(0 <= e < 6 for e in row)
    assert mx.device_status() == 0


def test_rows_apart_repeatability_and_workspace(mx):
    d, mats = layer(15, 10, 384, 160, 9)
    ref = check(mx, d, mats, 3)
    wide = torch.full((10, 400), float("nan"), dtype=BF16, device="cuda")
    wide[:, :384] = d["x"]
    out = torch.full((10, 392), 7.0, dtype=BF16, device="cuda")
    need = mx.mx_moe_few_tokens_workspace(10, 384, 160, 9, 3)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    for _ in range(3):                                  # garbage, then its own leavings
        got = mx.moe_few_tokens(wide[:, :384], d["router"], d["gate"], d["up"], d["down"], 3,
                                out=out[:, :384], workspace=ws, return_routing=True)
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
        assert torch.equal(got[2], ref[2])
        assert (out[:, 384:] == 7.0).all()
    assert mx.moe_few_tokens(d["x"][:0], d["router"], d["gate"], d["up"], d["down"],
                             3).shape == (0, 384)
    assert mx.device_status() == 0


def test_on_other_streams_and_in_a_graph(mx):
    d, mats = layer(16, 12, 512, 256, 8)
    e, mats_e = layer(17, 3, 512, 256, 8)
    ref, ref_e = check(mx, d, mats, 2)[0], check(mx, e, mats_e, 2)[0]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    outs = []
    for _ in range(8):
        for s, q in zip(streams, (d, e)):
            outs.append(mx.moe_few_tokens(q["x"], q["router"], q["gate"], q["up"], q["down"], 2,
                                          stream=s))
    torch.cuda.synchronize()
    for i, y in enumerate(outs):
        assert torch.equal(y, ref_e if i % 2 else ref)
    graph = torch.cuda.CUDAGraph()
    x = d["x"].clone()
    with torch.cuda.graph(graph):
        y = mx.moe_few_tokens(x, d["router"], d["gate"], d["up"], d["down"], 2)
    for shift in (0, 3):
        x.copy_(d["x"].roll(shift, 0))
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        want = mx.moe_few_tokens(x, d["router"], d["gate"], d["up"], d["down"], 2)
        assert torch.equal(y, want)
    assert mx.device_status() == 0


def test_refusals(mx):
    d, _ = layer(18, 4, 256, 128, 4)
    call = lambda top_k=2, **kw: mx.moe_few_tokens(  # noqa: E731
        top_k=top_k, **{**{k: d[k] for k in ("x", "router", "gate", "up", "down")}, **kw})
    call()
    g = d["gate"]
    for bad in (dict(x=d["x"].float()), dict(x=d["x"].cpu()), dict(x=d["x"][:, :128]),
                dict(router=d["router"].half()), dict(router=d["router"][:, :128]),
                dict(router=d["router"][:3]), dict(gate=d["down"]),
                dict(gate=mx.MxTensor(g.codes, g.scales, "e5m2")),
                dict(up=mx.MxTensor(g.codes[:3], g.scales, "e4m3")),
                dict(up=mx.MxTensor(g.codes, g.scales[:-1], "e4m3")),
                dict(out=torch.empty(4, 256, device="cuda")),
                dict(workspace=torch.empty(64, dtype=torch.uint8, device="cuda")),
                dict(top_k=0), dict(top_k=5)):
        with pytest.raises(ValueError):
            call(**bad)
    with pytest.raises(mx.MxError) as e:
        call(x=torch.zeros(65, 256, dtype=BF16, device="cuda"))
    assert e.value.status == 3
    narrow = {k: mx.MxTensor(d[k].codes, d[k].scales, "e2m1") for k in ("gate", "up")}
    with pytest.raises(mx.MxError) as e:                # the 4-bit container layout
        call(**narrow)
    assert e.value.status == 3
    with pytest.raises(mx.MxError) as e:                # rows of x off 16 bytes
        call(x=torch.zeros(4, 257, dtype=BF16, device="cuda")[:, 1:])
    assert e.value.status == 2
    assert mx.device_status() == 0


@pytest.mark.parametrize("tokens", [1, 4, 15, 16, 17, 40])
@pytest.mark.parametrize("hidden,inter,experts,top_k", [(128, 128, 3, 2), (640, 384, 5, 2),
                                                        (2048, 128, 4, 1), (256, 2048, 6, 3)])
def test_packed_4_bit_weights_by_token_count(mx, tokens, hidden, inter, experts, top_k):
    """Both roles of the operands: odd and even numbers of 128-channel tiles,
    sums in one block and in many."""
    d, mats = layer(tokens + hidden, tokens, hidden, inter, experts, "e2m1_packed")
    y, ids, w = check(mx, d, mats, top_k)
    again = mx.moe_few_tokens(d["x"], d["router"], d["gate"], d["up"], d["down"], top_k)
    assert torch.equal(again, y)
