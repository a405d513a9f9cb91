"""The block operators' C entries with a caller's buffers, calls on given
streams (the memory that a call takes for itself), tokens over a wide range,
and calls that autograd records.  Tolerances are those of test_gpu_norm and
test_gpu_moe_few."""
from types import SimpleNamespace

import numpy as np
import pytest
import torch

from mxcheck import ensure_built, to_f64
from oracle import block_oracle as B
from test_gpu_norm import BF16, EPS, FP32, TYPES, close, f64, inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mx():
    ensure_built()
    import mxfp8_block_scaled_mx_gb300 as mx
    return mx


def slices(off, sizes):
    """FP32 slices of one flat buffer of NaNs, each `off` floats past a
    16-byte boundary and four apart at least; the buffer, and where nothing
    may be written."""
    starts, at = [], 0
    for n in sizes:
        starts.append(at + off)
        at += (n + off + 7) // 4 * 4
    flat = torch.full((at + 4,), float("nan"), device="cuda")
    free = torch.ones(at + 4, dtype=torch.bool, device="cuda")
    for s, n in zip(starts, sizes):
        free[s:s + n] = False
    return flat, free, [flat[s:s + n] for s, n in zip(starts, sizes)]


def c_backward(mx, d, alpha, d_block, d_residual, d_post, d_pre, d_gate):
    """mx_norm_residual_backward with the caller's buffers; its status."""
    rows, cols = d["block"].shape
    code = {BF16: 0, FP32: 1}
    gates = 0 if d["gate"] is None else d["gate"].numel() // cols
    need = mx.mx_norm_residual_backward_workspace(rows, cols, gates)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    ptr = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    ld = lambda t: cols if t is None or rows == 1 else t.stride(0)  # noqa: E731
    return mx.mx_norm_residual_backward(
        rows, cols, ptr(d["d_residual"]), ld(d["d_residual"]), ptr(d["d_y"]), ld(d["d_y"]),
        ptr(d["block"]), ld(d["block"]), code[d["block"].dtype], ptr(d["residual"]),
        ld(d["residual"]), code[d["residual"].dtype], ptr(d["w_post"]), ptr(d["w_pre"]),
        ptr(d["gate"]), gates, code[d["w_pre"].dtype], alpha, EPS, ptr(d_block), ld(d_block),
        ptr(d_residual), ld(d_residual), ptr(d_post), ptr(d_pre), ptr(d_gate), ws.data_ptr(), need,
        torch.cuda.current_stream().cuda_stream)


# gates of whole blocks' rows, of several blocks' rows, of one row; rows by one
# run and by two, by a cluster, element by element, by phase
@pytest.mark.parametrize("rows,cols,gates", [(12, 256, 4), (5, 1024, 1), (7, 4096, 7), (40, 2560, 2),
                                             (700, 1104, 7), (650, 512, 325), (9, 8200, 3),
                                             (6, 16384, 6), (400, 5120, 1), (9744, 1032, 2)])
@pytest.mark.parametrize("c,s,w", TYPES)
def test_gradients_of_weights_off_16_bytes(mx, rows, cols, gates, c, s, w):
    """d_gate, d_w_pre and d_w_post as slices of a flat FP32 buffer, one, two
    and three floats off a 16-byte boundary, everything else aligned."""
    d = inputs(rows, cols, c, s, w, True, gates, seed=rows + cols)
    ref = B.norm_residual_backward(f64(d["d_residual"]), f64(d["d_y"]), f64(d["block"]),
                                   f64(d["residual"]), f64(d["w_pre"]), f64(d["w_post"]),
                                   f64(d["gate"]), 0.875, EPS)
    for off in (1, 2, 3):
        flat, free, (post, pre, gate) = slices(off, (cols, cols, gates * cols))
        assert all(t.data_ptr() % 16 == 4 * off for t in (post, pre, gate))
        d_block, d_residual = torch.empty_like(d["block"]), torch.empty_like(d["residual"])
        assert c_backward(mx, d, 0.875, d_block, d_residual, post, pre, gate) == 0
        assert mx.device_status() == 0
        close(d_block, ref["block"], ref["mag"]["block"])
        close(d_residual, ref["residual"], ref["mag"]["residual"])
        for name, t in (("w_post", post), ("w_pre", pre), ("gate", gate.view(d["gate"].shape))):
            close(t, ref[name], ref["mag"][name], rows)
        assert flat[free].isnan().all()                 # nothing between them was written


# ------------------------------------------------------------------ calls on a given stream

SLEEP = 40_000_000                                      # cycles: about 20 ms of one thread


def segment_stream(t):
    """Stream that owns the allocator's segment of a tensor."""
    for s in torch.cuda.memory_snapshot():
        if s["address"] <= t.data_ptr() < s["address"] + s["total_size"]:
            return s["stream"]
    raise AssertionError("no segment holds the tensor")


def moe_weights(mx, hidden, inter, experts):
    g = torch.Generator(device="cuda").manual_seed(3)

    def weight(rows, k):
        w = (torch.randn(experts * rows, k, generator=g, device="cuda") * 0.05).to(BF16)
        q = mx.quantize(w, "e4m3", "row")               # rows % 128 == 0: tiles by expert
        return mx.MxTensor(q.codes.view(experts, rows, k), q.scales, "e4m3")

    router = (torch.randn(experts, hidden, generator=g, device="cuda") * 0.05).to(BF16)
    return router, weight(inter, hidden), weight(inter, hidden), weight(hidden, inter)


def calls(mx):
    """Name -> a call on a stream that returns a list of its outputs."""
    rows, cols = 512, 2048
    d = inputs(rows, cols, BF16, BF16, BF16, True, 1, seed=2)
    args, kw = (d["block"], d["residual"], d["w_pre"]), dict(w_post=d["w_post"], gate=d["gate"])
    layer = moe_weights(mx, 1024, 256, 8)
    xs = [torch.randn(n, 1024, generator=torch.Generator().manual_seed(n)).to(BF16).cuda()
          for n in (40, 33)]

    def norm(stream=None, which=0):
        a = (args[0].flip(0), args[1], args[2]) if which else args
        torch.cuda.synchronize()
        return lambda: list(mx.norm_residual(*a, **kw, stream=stream))

    def back(stream=None, which=0):
        dy = d["d_y"].flip(0) if which else d["d_y"]
        torch.cuda.synchronize()
        return lambda: list(vars(mx.norm_residual_backward(d["d_residual"], dy, *args, **kw,
                                                           stream=stream)).values())

    def moe(stream=None, which=0):
        return lambda: list(mx.moe_few_tokens(xs[which], *layer, 2, return_routing=True,
                                              stream=stream))

    return dict(norm=norm, back=back, moe=moe)


@pytest.mark.parametrize("name", ["norm", "back", "moe"])
def test_outputs_come_from_the_given_streams_memory(mx, name):
    s = torch.cuda.Stream()
    make = calls(mx)[name]
    for t in make(s)():
        assert segment_stream(t) == s.cuda_stream
    for t in make()():
        assert segment_stream(t) == torch.cuda.current_stream().cuda_stream
    with torch.cuda.stream(s):                          # the default stream by its handle
        for t in make(torch.cuda.default_stream())():
            assert segment_stream(t) == torch.cuda.default_stream().cuda_stream
    torch.cuda.synchronize()
    assert mx.device_status() == 0


@pytest.mark.parametrize("name", ["norm", "back", "moe"])
def test_a_call_beside_one_that_is_still_queued(mx, name):
    """A call on the current stream, queued behind other work, and at once
    one of other inputs on another stream: neither takes the other's memory."""
    make = calls(mx)[name]
    ref = [make(which=i)() for i in (0, 1)]
    s = torch.cuda.Stream()
    for first, second in ((None, s), (s, None)):
        one, two = make(first, 0), make(second, 1)
        torch.cuda.synchronize()
        with torch.cuda.stream(first or torch.cuda.current_stream()):
            torch.cuda._sleep(SLEEP)
        got = [one(), two()]
        torch.cuda.synchronize()
        for a, b in zip(ref, got):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert mx.device_status() == 0


@pytest.mark.parametrize("name", ["norm", "back", "moe"])
def test_freed_memory_with_uses_still_queued(mx, name):
    """Tensors of the outputs' sizes, freed while copies of them are queued
    behind other work, then a call on another stream: the copies hold."""
    make = calls(mx)[name]
    s = torch.cuda.Stream()
    call = make(s)
    old = [torch.full_like(t, 7) for t in make()() for _ in range(4)]
    torch.cuda.synchronize()
    torch.cuda._sleep(SLEEP)
    kept = [t.clone() for t in old]
    del old
    outs = [call() for _ in range(3)]
    torch.cuda.synchronize()
    assert all(bool((t == 7).all()) for t in kept)
    assert all(torch.equal(a, b) for a, b in zip(outs[0], outs[-1]))
    assert mx.device_status() == 0


def test_routing_that_is_not_returned(mx):
    """The layer queued behind other work of its stream; tensors that the
    current stream takes meanwhile keep their values."""
    router, gate, up, down = moe_weights(mx, 1024, 256, 8)
    s = torch.cuda.Stream()
    x = torch.randn(64, 1024, device="cuda").to(BF16)
    ref = mx.moe_few_tokens(x, router, gate, up, down, 8)
    torch.cuda.synchronize()
    for _ in range(5):
        with torch.cuda.stream(s):
            torch.cuda._sleep(SLEEP)
        y = mx.moe_few_tokens(x, router, gate, up, down, 8, stream=s)
        mine = [torch.full((64, 8), i, dtype=torch.int32, device="cuda") for i in range(64)]
        mine_f = [torch.full((64, 1024), float(i), dtype=BF16, device="cuda") for i in range(8)]
        torch.cuda.synchronize()
        assert all(bool((t == i).all()) for i, t in enumerate(mine))
        assert all(bool((t == i).all()) for i, t in enumerate(mine_f))
        assert torch.equal(y, ref)
    assert mx.device_status() == 0


def test_outputs_that_the_caller_frees(mx):
    """Outputs of a call on another stream, read on the current one behind
    other work and freed there: later calls on that stream leave them alone."""
    make = calls(mx)
    s = torch.cuda.Stream()
    for name in ("norm", "back", "moe"):
        ref, call = make[name]()(), make[name](s)
        torch.cuda.synchronize()
        outs = call()
        torch.cuda.current_stream().wait_stream(s)
        torch.cuda._sleep(SLEEP)
        kept = [t.clone() for t in outs]
        del outs
        other = make[name](s, 1) if name == "moe" else None  # (others synchronize when made)
        for _ in range(4):
            (other or call)()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(ref, kept))
    assert mx.device_status() == 0


def test_a_given_stream_in_a_graph(mx):
    """Capture that forks to a second stream and joins it."""
    make = calls(mx)
    s = torch.cuda.Stream()
    for name in ("norm", "back", "moe"):
        ref, call = make[name]()(), make[name](s)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            s.wait_stream(torch.cuda.current_stream())
            got = call()
            torch.cuda.current_stream().wait_stream(s)
        for t in got:
            t.zero_()
        for _ in range(2):
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(ref, got))
    assert mx.device_status() == 0


# ------------------------------------------------------------------ tokens over a wide range

@pytest.mark.parametrize("tokens", [1, 5, 40])
@pytest.mark.parametrize("fmt", ["e4m3", "e2m1_packed"])
def test_tokens_whose_blocks_span_a_wide_range(mx, tokens, fmt):
    """Blocks of 32 channels with one of 1 and the others down to 2^-24 of
    it, beside weights of zero at the large channels.  Against the layer of
    what two E4M3 terms hold of x, the tolerances of test_gpu_moe_few, with
    2^-22 of its block's largest for the activation; against x itself also
    2^-22 of each block's largest for x."""
    from test_gpu_moe_few import layer
    d, _ = layer(tokens, tokens, 256, 128, 3, fmt)
    rng = np.random.default_rng(tokens)
    x = rng.normal(size=(tokens, 256)) * np.exp2(-rng.integers(8, 25, (tokens, 256)))
    x[:, ::32] = 1.0
    d["x"] = torch.from_numpy(x).to(BF16).cuda()
    d["router"][:, ::32] = 0
    mats = []
    for n, rows, k in (("gate", 128, 256), ("up", 128, 256), ("down", 256, 128)):
        codes = d[n].codes.clone()
        if n != "down" and fmt == "e4m3":
            codes[:, :, ::32] = 0
        elif n != "down":
            codes[:, :, ::16] &= 0xF0                   # the even element of a byte: low bits
        scales = d[n].scales.view(3, -1)
        mats.append([B.expert_weight(codes[e].cpu().numpy(), scales[e].cpu().numpy(), rows, k, fmt)
                     for e in range(3)])
        d[n] = mx.MxTensor(codes, d[n].scales, fmt)
    assert all((m[:, ::32] == 0).all() for m in mats[0] + mats[1])
    y, ids, w = mx.moe_few_tokens(d["x"], d["router"], d["gate"], d["up"], d["down"], 2,
                                  return_routing=True)
    assert mx.device_status() == 0
    x, got, ids, w = to_f64(d["x"]), to_f64(y), ids.cpu().numpy(), to_f64(w)
    held = np.stack([B.two_terms(v) for v in x])
    assert (held != x).any()
    for tokens_in, x_floor in ((held, 0.0), (x, 2.0 ** -22)):
        ref, tol = B.moe_layer(tokens_in, ids, w, *mats, 1e-4, 2.0 ** -8, x_floor, 2.0 ** -22)
        assert (np.abs(got - ref) <= tol + 2.0 ** -8 * np.abs(ref) + 1e-30).all()


# ------------------------------------------------------------------ softmax of a NaN

@pytest.mark.parametrize("experts", [6, 200])
@pytest.mark.parametrize("renormalize", [False, True])
def test_a_nan_logit_makes_the_softmax_nan(mx, experts, renormalize):
    """softmax of logits with a NaN among them is NaN, so are the winners'
    shares of it and y; the winners are still the largest numbers."""
    from test_gpu_moe_few import layer
    d, _ = layer(8, 5, 128, 64, experts, router=FP32)
    kw = dict(renormalize=renormalize, return_routing=True)
    args = [d[n] for n in ("gate", "up", "down")]
    y, ids, w = mx.moe_few_tokens(d["x"], d["router"], *args, 2, **kw)
    bad = d["router"].clone()
    last = next(e for e in range(experts - 1, -1, -1) if not (ids == e).any())
    bad[last, 3] = float("nan")                         # an expert that nobody chose
    y2, ids2, w2 = mx.moe_few_tokens(d["x"], bad, *args, 2, **kw)
    assert torch.equal(ids2, ids)
    assert w2.isnan().all() and y2.isnan().all()
    assert w.isfinite().all() and y.isfinite().all()
    x = d["x"].clone()
    x[1, 5], x[4, 0] = float("-inf"), float("inf")
    y3, ids3, w3 = mx.moe_few_tokens(x, d["router"], *args, 2, **kw)
    assert w3[[1, 4]].isnan().all() and y3[[1, 4]].isnan().all()
    assert torch.equal(ids3[[0, 2, 3]], ids[[0, 2, 3]]) and torch.equal(w3[[0, 2, 3]], w[[0, 2, 3]])
    assert mx.device_status() == 0


# ------------------------------------------------------------------ autograd

@pytest.mark.parametrize("rows,cols,gates,post", [(64, 256, 1, True), (40, 1111, 0, False),
                                                  (12, 4096, 4, True)])
@pytest.mark.parametrize("c,s,w", TYPES)
def test_recorded_gradients_are_those_of_the_backward_entry(mx, rows, cols, gates, post, c, s, w):
    d = inputs(rows, cols, c, s, w, post, gates, seed=cols)
    names = ("block", "residual", "w_pre", "w_post", "gate")
    plain = mx.norm_residual(*(d[n] for n in names), alpha=0.5)
    want = mx.norm_residual_backward(d["d_residual"], d["d_y"], d["block"], plain[0], d["w_pre"],
                                     w_post=d["w_post"], gate=d["gate"], alpha=0.5)
    p = {n: None if d[n] is None else d[n].clone().requires_grad_() for n in names}
    got = mx.norm_residual(*p.values(), alpha=0.5)
    assert all(torch.equal(a, b) for a, b in zip(got, plain))
    torch.autograd.backward(got, (d["d_residual"], d["d_y"]))
    for n, t in p.items():
        if t is not None:
            assert t.grad.dtype == t.dtype and torch.equal(t.grad, getattr(want, n).to(t.dtype))
    # gradients that are expanded, or absent for one output
    for which in (0, 1):
        ones = torch.ones_like(plain[which])
        want = mx.norm_residual_backward(ones if which == 0 else None,
                                         torch.zeros_like(d["d_y"]) if which == 0 else ones,
                                         d["block"], plain[0], d["w_pre"], w_post=d["w_post"],
                                         gate=d["gate"], alpha=0.5)
        q = {n: None if d[n] is None else d[n].clone().requires_grad_() for n in names}
        mx.norm_residual(*q.values(), alpha=0.5)[which].sum().backward()
        for n, t in q.items():
            if t is not None:
                assert torch.equal(t.grad, getattr(want, n).to(t.dtype))
    assert mx.device_status() == 0


def test_recorded_calls_on_a_stream_and_into_given_outputs(mx):
    d = inputs(48, 512, BF16, BF16, BF16, True, 1)
    w = d["w_pre"].clone().requires_grad_()
    ref = mx.norm_residual(d["block"], d["residual"], d["w_pre"], d["w_post"], d["gate"])
    s = torch.cuda.Stream()
    wide = torch.full((48, 520), 7.0, dtype=BF16, device="cuda")
    handle = SimpleNamespace(cuda_stream=s.cuda_stream)  # (another library's stream)
    for stream in (None, s, s.cuda_stream, handle, 0):
        mine = d["residual"].clone()
        torch.cuda.synchronize()
        res, y = mx.norm_residual(d["block"], mine, w, d["w_post"], d["gate"], out_residual=mine,
                                  out=wide[:, :512], stream=stream)
        torch.cuda.synchronize()
        assert res is mine and torch.equal(res, ref[0]) and torch.equal(y, ref[1])
        assert (wide[:, 512:] == 7.0).all()
        w.grad = None
        y.float().sum().backward()
        want = mx.norm_residual_backward(None, torch.ones_like(y), d["block"], ref[0], d["w_pre"],
                                         d["w_post"], d["gate"])
        assert torch.equal(w.grad, want.w_pre.to(BF16))
        wide = wide.detach()


def test_buffers_written_are_known_to_autograd(mx):
    """A given output that autograd saved for another operator: its backward
    pass says so."""
    d = inputs(8, 128, BF16, BF16, BF16, True, 0)
    layer = moe_weights(mx, 128, 128, 4)
    a = torch.ones(8, 128, dtype=BF16, device="cuda", requires_grad=True)
    for write in (lambda t: mx.norm_residual(d["block"], d["residual"], d["w_pre"], out=t),
                  lambda t: mx.norm_residual(d["block"], d["residual"], d["w_pre"], out_residual=t),
                  lambda t: mx.moe_few_tokens(d["block"], *layer, 2, out=t)):
        buffer = torch.ones(8, 128, dtype=BF16, device="cuda")
        loss = (a * buffer).sum()
        write(buffer)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()


def test_the_layer_records_that_it_has_no_gradient(mx):
    router, *mats = moe_weights(mx, 128, 128, 4)
    x = torch.randn(5, 128, device="cuda").to(BF16)
    ref = mx.moe_few_tokens(x, router, *mats, 2, return_routing=True)
    got = mx.moe_few_tokens(x.requires_grad_(), router, *mats, 2, return_routing=True)
    assert all(torch.equal(a, b) for a, b in zip(ref, got))
    with pytest.raises(RuntimeError, match="no gradient"):
        got[0].float().sum().backward()
    out = torch.empty_like(ref[0])
    assert torch.equal(mx.moe_few_tokens(x, router, *mats, 2, out=out), ref[0]) and out.requires_grad
    assert mx.device_status() == 0


# ------------------------------------------------------------------ promises of the interface

@pytest.mark.parametrize("rows,cols,gates", [(300, 1024, 3), (40, 4096, 0), (160, 9216, 1),
                                             (700, 1111, 7), (60, 5001, 0), (9800, 1111, 1)])
@pytest.mark.parametrize("c,s,w", TYPES)
def test_gradient_of_the_residual_in_place(mx, rows, cols, gates, c, s, w):
    """d_residual may be d_res itself: the same bits as apart, whichever form
    reads the rows (a ring, a cluster, in place, by phase)."""
    d = inputs(rows, cols, c, s, w, True, gates, seed=rows)
    ref = mx.norm_residual_backward(d["d_residual"], d["d_y"], d["block"], d["residual"], d["w_pre"],
                                    d["w_post"], d["gate"], 0.5, EPS)
    post, pre = torch.empty(2, cols, device="cuda")
    gate = None if d["gate"] is None else torch.empty(d["gate"].shape, device="cuda")
    if cols % 4:                                        # slices of one tensor may be off 16 bytes
        post, pre = post.clone(), pre.clone()
    d_block = torch.empty_like(d["block"])
    assert c_backward(mx, d, 0.5, d_block, d["d_residual"], post, pre, gate) == 0
    assert mx.device_status() == 0
    assert torch.equal(d_block, ref.block) and torch.equal(d["d_residual"], ref.residual)
    assert torch.equal(pre, ref.w_pre) and torch.equal(post, ref.w_post)
    assert gate is None or torch.equal(gate, ref.gate)


@pytest.mark.parametrize("cols,ld", [(2048, 1 << 30), (1111, (1 << 30) + 8), (9000, (1 << 30) + 8)])
def test_rows_far_apart(mx, cols, ld):
    """Three rows over more than 2^31 elements of every array: the same bits
    as rows side by side."""
    d = inputs(3, cols, BF16, BF16, BF16, True, 1, seed=cols)
    far = {}
    for n in ("block", "residual", "d_residual", "d_y", "out", "out_residual"):
        far[n] = torch.empty(2 * ld + cols, dtype=BF16, device="cuda").as_strided((3, cols), (ld, 1))
        if n in d:
            far[n].copy_(d[n])
    w = (d["w_pre"], d["w_post"], d["gate"])
    ref = mx.norm_residual(d["block"], d["residual"], *w)
    mx.norm_residual(far["block"], far["residual"], *w, out_residual=far["out_residual"], out=far["out"])
    assert torch.equal(far["out_residual"], ref[0]) and torch.equal(far["out"], ref[1])
    near = mx.norm_residual_backward(d["d_residual"], d["d_y"], d["block"], d["residual"], *w)
    post, pre = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
    gate = torch.empty(cols, device="cuda")
    assert c_backward(mx, {**d, **{n: far[n] for n in d if n in far}}, 1.0, far["out"],
                      far["out_residual"], post, pre, gate) == 0
    assert torch.equal(far["out"], near.block) and torch.equal(far["out_residual"], near.residual)
    for a, b in ((pre, near.w_pre), (post, near.w_post), (gate, near.gate)):
        assert torch.equal(a, b)
    assert mx.device_status() == 0


def test_more_than_2_31_elements(mx):
    """Rows past 2^31 elements, against calls on those rows alone."""
    rows, cols = (1 << 31) // 16384 + 40, 16384
    g = torch.Generator(device="cuda").manual_seed(1)
    n = lambda: torch.randn(rows, cols, generator=g, device="cuda", dtype=BF16)  # noqa: E731
    block, residual, dy = n(), n(), n()
    w = torch.ones(cols, device="cuda", dtype=BF16)
    tail = slice(rows - 64, rows)
    res, y = mx.norm_residual(block, residual, w, w)
    ref = mx.norm_residual(block[tail], residual[tail], w, w)
    assert torch.equal(res[tail], ref[0]) and torch.equal(y[tail], ref[1])
    del res, y
    got = mx.norm_residual_backward(None, dy, block, residual, w, w)
    ref = mx.norm_residual_backward(None, dy[tail], block[tail], residual[tail], w, w)
    assert torch.equal(got.block[tail], ref.block) and torch.equal(got.residual[tail], ref.residual)
    assert mx.device_status() == 0


@pytest.mark.parametrize("experts,tokens,top_k", [(128, 64, 8), (129, 20, 8), (160, 40, 6),
                                                  (257, 64, 8), (384, 17, 8), (512, 64, 32)])
def test_many_experts_and_tokens(mx, experts, tokens, top_k):
    from test_gpu_moe_few import check, layer
    d, mats = layer(experts + tokens, tokens, 64, 32, experts, router=FP32)
    check(mx, d, mats, top_k, renormalize=experts % 2 == 0)
