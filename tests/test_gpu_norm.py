"""norm_residual and its gradient against the float64 oracle.

Tolerances.  A row's sum of squares or products (c terms, FP32, each
thread at most 64 of them in sequence, then a tree) is off by less than
2^-17 of its sum of magnitudes; every other step rounds once.  So an FP32
result is within 2^-16 of the sum of the magnitudes of its terms, a BF16
one another 2^-8 of itself (half a unit in the last place), and a column sum
over R rows another R 2^-24.  The second norm and the gradient read the
stream as stored, so their reference starts from the stored values."""
import numpy as np
import pytest
import torch

from mxcheck import ensure_built, to_f64
from oracle import block_oracle as B

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32
TYPES = [(BF16, BF16, BF16), (BF16, FP32, FP32), (FP32, FP32, BF16), (FP32, FP32, FP32)]
REL = 2.0 ** -16
EPS = 1e-6


@pytest.fixture(scope="module")
def mx():
    ensure_built()
    import mxfp8_block_scaled_mx_gb300 as mx
    return mx


def close(got, ref, mag, rows=0):
    """Every element within its tolerance (`rows`: summed over that many)."""
    tol = (REL + rows * 2.0 ** -24) * mag + 1e-30
    if got.dtype == BF16:
        tol = tol + 2.0 ** -8 * np.abs(ref) + 2.0 ** -133
    err = np.abs(to_f64(got) - ref)
    assert np.isfinite(to_f64(got)).all()
    assert (err <= tol).all(), f"{float((err / tol).max()):.3g} x the tolerance"


def strided(t, pad):
    """The same rows, `pad` elements further apart, between NaNs."""
    wide = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), dtype=t.dtype, device="cuda")
    wide[:, :t.shape[1]] = t
    return wide[:, :t.shape[1]]


def inputs(rows, cols, c, s, w, post, gates, seed=0, pad=0):
    g = torch.Generator().manual_seed(seed)

    def n(*shape, std=1.0, mean=0.0, dtype=FP32):
        t = (torch.randn(*shape, generator=g) * std + mean).to(dtype).cuda()
        return strided(t, pad) if pad and len(shape) == 2 and shape[0] == rows and rows > 1 else t

    d = dict(block=n(rows, cols, std=0.5, dtype=c), residual=n(rows, cols, std=2.0, dtype=s),
             d_residual=n(rows, cols, dtype=s), d_y=n(rows, cols, dtype=c),
             w_pre=n(cols, std=0.1, mean=1.0, dtype=w))
    d["w_post"] = n(cols, std=0.1, mean=1.0, dtype=w) if post else None
    d["gate"] = None
    if gates:
        shape = (cols,) if gates == 1 else (gates, cols)
        d["gate"] = (torch.randn(*shape, generator=g) * 0.3 + 0.5).to(w).cuda()
    return d


def f64(t):
    return None if t is None else to_f64(t)


def check_forward(mx, d, alpha, eps=EPS, **kw):
    res, y = mx.norm_residual(d["block"], d["residual"], d["w_pre"], w_post=d["w_post"],
                              gate=d["gate"], alpha=alpha, eps=eps, **kw)
    ref, mag = B.norm_residual_stream(f64(d["block"]), f64(d["residual"]), f64(d["w_post"]),
                                      f64(d["gate"]), alpha, eps)
    close(res, ref, mag)
    ref = B.norm_rows(to_f64(res), f64(d["w_pre"]), eps)
    close(y, ref, np.abs(ref))
    assert mx.device_status() == 0
    return res, y


def check_backward(mx, d, alpha, eps=EPS, **kw):
    """Here d["residual"] stands for the stream that a forward pass stored."""
    got = mx.norm_residual_backward(d["d_residual"], d["d_y"], d["block"], d["residual"],
                                    d["w_pre"], w_post=d["w_post"], gate=d["gate"], alpha=alpha,
                                    eps=eps, **kw)
    ref = B.norm_residual_backward(f64(d["d_residual"]), f64(d["d_y"]), f64(d["block"]),
                                   f64(d["residual"]), f64(d["w_pre"]), f64(d["w_post"]),
                                   f64(d["gate"]), alpha, eps)
    mag, rows = ref["mag"], len(d["block"])
    close(got.block, ref["block"], mag["block"])
    close(got.residual, ref["residual"], mag["residual"])
    for name in ("w_pre", "w_post", "gate"):
        t = getattr(got, name)
        assert (t is None) == (ref[name] is None)
        if t is not None:
            assert t.dtype == FP32
            close(t, ref[name], mag[name], rows)
    assert mx.device_status() == 0
    return got


# one element, under and over a warp, odd rows, whole 16-byte runs, a single
# long row, rows that no register variant holds alike
SIZES = [(1, 1), (3, 7), (2, 33), (5, 64), (7, 1111), (4, 1000), (1, 7168), (3, 2048), (2, 4104),
         (9, 8192), (2, 16383), (2, 16384), (300, 136), (65, 257)]


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("c,s,w", TYPES)
def test_forward(mx, rows, cols, c, s, w):
    for post, gates in ((True, 0), (False, 1), (True, rows)):
        check_forward(mx, inputs(rows, cols, c, s, w, post, gates, seed=rows + cols), 0.875)


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("c,s,w", TYPES)
def test_backward(mx, rows, cols, c, s, w):
    for post, gates in ((True, 0), (False, 1), (True, rows), (True, 1)):
        check_backward(mx, inputs(rows, cols, c, s, w, post, gates, seed=rows + cols), 0.875)


@pytest.mark.parametrize("rows,gates", [(12, 4), (12, 2), (700, 7), (600, 3), (640, 320)])
@pytest.mark.parametrize("cols", [96, 515])
@pytest.mark.parametrize("post", [False, True])
def test_one_gate_per_sequence(mx, rows, gates, cols, post):
    d = inputs(rows, cols, BF16, FP32, FP32, post, gates, seed=rows + gates)
    check_forward(mx, d, 1.0)
    check_backward(mx, d, 1.0)


@pytest.mark.parametrize("cols", [8200, 9216, 12000, 16384])
@pytest.mark.parametrize("c,s,w", TYPES)
def test_rows_longer_than_a_block_holds(mx, cols, c, s, w):
    for rows, gates in ((160, 0), (9, 3), (7, 7)):
        d = inputs(rows, cols, c, s, w, True, gates, seed=cols)
        check_forward(mx, d, 0.5)
        check_backward(mx, d, 0.5)


@pytest.mark.parametrize("rows,gates", [(700, 350), (700, 700), (620, 1), (2000, 500)])
@pytest.mark.parametrize("cols", [1104, 333])
def test_many_gates_and_many_blocks(mx, rows, gates, cols):
    """More gates than blocks, gates of one row, two gates to a block."""
    check_backward(mx, inputs(rows, cols, BF16, BF16, BF16, True, gates, seed=gates), 1.0)


@pytest.mark.parametrize("pad", [1, 3, 8, 24])
@pytest.mark.parametrize("cols", [64, 1000])
def test_rows_apart_and_off_16_bytes(mx, pad, cols):
    """Rows with a leading dimension of their own, aligned and not."""
    for c, s in ((BF16, BF16), (FP32, FP32)):
        d = inputs(6, cols, c, s, BF16, True, 2, seed=pad, pad=pad)
        out = strided(torch.zeros(6, cols, dtype=c, device="cuda"), pad)
        res = strided(torch.zeros(6, cols, dtype=s, device="cuda"), pad)
        check_forward(mx, d, 0.5, out=out, out_residual=res)
        for t in (out, res):
            edge = torch.as_strided(t, (6, pad), (cols + pad, 1), cols)[:5]
            assert edge.isnan().all()                   # nothing between the rows was written
        check_backward(mx, d, 0.5)


def test_pointers_off_16_bytes(mx):
    for off in (1, 2, 5):
        d = inputs(5, 256, BF16, BF16, BF16, True, 1, seed=off)
        for k in ("block", "residual", "d_y", "d_residual"):
            flat = torch.zeros(5 * 256 + off, dtype=BF16, device="cuda")
            flat[off:] = d[k].reshape(-1)
            d[k] = flat[off:].view(5, 256)
        for k in ("w_pre", "w_post", "gate"):
            flat = torch.zeros(256 + off, dtype=BF16, device="cuda")
            flat[off:] = d[k]
            d[k] = flat[off:]
        check_forward(mx, d, 1.0)
        check_backward(mx, d, 1.0)


def test_no_gradient_from_later_blocks_and_zero_rows(mx):
    d = inputs(4, 128, BF16, FP32, FP32, True, 1)
    d["d_residual"] = None
    check_backward(mx, d, 1.0)
    d = inputs(4, 128, FP32, FP32, FP32, True, 1)
    d["block"][1] = 0
    d["residual"][2] = 0
    check_forward(mx, d, 0.0)                           # row 1: a stream of zeros
    check_backward(mx, d, 0.0)


def test_large_and_small_rows(mx):
    """Squares that come near FP32's limits, and eps that outweighs them."""
    for scale, eps in ((1e15, 0.0), (1e-12, 1e-30), (1e-6, 1.0)):
        d = inputs(3, 512, FP32, FP32, FP32, True, 0)
        d["block"] *= scale
        d["residual"] *= scale
        check_forward(mx, d, 1.0, eps=eps)
        check_backward(mx, d, 1.0, eps=eps)


def test_nan_stays_in_its_row(mx):
    d = inputs(6, 200, BF16, BF16, BF16, True, 0)
    clean = mx.norm_residual(d["block"], d["residual"], d["w_pre"], w_post=d["w_post"])
    back = mx.norm_residual_backward(None, d["d_y"], d["block"], d["residual"], d["w_pre"],
                                     w_post=d["w_post"])
    d["block"][2, 7] = float("nan")
    d["residual"][4, 0] = float("inf")
    keep = [0, 1, 3, 5]
    res, y = mx.norm_residual(d["block"], d["residual"], d["w_pre"], w_post=d["w_post"])
    assert torch.equal(res[keep], clean[0][keep]) and torch.equal(y[keep], clean[1][keep])
    assert y[2].isnan().all() and y[4, 0].isnan()
    got = mx.norm_residual_backward(None, d["d_y"], d["block"], d["residual"], d["w_pre"],
                                    w_post=d["w_post"])
    assert torch.equal(got.block[keep], back.block[keep])
    assert torch.equal(got.residual[keep], back.residual[keep])
    assert got.block[2].isnan().all() and got.residual[4].isnan().any()


def test_in_place_stream_empty_input_and_repeatability(mx):
    d = inputs(257, 1032, BF16, FP32, FP32, True, 1)
    ref = check_forward(mx, d, 0.5)
    mine = d["residual"].clone()
    res, y = mx.norm_residual(d["block"], mine, d["w_pre"], w_post=d["w_post"], gate=d["gate"],
                              alpha=0.5, out_residual=mine)
    assert res is mine and torch.equal(res, ref[0]) and torch.equal(y, ref[1])
    a, b = (check_backward(mx, d, 0.5) for _ in range(2))
    for name in ("block", "residual", "w_pre", "w_post", "gate"):
        assert torch.equal(getattr(a, name), getattr(b, name))
    # a workspace of the caller's, full of NaN
    need = mx.mx_norm_residual_backward_workspace(257, 1032, 1)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    c = check_backward(mx, d, 0.5, workspace=ws)
    assert torch.equal(a.w_pre, c.w_pre) and torch.equal(a.gate, c.gate)
    e = inputs(0, 64, BF16, BF16, BF16, True, 1)
    res, y = mx.norm_residual(e["block"], e["residual"], e["w_pre"], w_post=e["w_post"])
    assert res.shape == y.shape == (0, 64)
    g = mx.norm_residual_backward(None, e["d_y"], e["block"], e["residual"], e["w_pre"],
                                  w_post=e["w_post"], gate=e["gate"])
    for t in (g.w_pre, g.w_post, g.gate):
        assert (t == 0).all()
    assert mx.device_status() == 0


def test_gradient_against_differences(mx):
    """The gradient kernel against differences of the forward kernel.  FP32,
    a loss of about 200 terms near 1: rounding moves a difference by about
    2^-22 of the loss's magnitude (200) over twice the step, 1e-3; the
    step's own error is step^2 times a third derivative of order 1, 1e-3."""
    rows, cols, alpha, step = 2, 96, 0.75, 2.0 ** -5
    d = inputs(rows, cols, FP32, FP32, FP32, True, 1, seed=5)

    def loss(q):
        r, y = mx.norm_residual(q["block"], q["residual"], q["w_pre"], w_post=q["w_post"],
                                gate=q["gate"], alpha=alpha, eps=1e-3)
        return float((r.double() * d["d_residual"].double()).sum()
                     + (y.double() * d["d_y"].double()).sum())

    r, _ = mx.norm_residual(d["block"], d["residual"], d["w_pre"], w_post=d["w_post"],
                            gate=d["gate"], alpha=alpha, eps=1e-3)
    got = mx.norm_residual_backward(d["d_residual"], d["d_y"], d["block"], r, d["w_pre"],
                                    w_post=d["w_post"], gate=d["gate"], alpha=alpha, eps=1e-3)
    for name in ("block", "residual", "w_pre", "w_post", "gate"):
        for i in (0, 17, 95):
            hi, lo = ({**d, name: d[name].clone()} for _ in range(2))
            hi[name].view(-1)[i] += step
            lo[name].view(-1)[i] -= step
            diff = (loss(hi) - loss(lo)) / (2 * step)
            mine = float(getattr(got, name).view(-1)[i])
            assert abs(mine - diff) < 1e-2 * max(1.0, abs(diff)), (name, i, mine, diff)


def test_on_another_stream_and_in_a_graph(mx):
    d = inputs(130, 520, BF16, BF16, BF16, True, 1)
    ref = check_forward(mx, d, 1.0)
    back = check_backward(mx, d, 1.0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    args = (d["block"], d["residual"], d["w_pre"])
    kw = dict(w_post=d["w_post"], gate=d["gate"])
    got = mx.norm_residual(*args, **kw, stream=s)
    grads = mx.norm_residual_backward(d["d_residual"], d["d_y"], *args, **kw, stream=s)
    s.synchronize()
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    assert torch.equal(grads.w_pre, back.w_pre) and torch.equal(grads.gate, back.gate)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = mx.norm_residual(*args, **kw)
        grads = mx.norm_residual_backward(d["d_residual"], d["d_y"], *args, **kw)
    for _ in range(2):
        got[1].zero_()
        grads.w_post.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got[1], ref[1]) and torch.equal(grads.w_post, back.w_post)


def test_refusals(mx):
    d = inputs(4, 64, BF16, BF16, BF16, True, 2)
    call = lambda **kw: mx.norm_residual(**{**dict(  # noqa: E731
        block=d["block"], residual=d["residual"], w_pre=d["w_pre"], w_post=d["w_post"],
        gate=d["gate"]), **kw})
    call()
    for bad in (dict(block=d["block"].half()), dict(block=d["block"].cpu()),
                dict(block=d["block"][0]), dict(residual=d["residual"][:3]),
                dict(residual=d["residual"].t()), dict(w_pre=d["w_pre"][:63]),
                dict(w_post=d["w_post"].float()), dict(gate=d["gate"][:, :32]),
                dict(gate=torch.ones(3, 64, dtype=BF16, device="cuda")),
                dict(gate=torch.ones(2, 128, dtype=BF16, device="cuda")[:, ::2]),
                dict(residual=d["residual"][:1].expand(4, 64)),
                dict(out=torch.empty(4, 64, device="cuda")),
                dict(out_residual=torch.empty(4, 63, dtype=BF16, device="cuda"))):
        with pytest.raises(ValueError):
            call(**bad)
    with pytest.raises(mx.MxError) as e:                # an FP32 block on a BF16 stream
        call(block=d["block"].float())
    assert e.value.status == 3
    with pytest.raises(mx.MxError) as e:
        call(eps=-1.0)
    assert e.value.status == 1
    wide = torch.zeros(1, 16392, dtype=BF16, device="cuda")
    with pytest.raises(mx.MxError) as e:
        mx.norm_residual(wide, wide, wide[0])
    assert e.value.status == 3
    back = lambda **kw: mx.norm_residual_backward(**{**dict(  # noqa: E731
        d_residual=d["d_residual"], d_y=d["d_y"], block=d["block"], residual=d["residual"],
        w_pre=d["w_pre"]), **kw})
    back()
    for bad in (dict(d_y=d["d_y"].float()), dict(d_residual=d["d_residual"][:, :8]),
                dict(workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(ValueError):
            back(**bad)
    assert mx.device_status() == 0


def placed(t, ld, offset, fill=7.0):
    """t's values as rows `ld` apart, `offset` elements into a buffer of
    `fill`; the buffer, too."""
    rows, cols = t.shape
    flat = torch.full((offset + rows * ld + 16,), fill, dtype=t.dtype, device="cuda")
    view = flat[offset:offset + rows * ld].view(rows, ld)[:, :cols]
    view.copy_(t)
    return view, flat


@pytest.mark.parametrize("cols,ld", [(1, 3), (5, 5), (8, 9), (9, 9), (15, 21), (17, 17), (130, 131),
                                     (1017, 1017), (1018, 1025), (1111, 1111), (4089, 4089),
                                     (4090, 4097), (8191, 8191), (16377, 16377), (16378, 16379)])
@pytest.mark.parametrize("c,s,w", TYPES)
def test_rows_off_16_bytes(mx, cols, ld, c, s, w):
    """Rows that begin anywhere, in step in all arrays or not, with weights
    and gates off 16 bytes; what lies around the outputs stays."""
    rows = 11
    d = inputs(rows, cols, c, s, w, True, rows, seed=cols)
    d["w_pre"] = placed(d["w_pre"][None], cols, 3)[0][0]
    d["w_post"] = placed(d["w_post"][None], cols, 5)[0][0]
    d["gate"] = placed(d["gate"], cols, 1)[0]
    for base in (0, 3, 7):
        for apart in (0, 1):                             # every array as far into its 16 bytes, or not
            for i, n in enumerate(("block", "residual")):
                d[n] = placed(d[n], ld, base + apart * i)[0]
            out, flat_out = placed(torch.full((rows, cols), 7.0, dtype=c, device="cuda"), ld, base)
            res, flat_res = placed(torch.full((rows, cols), 7.0, dtype=s, device="cuda"), ld, base)
            check_forward(mx, d, 0.875, out_residual=res, out=out)
            kept = out.clone(), res.clone()
            for view, flat in ((out, flat_out), (res, flat_res)):
                view.fill_(7.0)
                assert bool((flat == 7.0).all())         # nothing around it was written
            before = d["residual"].clone()
            mx.norm_residual(d["block"], d["residual"], d["w_pre"], w_post=d["w_post"],
                             gate=d["gate"], alpha=0.875, out_residual=d["residual"], out=out)
            assert torch.equal(out, kept[0]) and torch.equal(d["residual"], kept[1])
            d["residual"] = before


@pytest.mark.parametrize("cols", [1032, 1536, 2560, 3584])
@pytest.mark.parametrize("c,s,w", TYPES)
def test_gradient_rows_of_one_or_two_runs(mx, cols, c, s, w):
    for rows, gates in ((1, 0), (40, 0), (700, 7), (650, 1)):
        check_backward(mx, inputs(rows, cols, c, s, w, True, gates, seed=cols), 0.5)


@pytest.mark.parametrize("cols,ld", [(1, 1), (3, 11), (33, 34), (130, 130), (132, 140), (1018, 1026),
                                     (1111, 1111), (1000, 1000), (2049, 2057), (4089, 4089),
                                     (4090, 4098), (8185, 8185), (8186, 8186)])
@pytest.mark.parametrize("c,s,w", TYPES)
def test_gradient_rows_off_16_bytes(mx, cols, ld, c, s, w):
    """Rows that begin anywhere, in step in all arrays or not; gates of few and
    many rows, none; more rows than blocks and fewer."""
    for rows, gates, base in ((1, 0, 0), (7, 0, 8), (17, 1, 0), (96, 2, 3), (97, 97, 0), (640, 16, 8),
                              (1300, 0, 0), (1300, 13, 0)):
        if rows * cols > 3_000_000:
            rows, gates = 320, min(gates, 4)
        d = inputs(rows, cols, c, s, w, True, gates, seed=rows + cols)
        d["w_pre"] = placed(d["w_pre"][None], cols, 3)[0][0]
        d["w_post"] = placed(d["w_post"][None], cols, 5)[0][0]
        for n in ("block", "residual", "d_residual", "d_y"):
            d[n] = placed(d[n], ld, base)[0]
        got = check_backward(mx, d, 0.875)
        again = check_backward(mx, d, 0.875)
        for name in ("block", "residual", "w_pre", "w_post", "gate"):
            a, b = getattr(got, name), getattr(again, name)
            assert a is None or torch.equal(a, b)


@pytest.mark.parametrize("rows,cols,gates", [(9800, 1111, 0), (9800, 1026, 350), (9744, 1028, 1),
                                             (300, 4101, 0), (320, 5002, 20), (330, 4100, 1),
                                             (700, 7999, 7)])
@pytest.mark.parametrize("c,s,w", TYPES[:3])
def test_gradient_of_many_rows_off_16_bytes(mx, rows, cols, gates, c, s, w):
    """Rows by phase: eight, four and two phases, gates of one run of rows and
    of many, within blocks and across."""
    d = inputs(rows, cols, c, s, w, True, gates, seed=rows + cols, pad=0 if cols % 4 else 1)
    if cols % 4 == 0:                                    # in step, off 16 bytes by the weights alone
        for n in ("block", "residual", "d_residual", "d_y"):
            d[n] = placed(d[n].contiguous(), cols + 8, 8)[0]
        d["w_pre"] = placed(d["w_pre"][None], cols, 3)[0][0]
    got = check_backward(mx, d, 0.875)
    again = check_backward(mx, d, 0.875)
    assert torch.equal(got.w_pre, again.w_pre) and torch.equal(got.w_post, again.w_post)
