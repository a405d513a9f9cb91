"""The block operators' C entries and calls on other streams: pointers as a
caller with buffers of its own passes them, and memory that a call takes for
itself.  Tolerances are those of test_gpu_norm and test_gpu_moe_few."""
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
