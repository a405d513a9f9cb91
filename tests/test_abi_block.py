"""Host-only checks of the block operators' C entries: sizes of workspaces,
and refusal of invalid arguments before a device is touched."""
import pytest

from mxcheck import ensure_built

FAKE = 0x10000


@pytest.fixture(scope="module")
def mx():
    ensure_built()
    import mxfp8_block_scaled_mx_gb300 as mx
    return mx


NORM = dict(rows=4, cols=64, block=FAKE, ldb=64, c=0, residual=FAKE, ldr=64, s=0, w_post=FAKE,
            w_pre=FAKE, gate=FAKE, gates=2, w=0, alpha=1.0, eps=1e-6, res_out=FAKE, ldo=64, y=FAKE,
            ldy=64, stream=0)
BACK = dict(rows=4, cols=64, d_res=FAKE, ldd=64, dy=FAKE, lddy=64, block=FAKE, ldb=64, c=0,
            res_out=FAKE, ldr=64, s=0, w_post=FAKE, w_pre=FAKE, gate=FAKE, gates=2, w=0, alpha=1.0,
            eps=1e-6, d_block=FAKE, lddb=64, d_residual=FAKE, lddr=64, d_w_post=FAKE, d_w_pre=FAKE,
            d_gate=FAKE, workspace=FAKE, workspace_bytes=1 << 40, stream=0)
MOE = dict(tokens=4, hidden=256, inter=128, experts=4, top_k=2, x=FAKE, ldx=256, router=FAKE,
           router_dtype=0, gate=FAKE, gate_scales=FAKE, up=FAKE, up_scales=FAKE, fmt_gu=0,
           down=FAKE, down_scales=FAKE, fmt_d=0, renormalize=1, y=FAKE, ldy=256, ids=FAKE,
           weights=FAKE, workspace=FAKE, workspace_bytes=1 << 40, stream=0)


def test_norm_rejects_bad_arguments_on_the_host(mx):
    call = lambda **kw: mx.mx_norm_residual(*{**NORM, **kw}.values())  # noqa: E731
    for name in ("block", "residual", "w_pre", "res_out", "y"):
        assert call(**{name: None}) == 1
    for name in ("ldb", "ldr", "ldo", "ldy"):
        assert call(**{name: 63}) == 1
    for name in ("c", "s", "w"):
        assert call(**{name: 2}) == 1
    assert call(rows=-1) == 1 and call(cols=0) == 1
    assert call(gates=3) == 1 and call(gates=0) == 1
    assert call(eps=-1.0) == 1 and call(eps=float("nan")) == 1
    wide = dict(cols=16385, ldb=16385, ldr=16385, ldo=16385, ldy=16385)
    assert call(**wide) == 3
    assert call(rows=1 << 31) == 3
    assert call(c=1) == 3                      # an FP32 block on a BF16 stream
    assert call(block=FAKE + 1) == 2 and call(s=1, residual=FAKE + 2) == 2
    assert call(w=1, gate=FAKE + 2) == 2


def test_norm_backward_rejects_bad_arguments_on_the_host(mx):
    call = lambda **kw: mx.mx_norm_residual_backward(*{**BACK, **kw}.values())  # noqa: E731
    for name in ("dy", "block", "res_out", "w_pre", "d_block", "d_residual", "d_w_pre",
                 "workspace", "d_w_post", "d_gate", "w_post", "gate"):
        assert call(**{name: None}) == 1, name
    for name in ("ldd", "lddy", "ldb", "ldr", "lddb", "lddr"):
        assert call(**{name: 63}) == 1
    assert call(workspace_bytes=0) == 1
    assert call(gates=3) == 1 and call(c=3) == 1
    assert call(c=1) == 3
    assert call(workspace=FAKE + 8) == 2 and call(d_gate=FAKE + 2) == 2 and call(dy=FAKE + 1) == 2
    size = mx.mx_norm_residual_backward_workspace
    assert size(4, 64, 2) > 0
    assert size(4, 64, 3) == 0 and size(-1, 64, 0) == 0 and size(4, 0, 0) == 0
    assert size(4, 16385, 0) == 0 and size(4, 64, -1) == 0


def test_moe_rejects_bad_arguments_on_the_host(mx):
    call = lambda **kw: mx.mx_moe_few_tokens(*{**MOE, **kw}.values())  # noqa: E731
    for name in ("x", "router", "gate", "gate_scales", "up", "up_scales", "down", "down_scales",
                 "y", "ids", "weights", "workspace"):
        assert call(**{name: None}) == 1, name
    assert call(tokens=-1) == 1 and call(tokens=65) == 3
    assert call(hidden=264, ldx=264, ldy=264) == 1 and call(inter=8) == 1
    assert call(experts=0) == 1 and call(experts=513) == 1
    assert call(top_k=0) == 1 and call(top_k=5) == 1
    assert call(experts=64, top_k=33) == 1
    assert call(ldx=248) == 1 and call(ldy=248) == 1
    assert call(router_dtype=2) == 1
    for name in ("fmt_gu", "fmt_d"):
        assert call(**{name: 8}) == 1
        assert call(**{name: 4}) == 3 and call(**{name: 5}) == 3
    assert call(fmt_gu=7, hidden=272, ldx=272, ldy=272) == 1   # packed: whole 128-element tiles
    assert call(fmt_d=7, inter=144) == 1
    assert call(workspace_bytes=64) == 1
    for name in ("x", "router", "gate", "gate_scales", "up", "up_scales", "down", "down_scales",
                 "y", "workspace"):
        assert call(**{name: FAKE + 8}) == 2, name
    assert call(ldx=260) == 2 and call(ldy=260) == 2
    assert call(fmt_gu=7, gate=FAKE + 16) == 2 and call(fmt_d=7, down=FAKE + 16) == 2
    assert call(ids=FAKE + 2) == 2
    size = mx.mx_moe_few_tokens_workspace
    assert size(4, 256, 128, 4, 2) > 0
    assert size(65, 256, 128, 4, 2) == 0 and size(4, 250, 128, 4, 2) == 0
    assert size(4, 256, 128, 4, 5) == 0


def test_tensor_api_refuses_host_tensors(mx, monkeypatch):
    """Without a GPU too, and before anything is launched; without the built
    module every call raises."""
    import torch
    x = torch.zeros(4, 128, dtype=torch.bfloat16)
    w = torch.ones(128, dtype=torch.bfloat16)
    codes = mx.MxTensor(torch.zeros(2, 128, 128, dtype=torch.uint8),
                        torch.zeros(1024, dtype=torch.uint8), "e4m3")
    calls = (lambda: mx.norm_residual(x, x, w), lambda: mx.norm_residual_backward(None, x, x, x, w),
             lambda: mx.moe_few_tokens(x, torch.zeros(2, 128), codes, codes, codes, 1))
    for call in calls:
        with pytest.raises(ValueError):
            call()
    for bad in (None, 3, [x]):
        with pytest.raises(ValueError):
            mx.norm_residual(bad, x, w)
        with pytest.raises(ValueError):
            mx.moe_few_tokens(bad, x, codes, codes, codes, 1)
    monkeypatch.setattr(mx, "_binding", None)
    monkeypatch.setattr(mx, "BINDING_PATH", "/nowhere/_binding.so")
    for call in calls:
        with pytest.raises(RuntimeError):
            call()
