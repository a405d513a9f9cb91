"""Pins of the block operators' oracle: its gradients against differences of
its own forward pass, its routing and layer against hand-made cases."""
import numpy as np
import pytest

from oracle import block_oracle as B
from oracle import mx_oracle as O


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gates", [0, 1, 2, 6])
def test_norm_gradients_against_differences(post, gates):
    rng = np.random.default_rng(gates * 2 + post)
    rows, cols, alpha, eps = 6, 11, 0.75, 1e-3
    p = dict(block=rng.normal(size=(rows, cols)), residual=rng.normal(size=(rows, cols)),
             w_pre=rng.normal(1, 0.2, cols))
    if post:
        p["w_post"] = rng.normal(1, 0.2, cols)
    if gates:
        p["gate"] = rng.normal(0.5, 0.3, (gates, cols))
    d_res, dy = rng.normal(size=(rows, cols)), rng.normal(size=(rows, cols))

    def loss(q):
        s, _ = B.norm_residual_stream(q["block"], q["residual"], q.get("w_post"), q.get("gate"),
                                      alpha, eps)
        return (s * d_res).sum() + (B.norm_rows(s, q["w_pre"], eps) * dy).sum()

    stream, _ = B.norm_residual_stream(p["block"], p["residual"], p.get("w_post"), p.get("gate"),
                                       alpha, eps)
    d = B.norm_residual_backward(d_res, dy, p["block"], stream, p["w_pre"], p.get("w_post"),
                                 p.get("gate"), alpha, eps)
    # a central difference is off by step^2/6 times the third derivative
    # (~1e-10 here) and by rounding, 2^-52 of the loss over the step (~1e-10)
    step = 1e-5
    for name, v in p.items():
        for i in rng.choice(v.size, min(v.size, 12), replace=False):
            hi, lo = ({**p, name: v.copy()} for _ in range(2))
            hi[name].flat[i] += step
            lo[name].flat[i] -= step
            diff = (loss(hi) - loss(lo)) / (2 * step)
            assert abs(d[name].flat[i] - diff) < 1e-7 * max(1, abs(diff)), (name, i)


def test_norm_of_ones_and_zeros():
    ones = np.ones((1, 8))
    s, _ = B.norm_residual_stream(2 * ones, 3 * ones, np.full(8, 5.0), None, 0.5, 0.0)
    assert np.allclose(s, 1.5 + 5)                    # n(2) = 1, times 5
    assert np.allclose(B.norm_rows(s, np.full(8, 2.0), 0.0), 2)
    s, _ = B.norm_residual_stream(0 * ones, ones, np.ones(8), None, 1.0, 1e-6)
    assert np.array_equal(s, ones)                    # an empty block leaves the stream


def test_routing():
    z = np.log(np.array([[1.0, 4, 2, 1], [1, 1, 1, 1], [8, 1, 8, 3]]))
    ids, w = B.route(z, 2, False)
    assert ids.tolist() == [[1, 2], [0, 1], [0, 2]]   # ties: the lowest index
    assert np.allclose(w, [[0.5, 0.25], [0.25, 0.25], [0.4, 0.4]])
    assert np.allclose(B.route(z, 2, True)[1], [[2 / 3, 1 / 3], [0.5, 0.5], [0.5, 0.5]])


def test_layer_of_identities_is_the_weighted_activation():
    n = 32
    eye = [np.eye(n), 2 * np.eye(n)]
    x = np.linspace(-2, 2, n)[None]
    y, _ = B.moe_layer(x, np.array([[1, 0]]), np.array([[0.25, 0.75]]), eye, eye, eye, 0, 0)
    s = x / (1 + np.exp(-x))
    s2 = 2 * x / (1 + np.exp(-2 * x))
    assert np.allclose(y, 0.75 * s * x + 0.25 * 2 * s2 * 2 * x)


def test_expert_weight_is_the_dequantized_operand():
    rng = np.random.default_rng(0)
    for fmt in ("e4m3", "e5m2", "e2m1"):
        q = O.quantize(rng.normal(size=(40, 128)), fmt, "row")
        got = B.expert_weight(O.pack_dense(q.codes, fmt), O.swizzle_scales(q.scales), 40, 128,
                              fmt + "_packed" if fmt == "e2m1" else fmt)
        assert np.array_equal(got, O.dequantize(q))
