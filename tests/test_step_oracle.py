"""Checks of the oracle of the operators between the products: gradients against
differences, closed forms."""
import numpy as np
import pytest

from oracle import step_oracle as S


def difference(f, x, i, h=1e-6):
    a, b = x.copy(), x.copy()
    a.flat[i] += h
    b.flat[i] -= h
    return (f(a) - f(b)) / (2 * h)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotated_norm_and_its_gradient(interleaved):
    g = np.random.default_rng(1)
    x, w, dy = g.normal(size=(3, 2, 10)), g.normal(size=10), g.normal(size=(3, 2, 10))
    pos, freq = np.array([0, 7, -3]), np.array([1.0, 0.3, 0.01])
    args = (pos, freq, interleaved, 1.5, 1e-3)
    y, _ = S.norm_rotate(x, w, *args)
    # position 0 scales only; turning keeps a pair's length
    n = x / np.sqrt(np.mean(x * x, -1, keepdims=True) + 1e-3) * w
    assert np.allclose(y[0, :, :6], 1.5 * n[0, :, :6]) and np.allclose(y[..., 6:], n[..., 6:])
    assert np.allclose((y[..., :6] ** 2).sum(-1), 2.25 * (n[..., :6] ** 2).sum(-1))
    dx, _, dw, _ = S.norm_rotate_backward(dy, x, w, *args)
    for i in range(0, x.size, 7):
        assert np.isclose(dx.flat[i], difference(lambda v: (S.norm_rotate(v, w, *args)[0] * dy).sum(), x, i), rtol=1e-6)
    for i in range(10):
        assert np.isclose(dw[i], difference(lambda v: (S.norm_rotate(x, v, *args)[0] * dy).sum(), w, i), rtol=1e-6)


def test_angles_of_far_positions_are_exact():
    x = np.array([[[1.0, 0.0]]])
    # 2 pi / 8 radians a position: every eighth position is a whole turn (the
    # frequency as a double is off by 2^-54 of itself at most)
    f = np.array([np.pi / 4])
    for k in (1, 8 * 10 ** 6 + 1):
        y, _ = S._turn(x, np.array([k]), f, True, 1.0, 1.0)
        assert np.allclose(y, [[[np.sqrt(0.5), np.sqrt(0.5)]]], atol=1e-8)


@pytest.mark.parametrize("renormalize", [False, True])
def test_routing_gradient(renormalize):
    g = np.random.default_rng(2)
    z, mask = g.normal(size=(6, 5)), np.array([1, 1, 0, 1, 0, 1])
    dw, db, dl = g.normal(size=(6, 2)), 0.7, g.normal(size=6)
    r = S.route(z, 2, renormalize, mask)
    assert r["counts"].sum() == 8 and r["offsets"][-1] == 12
    assert sorted(r["order"]) == list(range(12))

    def total(v):
        q = S.route(v, 2, renormalize, mask)
        return (q["weights"] * dw).sum() + db * q["balance"] + (q["lse"] * dl).sum()

    d, mag = S.route_backward(r, 2, renormalize, dw, db, dl)
    assert (np.abs(d) <= mag * (1 + 1e-12)).all()
    for i in range(z.size):
        assert np.isclose(d.flat[i], difference(total, z, i), rtol=1e-6, atol=1e-9)


def test_routing_of_special_logits():
    z = np.array([[1.0, 1.0, 3.0, 1.0], [np.nan, 2.0, -np.inf, np.nan]])
    r = S.route(z, 3, True, None)
    assert r["ids"].tolist() == [[2, 0, 1], [1, 2, 0]]
    assert np.isnan(r["weights"][1]).all()
    assert S.route(np.zeros((4, 4)), 1, False, None)["balance"] == pytest.approx(1.0)
    assert S.route(np.zeros((2, 4)), 1, False, np.zeros(2))["balance"] == 0.0


def test_cross_entropy_gradient():
    g = np.random.default_rng(3)
    x, w = g.normal(size=(4, 3)), g.normal(size=(6, 3))
    labels = np.array([5, -100, 0, 2])
    dl, ds = g.normal(size=4), g.normal(size=4)

    def total(a, b):
        loss, lse, _, _ = S.cross_entropy(a, b, labels, -100)
        return (loss * dl).sum() + (lse * ds).sum()

    loss, lse, z, _ = S.cross_entropy(x, w, labels, -100)
    assert loss[1] == 0 and np.allclose(np.exp(z - lse[:, None]).sum(1), 1)
    d = S.cross_entropy_backward(x, w, labels, -100, dl, ds, z, lse)
    for i in range(x.size):
        assert np.isclose(d["dx"].flat[i], difference(lambda v: total(v, w), x, i), rtol=1e-6, atol=1e-9)
    for i in range(w.size):
        assert np.isclose(d["dw"].flat[i], difference(lambda v: total(x, v), w, i), rtol=1e-6, atol=1e-9)
