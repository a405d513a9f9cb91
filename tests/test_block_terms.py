"""How the expert layer's operands hold a value: two E4M3 terms over a power
of two per 32 channels, and the error that this leaves."""
import numpy as np
import pytest

from oracle import block_oracle as B


def bf16(v):
    """float64 values rounded to 8 significant bits (exponents are in range)."""
    step = np.exp2(np.frexp(v)[1] - 8.0)
    return np.rint(v / step) * step


@pytest.mark.parametrize("spread", [0, 8, 13, 20, 40])
@pytest.mark.parametrize("lift", [-60, 0, 60])
def test_bf16_values(spread, lift):
    """Exactly from 2^-14 of the block's largest up, below within 2^-22 of it
    (half of lo's last step, 2^-9 / 32, against a largest of 2^7 at least)."""
    rng = np.random.default_rng(spread)
    for _ in range(200):
        v = bf16(rng.normal(size=96) * np.exp2(lift - rng.integers(0, spread + 1, 96)))
        largest = np.repeat(np.abs(v.reshape(3, 32)).max(1), 32)
        err = np.abs(B.two_terms(v) - v)
        assert (err[np.abs(v) >= 2.0 ** -14 * largest] == 0).all()
        assert (err <= 2.0 ** -22 * largest).all()


def test_small_values_beside_a_large_one_are_not_exact():
    v = np.zeros(32)
    v[0], v[1], v[2] = 1.0, bf16(2.0 ** -17 * 1.7), 2.0 ** -24
    got = B.two_terms(v)
    assert got[0] == v[0] and got[1] != v[1] and got[2] == 0
    assert abs(got[1] - v[1]) <= 2.0 ** -22


def test_values_of_any_precision():
    """An activation: half a unit of 8 significant bits, or 2^-22 of the
    block's largest."""
    rng = np.random.default_rng(1)
    for _ in range(200):
        v = rng.normal(size=64) * np.exp2(-rng.integers(0, 30, 64))
        largest = np.repeat(np.abs(v.reshape(2, 32)).max(1), 32)
        assert (np.abs(B.two_terms(v) - v) <= np.maximum(2.0 ** -8 * np.abs(v), 2.0 ** -22 * largest)).all()
    assert (B.two_terms(np.zeros(40)) == 0).all()


def layer(rng, h, inter):
    """Gate, up and down of one expert, zero at every block's first channel."""
    gate, up, down = (rng.normal(size=(1, *n)) for n in ((inter, h), (inter, h), (h, inter)))
    gate[:, :, ::32] = up[:, :, ::32] = 0
    return gate, up, down


def test_layer_bound_covers_what_the_terms_lose():
    """Tokens whose blocks span 2^24, beside weights of zero at the largest
    channel: products of what the terms hold are within the oracle's bound
    with 2^-22 of the largest besides."""
    rng = np.random.default_rng(2)
    x = bf16(rng.normal(size=(3, 64)) * np.exp2(-rng.integers(12, 24, (3, 64))))
    x[:, ::32] = 1.0
    mats = layer(rng, 64, 32)
    ids, w = np.zeros((3, 1), int), np.ones((3, 1))
    got, _ = B.moe_layer(np.stack([B.two_terms(v) for v in x]), ids, w, *mats, 0, 0)
    ref, tol = B.moe_layer(x, ids, w, *mats, 1e-4, 2.0 ** -8, 2.0 ** -22, 2.0 ** -22)
    assert (np.abs(got - ref) <= tol).all()


def test_layer_loses_channels_far_below_their_blocks_largest():
    """2^-24 beside 1 is held as zero (half of the last step is 2^-22): with
    weights of zero at the 1 nothing is left of the layer, which a bound that
    takes x exactly does not allow and the one with 2^-22 of the largest does."""
    rng = np.random.default_rng(3)
    x = np.full((1, 64), 2.0 ** -24)
    x[:, ::32] = 1.0
    mats = layer(rng, 64, 32)
    ids, w = np.zeros((1, 1), int), np.ones((1, 1))
    got, _ = B.moe_layer(np.stack([B.two_terms(v) for v in x]), ids, w, *mats, 0, 0)
    assert (got == 0).all()
    ref, tol = B.moe_layer(x, ids, w, *mats, 1e-4, 2.0 ** -8)
    assert (np.abs(ref) > tol).any()
    _, tol = B.moe_layer(x, ids, w, *mats, 1e-4, 2.0 ** -8, 2.0 ** -22, 2.0 ** -22)
    assert (np.abs(ref) <= tol).all()
