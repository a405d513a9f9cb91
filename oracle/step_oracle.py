"""CPU oracle of the training step's operators between the products: the norms
of query and key heads with their rotation, routing with its balance loss, and
the cross entropy over a vocabulary, each with its gradient.

TEST INFRASTRUCTURE ONLY, like mx_oracle.  Plain definitions in float64.  Next
to each value it gives the sum of the magnitudes behind it, from which the
tests take their tolerances.
"""
from fractions import Fraction

import numpy as np

TWO_PI = Fraction("6.283185307179586476925286766559005768394338798750211641949889")


def _pairs(rotary, interleaved):
    i = np.arange(rotary // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rotary // 2)


def _turn(v, positions, frequencies, interleaved, scale, sign):
    """(v with its pairs turned, magnitudes) for v [tokens, heads, dim]."""
    # the angle modulo a turn, exactly
    angle = np.array([[float(int(t) * f % 1) for f in [Fraction(float(f)) / TWO_PI for f in frequencies]]
                      for t in positions]).reshape(len(positions), 1, len(frequencies)) * 2 * np.pi
    a, b = _pairs(2 * len(frequencies), interleaved)
    c, s = scale * np.cos(angle), sign * scale * np.sin(angle)
    out, mag = v.copy(), np.abs(v)
    out[..., a] = v[..., a] * c - v[..., b] * s
    out[..., b] = v[..., a] * s + v[..., b] * c
    mag[..., a] = mag[..., b] = abs(scale) * (np.abs(v[..., a]) + np.abs(v[..., b]))
    return out, mag


def norm_rotate(x, w, positions, frequencies, interleaved, scale, eps):
    """(y, magnitudes) of one tensor of heads."""
    n = x / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps) * w
    return _turn(n, positions, frequencies, interleaved, scale, 1.0)


def norm_rotate_backward(dy, x, w, positions, frequencies, interleaved, scale, eps):
    """(dx, its magnitudes, dw, its magnitudes)."""
    dn, mag = _turn(dy, positions, frequencies, interleaved, scale, -1.0)
    rho = 1 / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps)
    dx = rho * (w * dn - x * rho ** 2 * np.mean(w * dn * x, -1, keepdims=True))
    dx_mag = rho * (np.abs(w) * mag + np.abs(x) * rho ** 2 * np.mean(np.abs(w * x) * mag, -1, keepdims=True))
    return dx, dx_mag, (dn * x * rho).sum((0, 1)), (mag * np.abs(x) * rho).sum((0, 1))


def softmax(z):
    with np.errstate(invalid="ignore", over="ignore"):
        p = np.exp(z - z.max(1, keepdims=True))
        return p / p.sum(1, keepdims=True)


def route(z, top_k, renormalize, mask):
    """What mx.route returns, as a dict (and p)."""
    tokens, experts = z.shape
    # equal ones by index, NaN below -infinity
    ids = np.argsort(-z, axis=1, kind="stable")[:, :top_k]
    for t in np.nonzero(np.isnan(z).any(1))[0]:
        ids[t] = sorted(range(experts), key=lambda e: (np.isnan(z[t, e]), 0.0 if np.isnan(z[t, e]) else -z[t, e], e))[:top_k]
    p = softmax(z) if tokens else z
    w = np.take_along_axis(p, ids, 1)
    if renormalize:
        w = w / w.sum(1, keepdims=True)
    count = np.ones(tokens, bool) if mask is None else mask.astype(bool)
    flat = ids.reshape(-1)
    load = np.bincount(flat, minlength=experts)
    counts = np.bincount(ids[count].reshape(-1), minlength=experts)
    n = int(count.sum())
    balance = float(experts * np.sum(counts / (n * top_k) * p[count].mean(0))) if n else 0.0
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        top = z.max(1) if tokens else np.zeros(0)
        lse = top + np.log(np.exp(z - top[:, None]).sum(1)) if tokens else np.zeros(0)
    return dict(ids=ids, weights=w, counts=counts, offsets=np.concatenate([[0], np.cumsum(load)]),
                order=np.argsort(flat, kind="stable"), balance=balance, lse=lse, p=p, n=n, mask=count)


def route_backward(r, top_k, renormalize, d_weights, d_balance, d_lse):
    """(d_logits, magnitudes) from route's dict."""
    p, ids, w = r["p"], r["ids"], r["weights"]
    experts = p.shape[1]
    g, mag = np.zeros_like(p), np.zeros_like(p)
    if r["n"]:
        share = d_balance * experts * r["counts"] / (r["n"] ** 2 * top_k)
        g[r["mask"]] += share
        mag[r["mask"]] += np.abs(share)
    inner = (p * g).sum(1, keepdims=True)
    dz, dm = p * (g - inner), p * (mag + (p * mag).sum(1, keepdims=True))
    dot, dot_mag = (w * d_weights).sum(1, keepdims=True), np.abs(w * d_weights).sum(1, keepdims=True)
    add = w * (d_weights - (dot if renormalize else 0.0))
    add_mag = np.abs(w) * (np.abs(d_weights) + (dot_mag if renormalize else 0.0))
    for t in range(len(p)):
        dz[t, ids[t]] += add[t]
        dm[t, ids[t]] += add_mag[t]
    if not renormalize:
        dz -= p * dot
        dm += p * dot_mag
    return dz + p * d_lse[:, None], dm + p * np.abs(d_lse)[:, None]


def cross_entropy(x, w, labels, ignore):
    """(loss, lse, z, the largest sum of magnitudes behind a z of each row)."""
    z = x @ w.T
    top = z.max(1)
    lse = top + np.log(np.exp(z - top[:, None]).sum(1))
    valid = labels != ignore
    at = np.where(valid, labels, 0)
    loss = np.where(valid, lse - z[np.arange(len(z)), at], 0.0)
    return loss, lse, z, (np.abs(x) @ np.abs(w).T).max(1)


def cross_entropy_backward(x, w, labels, ignore, d_loss, d_lse, z, lse):
    """dict of dz, dx, dw and of the sums of magnitudes |dz| |w|, |dz| |x|, and
    the same with the softmax's part alone (p)."""
    valid = labels != ignore
    d = np.where(valid, d_loss, 0.0)
    p = np.exp(z - lse[:, None]) * (d + d_lse)[:, None]
    dz = p.copy()
    rows = np.nonzero(valid)[0]
    dz[rows, labels[rows]] -= d[rows]
    return dict(dz=dz, dx=dz @ w, dw=dz.T @ x, dx_mag=np.abs(dz) @ np.abs(w),
                dw_mag=np.abs(dz).T @ np.abs(x), p_x=np.abs(p) @ np.abs(w), p_w=np.abs(p).T @ np.abs(x))
