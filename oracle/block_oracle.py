"""CPU oracle of the operators around the products: the norms before and
after a block (with its gate and residual scale), their gradients, and the
mixture-of-experts layer for a few tokens.

TEST INFRASTRUCTURE ONLY, like mx_oracle.  Plain definitions in float64,
row by row, with no fusion.  Next to each value it gives the sum of the
magnitudes behind it, from which the tests take their tolerances.
"""
import numpy as np

from . import mx_oracle as O


def rms(v, w, eps):
    """v_c w_c / sqrt(mean(v^2) + eps) of one row."""
    return v * w / np.sqrt(np.mean(v * v) + eps)


def _gate_row(gate, rows, t):
    if gate is None:
        return 1.0
    g = gate.reshape(-1, gate.shape[-1])
    return g[t // (rows // len(g))]


def norm_residual_stream(block, residual, w_post, gate, alpha, eps):
    """(alpha * residual + g * n(block; w_post), |alpha residual| + |g n|)."""
    out, mag = np.empty_like(block), np.empty_like(block)
    for t in range(len(block)):
        n = block[t] if w_post is None else rms(block[t], w_post, eps)
        a, b = alpha * residual[t], _gate_row(gate, len(block), t) * n
        out[t], mag[t] = a + b, np.abs(a) + np.abs(b)
    return out, mag


def norm_rows(v, w, eps):
    return np.stack([rms(r, w, eps) for r in v]) if len(v) else np.empty_like(v)


def norm_residual_backward(d_res, dy, block, stream, w_pre, w_post, gate, alpha, eps):
    """Gradients of the two-norm step and, under `mag`, the magnitudes of the
    terms that each sums."""
    rows, cols = block.shape
    gates = 0 if gate is None else len(gate.reshape(-1, cols))
    z = np.zeros((rows, cols))
    d = dict(block=z.copy(), residual=z.copy(), w_pre=np.zeros(cols),
             w_post=None if w_post is None else np.zeros(cols),
             gate=None if gate is None else np.zeros((gates, cols)))
    mag = {k: None if v is None else np.zeros_like(v) for k, v in d.items()}
    for t in range(rows):
        r, b = stream[t], block[t]
        rho = 1 / np.sqrt(np.mean(r * r) + eps)
        a = np.zeros(cols) if d_res is None else d_res[t]
        wdy = w_pre * dy[t]
        big = a + rho * wdy - r * rho ** 3 * np.mean(wdy * r)
        bmag = np.abs(a) + np.abs(rho * wdy) + np.abs(r) * rho ** 3 * np.mean(np.abs(wdy * r))
        d["w_pre"] += dy[t] * r * rho
        mag["w_pre"] += np.abs(dy[t] * r * rho)
        g = _gate_row(gate, rows, t)
        u, umag = g * big, np.abs(g) * bmag
        if w_post is None:
            n = b
            d["block"][t], mag["block"][t] = u, umag
        else:
            s = 1 / np.sqrt(np.mean(b * b) + eps)
            n = b * s * w_post
            d["block"][t] = s * w_post * u - b * s ** 3 * np.mean(w_post * u * b)
            mag["block"][t] = (np.abs(s * w_post) * umag
                               + np.abs(b) * s ** 3 * np.mean(np.abs(w_post * b) * umag))
            d["w_post"] += u * b * s
            mag["w_post"] += umag * np.abs(b * s)
        d["residual"][t], mag["residual"][t] = alpha * big, abs(alpha) * bmag
        if gate is not None:
            at = t // (rows // gates)
            d["gate"][at] += big * n
            mag["gate"][at] += bmag * np.abs(n)
    if gate is not None:
        d["gate"], mag["gate"] = d["gate"].reshape(gate.shape), mag["gate"].reshape(gate.shape)
    d["mag"] = mag
    return d


def route(logits, top_k, renormalize):
    """Winners (largest logit first, equal ones by index) and their weights."""
    ids = np.argsort(-logits, axis=1, kind="stable")[:, :top_k]
    p = np.exp(logits - logits.max(axis=1, keepdims=True))
    p /= p.sum(axis=1, keepdims=True)
    w = np.take_along_axis(p, ids, 1)
    return ids, w / w.sum(axis=1, keepdims=True) if renormalize else w


def expert_weight(codes, scales, rows, k, fmt):
    """float64 [rows, k] of one expert's codes [rows, bytes] and swizzled scales."""
    name = fmt.replace("_packed", "")
    if fmt.endswith("_packed"):
        codes = O.unpack_dense(codes, name)
    blocks = -(-k // 32)
    s = O.e8m0_values(O.unswizzle_scales(scales, rows, blocks))
    return O.decode_table(name)[codes] * np.repeat(s, 32, axis=1)[:, :k]


def _e4m3_round(v):
    """Nearest E4M3 value, ties to even (4 significant bits, steps of 2^-9 at
    least; no value here is near the largest, 448)."""
    step = np.exp2(np.maximum(np.frexp(v)[1] - 4, -9))
    return np.rint(v / step) * step


def _block_largest(v):
    """The largest magnitude of each element's 32-element block of a row."""
    return np.repeat([np.abs(v[i:i + 32]).max() for i in range(0, len(v), 32)], 32)[:len(v)]


def two_terms(v):
    """A row as the expert layer's tensor-core operand holds it: per 32
    elements a power of two S that brings the largest into [128, 256), and
    E4M3 terms hi of v / S, lo of the rest times 32."""
    top = _block_largest(v)
    s = np.exp2(np.frexp(top)[1] - 8.0)
    u = v / np.where(top > 0, s, 1.0)
    hi = _e4m3_round(u)
    return (hi + _e4m3_round((u - hi) * 32) / 32) * np.where(top > 0, s, 1.0)


def moe_layer(x, ids, weights, gate, up, down, product_tol, h_rel, x_floor=0.0, h_floor=0.0):
    """sum_e w_e down_e (silu(gate_e x) * (up_e x)) for given winners, and a
    bound of the error of a computation whose products are off by at most
    product_tol times their sum of magnitudes and which rounds the weighted
    activation by a relative h_rel (plus h_rel^3 of the largest of its
    32-element block, where small values lose bits).  x_floor: elements of x
    below 2^-14 of the largest of their 32-element block are off by up to that
    much of it; h_floor: so are those of the activation, all of them.  gate,
    up, down: lists of float64 matrices by expert."""
    y, tol = np.zeros_like(x), np.zeros_like(x)
    for t in range(len(x)):
        largest = _block_largest(x[t])
        dx = np.where(np.abs(x[t]) < 2.0 ** -14 * largest, x_floor * largest, 0.0)
        for e, w in zip(ids[t], weights[t]):
            a, b = gate[e] @ x[t], up[e] @ x[t]
            da = product_tol * (np.abs(gate[e]) @ np.abs(x[t])) + np.abs(gate[e]) @ dx
            db = product_tol * (np.abs(up[e]) @ np.abs(x[t])) + np.abs(up[e]) @ dx
            act = a / (1 + np.exp(-a))
            h = w * act * b
            dh = abs(w) * (1.1 * da * (np.abs(b) + db) + np.abs(act) * db)
            dh += h_rel * np.abs(h) + (h_rel ** 3 + h_floor) * _block_largest(h)
            y[t] += down[e] @ h
            tol[t] += np.abs(down[e]) @ (dh + product_tol * (np.abs(h) + dh))
    return y, tol
