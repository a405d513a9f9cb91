"""Cases, plain forms and exact forms of the training step's operators between
the products of a mixture-of-experts model.

Three operators, each with its gradient, as such a model's step meets them:

* `norm_rotate`: the norms of the query and key heads that the first product of
  an attention block gives, with the rotation by position in the same pass;
* `route`: the experts of every token from the router's logits, with the counts,
  offsets and order that the grouped products take, and the balance loss;
* `linear_cross_entropy`: the vocabulary product and the softmax cross entropy of
  its logits, which are not kept.

`run` computes them in plain torch operations in 32 bits (angles in 64) where
`own` is false, and with the framework's entry points where it is true.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
_SIZE = {"bf16": 2, "fp32": 4}
EPS = 1e-6
IGNORE = -100


# ------------------------------------------------------------------ cases

def listed():
    rot = dict(op="rotate", back=False, q_heads=32, k_heads=8, dim=128, rotary=128, interleaved=False,
               factor=1.0, x="bf16", w="bf16")
    route = dict(op="route", back=True, renormalize=True, masked=False, logits="fp32")
    loss = dict(op="loss", back=True, ignored=0.1, z_loss=False)
    return [
        # decoding: one token's heads, far into a long context
        dict(rot, name="rotate_1x40x128", tokens=1, factor=8.0),
        # the heads of a training step's or a prompt's tokens
        dict(rot, name="rotate_16384x40x128", tokens=16384),
        # the gradient of such a step, and of an odd one: part of each head rotated in
        # adjacent pairs, all in FP32
        dict(rot, name="rotate_back_16384x40x128", tokens=16384, back=True),
        dict(rot, name="rotate_back_777x7x80", tokens=777, back=True, q_heads=6, k_heads=1, dim=80,
             rotary=32, interleaved=True, factor=4.0, x="fp32", w="fp32"),
        # one token through many small experts: latency counts
        dict(route, name="route_1x128_top8", tokens=1, experts=128, top_k=8, back=False),
        # the tokens of the mixture-of-experts benchmark over its 64 experts, both directions
        dict(route, name="route_65536x64_top8", tokens=65536, experts=64, top_k=8),
        # odd sizes, padding tokens, bf16 logits with ties, weights as they are
        dict(route, name="route_4097x20_top3", tokens=4097, experts=20, top_k=3, renormalize=False,
             masked=True, logits="bf16"),
        # scoring one token
        dict(loss, name="loss_1x4096x131072", tokens=1, hidden=4096, vocab=131072, back=False,
             ignored=0.0),
        # scoring a text: losses alone, a vocabulary of odd size
        dict(loss, name="loss_777x2048x50257", tokens=777, hidden=2048, vocab=50257, back=False),
        # training: losses and both gradients of a small batch, of an odd one with a term in the
        # normalizer's square, and of a large one
        dict(loss, name="loss_back_2048x2048x32768", tokens=2048, hidden=2048, vocab=32768),
        dict(loss, name="loss_back_333x1000x18433", tokens=333, hidden=1000, vocab=18433,
             z_loss=True),
        dict(loss, name="loss_back_4096x7168x131072", tokens=4096, hidden=7168, vocab=131072),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotate", "route", "loss"])
    while True:
        if op == "rotate":
            dim = rng.choice([64, 80, 96, 128, 128, 192, 256, rng.randint(4, 256)])
            c = dict(op=op, tokens=_log(rng, 1, 16384), q_heads=_log(rng, 1, 64),
                     k_heads=_log(rng, 1, 16), dim=dim,
                     rotary=dim // 2 * 2 if rng.random() < 0.5 else 2 * rng.randint(1, dim // 2),
                     interleaved=rng.random() < 0.4, factor=rng.choice([1.0, 1.0, 4.0, 16.0]),
                     back=rng.random() < 0.5, x=rng.choice(["bf16", "bf16", "fp32"]),
                     w=rng.choice(["bf16", "fp32"]))
            fits = c["tokens"] * (c["q_heads"] + c["k_heads"]) * dim * _SIZE[c["x"]] <= 16384 * 40 * 256
        elif op == "route":
            experts = _log(rng, 2, 512)
            c = dict(op=op, tokens=_log(rng, 1, 65536), experts=experts,
                     top_k=rng.randint(1, min(8, experts)), back=rng.random() < 0.6,
                     renormalize=rng.random() < 0.5, masked=rng.random() < 0.5,
                     logits=rng.choice(["bf16", "fp32"]))
            fits = c["tokens"] * experts <= 65536 * 64
        else:
            c = dict(op=op, tokens=_log(rng, 1, 4096), hidden=8 * _log(rng, 8, 896),
                     vocab=_log(rng, 1000, 131072), back=rng.random() < 0.6,
                     ignored=rng.choice([0.0, 0.1, 0.5]), z_loss=rng.random() < 0.3)
            fits = True
        if fits:
            return c


def work(case):
    t = case["tokens"]
    if case["op"] == "rotate":
        n = t * (case["q_heads"] + case["k_heads"]) * case["dim"]
        tables = 2 * case["dim"] * _SIZE[case["w"]] + 4 * case["rotary"] + 8 * t
        grads = 8 * case["dim"] if case["back"] else 0
        return {"bytes": n * _SIZE[case["x"]] * (3 if case["back"] else 2) + tables + grads,
                "flops": n * (16 if case["back"] else 8)}
    if case["op"] == "route":
        e, k = case["experts"], case["top_k"]
        # logits in; ids, weights and order out; counts and offsets
        size = t * e * _SIZE[case["logits"]] + 12 * t * k + 8 * e + (t if case["masked"] else 0)
        if case["back"]:  # the weights' gradient in, the logits' out
            size += 4 * t * k + t * e * _SIZE[case["logits"]]
        return {"bytes": size, "flops": t * e * (12 if case["back"] else 6)}
    h, v = case["hidden"], case["vocab"]
    products = 3 if case["back"] else 1
    return {"bytes": 2 * (t * h + v * h) * (2 if case["back"] else 1) + 24 * t,
            "flops": 2 * products * t * h * v}


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def normal(*shape, std=1.0, mean=0.0, dtype=torch.float32):
        return (torch.randn(shape, generator=g, device=dev) * std + mean).to(dtype)

    def integers(lo, hi, *shape):
        return torch.randint(lo, hi, shape, generator=g, device=dev)

    s = dict(case)
    t = case["tokens"]
    if case["op"] == "rotate":
        hq, hk, d = case["q_heads"], case["k_heads"], case["dim"]
        x, w = _DT[case["x"]], _DT[case["w"]]
        # queries and keys are parts of one product's rows, values behind them
        rows = normal(t, hq + 2 * hk, d, std=1.5, dtype=x)
        s["q"], s["k"] = rows[:, :hq], rows[:, hq:hq + hk]
        s["w_q"], s["w_k"] = (normal(d, std=0.1, mean=1.0, dtype=w) for _ in range(2))
        # a run of positions that starts anywhere in a long context
        s["positions"] = torch.arange(t, device=dev) + integers(0, 1 << 17, 1)
        half = case["rotary"] // 2
        i = torch.arange(half, dtype=torch.float64, device=dev)
        f = torch.exp(i * (-math.log(500000.0) / half))
        # for contexts longer than the trained one the slow frequencies are divided by the factor
        slow = ((i / half - 0.25) * 2).clamp(0, 1)
        s["frequencies"] = f * (1 - slow) + f / case["factor"] * slow
        s["scale"] = 1.0 + 0.1 * math.log(case["factor"])
        if case["back"]:
            s["d_q"] = normal(t, hq, d, std=1e-3, dtype=x)
            s["d_k"] = normal(t, hk, d, std=1e-3, dtype=x)
        return s
    if case["op"] == "route":
        e = case["experts"]
        s["logits"] = (normal(t, e) + normal(e, std=0.5)).to(_DT[case["logits"]])
        # padding: the last tokens of a batch's sequences
        s["mask"] = integers(0, 4, t) > 0 if case["masked"] else None
        if case["back"]:
            s["d_weights"] = normal(t, case["top_k"], std=1e-3)
            s["d_balance"] = normal(std=1e-3, mean=1e-2)
        return s
    h, v = case["hidden"], case["vocab"]
    s["weight"] = normal(v, h, std=2.0 / math.sqrt(h), dtype=torch.bfloat16)
    labels = integers(0, v, t)
    s["x"] = (normal(t, h) + s["weight"][labels].float()).to(torch.bfloat16)
    hidden = torch.rand((t,), generator=g, device=dev) < case["ignored"]
    s["labels"] = torch.where(hidden, IGNORE, labels)
    if case["back"]:
        # the mean over the tokens that count
        s["d_loss"] = torch.full((t,), 1.0 / t, device=dev)
        s["d_lse"] = normal(t, std=1e-3 / t) if case["z_loss"] else None
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    if own:
        return _run_own(s)
    if s["op"] == "rotate":
        return _plain_rotate_backward(s) if s["back"] else _plain_rotate(s)
    return _plain_route(s) if s["op"] == "route" else _plain_loss(s)


def _run_own(s):
    import mxfp8_block_scaled_mx_gb300 as mx
    if s["op"] == "rotate":
        how = dict(interleaved=s["interleaved"], scale=s["scale"], eps=EPS)
        args = (s["q"], s["k"], s["w_q"], s["w_k"], s["positions"], s["frequencies"])
        if s["back"]:
            d = mx.norm_rotate_backward(s["d_q"], s["d_k"], *args, **how)
            return {"q": d.q, "k": d.k, "w_q": d.w_q, "w_k": d.w_k}
        q, k = mx.norm_rotate(*args, **how)
        return {"q": q, "k": k}
    if s["op"] == "route":
        r = mx.route(s["logits"], s["top_k"], renormalize=s["renormalize"], mask=s["mask"])
        out = {"ids": r.ids, "weights": r.weights, "counts": r.counts, "offsets": r.offsets,
               "order": r.order, "balance": r.balance}
        if s["back"]:
            out["d_logits"] = mx.route_backward(s["d_weights"], s["d_balance"], s["logits"], r,
                                                renormalize=s["renormalize"], mask=s["mask"])
        return out
    loss, lse = mx.linear_cross_entropy(s["x"], s["weight"], s["labels"], ignore_index=IGNORE)
    out = {"loss": loss, "lse": lse}
    if s["back"]:
        out["x"], out["weight"] = mx.linear_cross_entropy_backward(
            s["d_loss"], s["d_lse"], s["x"], s["weight"], s["labels"], lse, ignore_index=IGNORE)
    return out


def _turned(x1, x2, c, sn):
    return x1 * c - x2 * sn, x1 * sn + x2 * c


def _rotate(x, s, sign):
    """The first `rotary` channels of [tokens, heads, dim], in pairs, by each token's angles."""
    r = s["rotary"]
    angle = s["positions"].double()[:, None] * s["frequencies"]
    c = (angle.cos() * s["scale"]).float()[:, None]
    sn = (angle.sin() * (sign * s["scale"])).float()[:, None]
    if s["interleaved"]:
        turned = torch.stack(_turned(x[..., 0:r:2], x[..., 1:r:2], c, sn), -1).flatten(-2)
    else:
        turned = torch.cat(_turned(x[..., :r // 2], x[..., r // 2:r], c, sn), -1)
    return torch.cat([turned, x[..., r:]], -1)


def _plain_rotate(s):
    def one(x, w):
        x = x.float()
        n = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()
        return _rotate(n, s, 1.0).to(s["q"].dtype)

    return {"q": one(s["q"], s["w_q"]), "k": one(s["k"], s["w_k"])}


def _plain_rotate_backward(s):
    def one(dy, x, w):
        x, w = x.float(), w.float()
        dn = _rotate(dy.float(), s, -1.0)
        rho = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
        wd = w * dn
        dx = rho * wd - x * rho ** 3 * (wd * x).mean(-1, keepdim=True)
        return dx.to(s["q"].dtype), (dn * x * rho).sum((0, 1))

    dq, dwq = one(s["d_q"], s["q"], s["w_q"])
    dk, dwk = one(s["d_k"], s["k"], s["w_k"])
    return {"q": dq, "k": dk, "w_q": dwq, "w_k": dwk}


def _plain_route(s):
    t, e, k = s["tokens"], s["experts"], s["top_k"]
    z = s["logits"].float()
    p = torch.exp(z - z.amax(1, keepdim=True))
    p = p / p.sum(1, keepdim=True)
    ids = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :k]
    picked = p.gather(1, ids)
    total = picked.sum(1, keepdim=True) if s["renormalize"] else torch.ones_like(picked[:, :1])
    weights = picked / total
    flat = ids.flatten()
    order = torch.sort(flat, stable=True).indices
    load = (flat[:, None] == torch.arange(e, device=z.device)).sum(0)
    offsets = torch.cat([load.new_zeros(1), load.cumsum(0)])
    valid = torch.ones_like(z[:, 0]) if s["mask"] is None else s["mask"].float()
    n = valid.sum()
    chosen = torch.zeros_like(z).scatter(1, ids, 1.0)
    counts = (chosen * valid[:, None]).sum(0)
    share = counts * (e / (n * k).clamp(min=1))
    per = valid[:, None] / n.clamp(min=1)
    balance = (share * (p * per).sum(0)).sum()
    out = {"ids": ids.int(), "weights": weights, "counts": counts.int(), "offsets": offsets.int(),
           "order": order.int(), "balance": balance}
    if s["back"]:
        dw = s["d_weights"]
        dw = (dw - (dw * weights).sum(1, keepdim=True)) / total if s["renormalize"] else dw
        dp = (s["d_balance"] * share * per).scatter_add(1, ids, dw)
        out["d_logits"] = (p * (dp - (p * dp).sum(1, keepdim=True))).to(s["logits"].dtype)
    return out


def _plain_loss(s):
    x, w, labels = s["x"].float(), s["weight"].float(), s["labels"]
    valid = labels != IGNORE
    at = torch.where(valid, labels, 0)[:, None]
    z = x @ w.T
    top = z.amax(1, keepdim=True)
    lse = top[:, 0] + torch.exp(z - top).sum(1).log()
    loss = torch.where(valid, lse - z.gather(1, at)[:, 0], 0.0)
    out = {"loss": loss, "lse": lse}
    if s["back"]:
        d = torch.where(valid, s["d_loss"], 0.0)
        both = d if s["d_lse"] is None else d + s["d_lse"]
        dz = z.sub_(lse[:, None]).exp_().mul_(both[:, None]).scatter_add_(1, at, -d[:, None])
        out["x"], out["weight"] = (dz @ w).to(torch.bfloat16), (dz.T @ x).to(torch.bfloat16)
    return out


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    if case["op"] == "loss" and work(case)["flops"] > 8e12:
        return None
    s = prepare(case, seed)

    def heads(name):
        x, w = s[name].double(), s["w_" + name].double()
        d, half = case["dim"], case["rotary"] // 2
        i = torch.arange(half, device=x.device)
        a, b = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + half)
        turn = torch.polar(torch.full((1, 1), s["scale"], dtype=torch.float64, device=x.device),
                           torch.outer(s["positions"].double(), s["frequencies"]))[:, None]
        norm = torch.sqrt((x * x).sum(-1, keepdim=True) / d + EPS)
        unit = x / norm
        y = (s["d_" + name].double() if case["back"] else unit * w).clone()
        turned = torch.complex(y[..., a], y[..., b]) * (turn.conj() if case["back"] else turn)
        y[..., a], y[..., b] = turned.real, turned.imag
        if not case["back"]:
            return y, None
        inner = (w * y * unit).sum(-1, keepdim=True) / d
        return (w * y - unit * inner) / norm, torch.einsum("thd,thd->d", y, unit)

    def rotate():
        (q, wq), (k, wk) = heads("q"), heads("k")
        return {"q": q, "k": k, "w_q": wq, "w_k": wk} if case["back"] else {"q": q, "k": k}

    def route():
        z, k, e = s["logits"].double(), case["top_k"], case["experts"]
        p = torch.exp(z - torch.log(torch.exp(z).sum(1))[:, None])
        ids = torch.argsort(-z, dim=1, stable=True)[:, :k]
        mine = torch.stack([torch.zeros_like(z[:, 0]) + p[torch.arange(len(z), device=z.device), ids[:, j]]
                            for j in range(k)], 1)
        scale = mine.sum(1) if case["renormalize"] else torch.ones_like(mine[:, 0])
        weights = mine / scale[:, None]
        rows = torch.arange(len(z), device=z.device) if s["mask"] is None else s["mask"].nonzero()[:, 0]
        n = max(1, len(rows))
        counts = torch.bincount(ids[rows].flatten(), minlength=e)
        load = torch.bincount(ids.flatten(), minlength=e).tolist()
        offsets = torch.tensor([sum(load[:j]) for j in range(e + 1)], device=z.device)
        key = ids.flatten() * ids.numel() + torch.arange(ids.numel(), device=z.device)
        share = counts.double() * e / (n * k)
        out = {"ids": ids.int(), "weights": weights, "counts": counts.int(), "offsets": offsets.int(),
               "order": torch.argsort(key).int(), "balance": (p[rows].sum(0) / n * share).sum()}
        if case["back"]:
            # d p_j / d z_i = p_j ([i = j] - p_i), term by term of the chosen ones
            dz = torch.zeros_like(z)
            dz[rows] = s["d_balance"].double() / n * p[rows] * (share - (p[rows] @ share)[:, None])
            dw = s["d_weights"].double()
            if case["renormalize"]:  # the weights are a softmax of the chosen logits alone
                here = weights * (dw - torch.einsum("tk,tk->t", dw, weights)[:, None])
                rest = 0.0
            else:
                here = weights * dw
                rest = here.sum(1)[:, None] * p
            out["d_logits"] = dz - rest + torch.zeros_like(z).scatter(1, ids, here)
        return out

    def loss():
        x, w, labels = s["x"].double(), s["weight"].double(), s["labels"]
        z = x @ w.T
        lse = torch.logsumexp(z, 1)
        rows = (labels != IGNORE).nonzero()[:, 0]
        value = torch.zeros_like(lse)
        value[rows] = lse[rows] - z[rows, labels[rows]]
        out = {"loss": value, "lse": lse}
        if case["back"]:
            d = torch.zeros_like(lse)
            d[rows] = s["d_loss"].double()[rows]
            z = torch.exp(z - lse[:, None])
            z *= (d if s["d_lse"] is None else d + s["d_lse"].double())[:, None]
            z[rows, labels[rows]] -= d[rows]
            out["x"], out["weight"] = z @ w, z.T @ x
        return out

    return {"rotate": rotate, "route": route, "loss": loss}[case["op"]]()
