"""Cases, plain forms and exact forms of the operators around the MX products.

Three operators, as a mixture-of-experts block uses them:

* `norm_residual`: the post-norm of a block's output, its gate, the scaled
  residual and the next block's pre-norm, in one pass;
* `norm_residual_backward`: its gradients;
* `moe_few_tokens`: a whole mixture-of-experts layer (router, top-k, gated
  feed-forward of the chosen experts, weighted sum) for 1 to 64 tokens, with
  the expert weights in MX formats.

`run` computes them in plain torch operations in 32 bits where `own` is
false, and with the framework's entry points where it is true.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
_SIZE = {"bf16": 2, "fp32": 4}
# Bits of storage per weight element, and the spread of its codes: the block
# scale brings a block's largest value near the format's largest.
_BITS = {"e4m3": 8, "e5m2": 8, "e2m1_packed": 4}
_SPREAD = {"e4m3": 128.0, "e5m2": 16384.0, "e2m1_packed": 2.2}
_SCALE = {"e4m3": -13, "e5m2": -20, "e2m1_packed": -7}
_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


# ------------------------------------------------------------------ cases

def listed():
    moe = dict(op="moe", renormalize=True, router="bf16")
    fwd = dict(op="norm", post=True, gates=0, alpha=1.0, c="bf16", s="bf16", w="bf16")
    bwd = dict(op="norm_backward", post=True, gates=0, alpha=1.0, c="bf16", s="bf16", w="bf16")
    return [
        # one token of a model with many small experts: latency counts
        dict(moe, name="moe_1x2048_128e", tokens=1, hidden=2048, inter=768, experts=128, top_k=8,
             fmt="e4m3"),
        # one token, wide experts with 4-bit weights
        dict(moe, name="moe_1x7168_fp4", tokens=1, hidden=7168, inter=2048, experts=32, top_k=8,
             fmt="e2m1_packed"),
        # a small batch over the 64 experts of the mixture-of-experts benchmark
        dict(moe, name="moe_16x7168_64e", tokens=16, hidden=7168, inter=2048, experts=64, top_k=8,
             fmt="e4m3"),
        # the largest batch: every expert is active
        dict(moe, name="moe_64x4096_64e", tokens=64, hidden=4096, inter=1536, experts=64, top_k=6,
             fmt="e4m3", renormalize=False, router="fp32"),
        # odd everything: partial blocks along both contractions, partial row tiles
        dict(moe, name="moe_13x1360_20e", tokens=13, hidden=1360, inter=720, experts=20, top_k=3,
             fmt="e5m2"),
        # decoding: one row through both norms and a per-channel gate
        dict(fwd, name="norm_1x7168", rows=1, cols=7168, gates=1),
        # a training step's rows, both norms
        dict(fwd, name="norm_16384x7168", rows=16384, cols=7168),
        # four sequences with a gate each, residual kept in FP32 and scaled
        dict(fwd, name="norm_8192x2048_gated", rows=8192, cols=2048, gates=4, alpha=0.875,
             s="fp32", w="fp32"),
        # odd rows of odd length (no 16-byte rows), pre-norm only, FP32
        dict(fwd, name="norm_777x1111", rows=777, cols=1111, post=False, c="fp32", s="fp32",
             w="fp32"),
        # the gradients of the two training cases, and of a small odd one
        dict(bwd, name="norm_back_16384x7168", rows=16384, cols=7168),
        dict(bwd, name="norm_back_8192x2048_gated", rows=8192, cols=2048, gates=4, alpha=0.875,
             s="fp32", w="fp32"),
        dict(bwd, name="norm_back_333x1111", rows=333, cols=1111, gates=1, s="fp32", w="fp32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.5:
        fmt = rng.choice(["e4m3", "e4m3", "e2m1_packed", "e5m2"])
        # contraction lengths: whole 16-element runs, whole 128 in packed storage
        step = 128 if fmt == "e2m1_packed" else 16
        while True:
            experts = _log(rng, 4, 128)
            c = dict(op="moe", tokens=_log(rng, 1, 64), hidden=step * _log(rng, 512 // step, 7168 // step),
                     inter=step * _log(rng, 256 // step, 2048 // step), experts=experts,
                     top_k=rng.randint(1, min(8, experts)), fmt=fmt,
                     renormalize=rng.random() < 0.5, router=rng.choice(["bf16", "fp32"]))
            if 3072 in (c["hidden"], c["inter"]):
                continue
            if experts * c["hidden"] * c["inter"] <= 48 * 7168 * 2048:
                return c
    while True:
        rows, cols = _log(rng, 1, 16384), _log(rng, 64, 8192)
        if rng.random() < 0.6:
            cols = max(64, cols // 8 * 8)  # most models' rows are whole 16-byte runs
        gates = rng.choice([0, 0, 1, rng.randint(2, 8), rows])
        rows = max(1, rows // max(1, gates)) * max(1, gates)
        # the stream is at least as wide as the blocks' type
        c, stream = rng.choice([("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "fp32")])
        size = rows * cols * (_SIZE[c] + _SIZE[stream] + (_SIZE["fp32"] if gates == rows else 0))
        if size <= 16384 * 7168 * 4 and 3072 not in (rows, cols):
            return dict(op=rng.choice(["norm", "norm_backward"]), rows=rows, cols=cols, gates=gates,
                        post=rng.random() < 0.7, alpha=rng.choice([1.0, 0.875, 0.25]), c=c, s=stream,
                        w=rng.choice(["bf16", "fp32"]))


def _active(case):
    """Distinct experts that the tokens choose, on average, of equally likely ones."""
    return case["experts"] * (1 - (1 - case["top_k"] / case["experts"]) ** case["tokens"])


def work(case):
    if case["op"] == "moe":
        t, h, i, e, k = (case[n] for n in ("tokens", "hidden", "inter", "experts", "top_k"))
        weights = 3 * h * i * (_BITS[case["fmt"]] / 8 + 1 / 32)
        return {"bytes": int(_active(case) * weights + e * h * _SIZE[case["router"]] + 4 * t * h
                             + 8 * t * k),
                "flops": int(2 * t * e * h + 6 * t * k * h * i)}
    n, h = case["rows"] * case["cols"], case["cols"]
    sides = 2 if case["op"] == "norm" else 3
    weights = (1 + case["post"] + case["gates"]) * h * _SIZE[case["w"]]
    grads = (1 + case["post"] + case["gates"]) * h * 4 if case["op"] == "norm_backward" else 0
    return {"bytes": sides * n * (_SIZE[case["c"]] + _SIZE[case["s"]]) + weights + grads,
            "flops": (14 if case["op"] == "norm" else 30) * n}


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def normal(*shape, std=1.0, mean=0.0, dtype=torch.float32):
        return (torch.randn(shape, generator=g, device=dev) * std + mean).to(dtype)

    def weight(experts, rows, k, fmt):
        """MX weights of one projection: codes [experts, rows, k] (K contiguous) and,
        per expert, block scales in 512-byte tiles of 128 rows x 4 blocks."""
        codes = torch.empty((experts, rows, k * _BITS[fmt] // 8), dtype=torch.uint8, device=dev)
        for e in range(experts):
            v = torch.randn((rows, k), generator=g, device=dev) * _SPREAD[fmt]
            if fmt == "e4m3":
                codes[e] = v.clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            elif fmt == "e5m2":
                codes[e] = v.clamp_(-57344, 57344).to(torch.float8_e5m2).view(torch.uint8)
            else:
                edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=dev)
                c = torch.bucketize(v.abs(), edges, out_int32=True).to(torch.uint8)
                c |= (v < 0).to(torch.uint8) << 3
                codes[e] = c[:, 0::2] | (c[:, 1::2] << 4)
        tiles = -(-rows // 128) * -(-k // 128)
        scales = torch.randint(127 + _SCALE[fmt] - 1, 127 + _SCALE[fmt] + 2, (experts, tiles * 512),
                               generator=g, device=dev, dtype=torch.int32)
        return codes, scales.to(torch.uint8)

    s = dict(case)
    if case["op"] == "moe":
        t, h, i, e = (case[n] for n in ("tokens", "hidden", "inter", "experts"))
        s["x"] = normal(t, h, dtype=torch.bfloat16)
        s["w_router"] = normal(e, h, std=0.02, dtype=_DT[case["router"]])
        s["gate"], s["gate_scales"] = weight(e, i, h, case["fmt"])
        s["up"], s["up_scales"] = weight(e, i, h, case["fmt"])
        s["down"], s["down_scales"] = weight(e, h, i, case["fmt"])
        return s
    rows, cols = case["rows"], case["cols"]
    c, r, w = _DT[case["c"]], _DT[case["s"]], _DT[case["w"]]
    s["block"] = normal(rows, cols, std=0.5, dtype=c)
    s["residual"] = normal(rows, cols, std=2.0, dtype=r)
    s["w_pre"] = normal(cols, std=0.1, mean=1.0, dtype=w)
    s["w_post"] = normal(cols, std=0.1, mean=1.0, dtype=w) if case["post"] else None
    shape = (cols,) if case["gates"] == 1 else (case["gates"], cols)
    s["gate"] = normal(*shape, std=0.3, mean=0.5, dtype=w) if case["gates"] else None
    if case["op"] == "norm_backward":
        s["d_residual"] = normal(rows, cols, std=1e-3, dtype=r)
        s["d_y"] = normal(rows, cols, std=1e-3, dtype=c)
    return s


# ------------------------------------------------------------------ one pass

EPS = 1e-6


def run(s):
    if own:
        return _run_own(s)
    if s["op"] == "moe":
        return _plain_moe(s)
    return _plain_norm(s) if s["op"] == "norm" else _plain_norm_backward(s)


def _run_own(s):
    import mxfp8_block_scaled_mx_gb300 as mx
    if s["op"] == "moe":
        y, ids, weights = mx.moe_few_tokens(
            s["x"], s["w_router"], mx.MxTensor(s["gate"], s["gate_scales"], s["fmt"]),
            mx.MxTensor(s["up"], s["up_scales"], s["fmt"]),
            mx.MxTensor(s["down"], s["down_scales"], s["fmt"]), s["top_k"],
            renormalize=s["renormalize"], return_routing=True)
        return {"y": y, "ids": ids, "weights": weights}
    if s["op"] == "norm":
        residual, y = mx.norm_residual(s["block"], s["residual"], s["w_pre"], w_post=s["w_post"],
                                       gate=s["gate"], alpha=s["alpha"], eps=EPS)
        return {"residual": residual, "y": y}
    d = mx.norm_residual_backward(s["d_residual"], s["d_y"], s["block"], s["residual"], s["w_pre"],
                                  w_post=s["w_post"], gate=s["gate"], alpha=s["alpha"], eps=EPS)
    return {"block": d.block, "residual": d.residual, "w_pre": d.w_pre, "w_post": d.w_post,
            "gate": d.gate}


def _gate_rows(s):
    """The gate of every row, FP32 (1 without one); row t of T takes gate t * G // T."""
    gate = s["gate"]
    if gate is None:
        return 1.0
    gate = gate.float().reshape(-1, s["cols"])
    return gate.repeat_interleave(s["rows"] // gate.shape[0], 0)


def _plain_norm(s):
    b = s["block"].float()
    if s["w_post"] is not None:
        b = b * torch.rsqrt(b.square().mean(1, keepdim=True) + EPS) * s["w_post"].float()
    stream = (s["alpha"] * s["residual"].float() + _gate_rows(s) * b).to(s["residual"].dtype)
    r = stream.float()  # the norm reads the stream as the next block will
    y = r * torch.rsqrt(r.square().mean(1, keepdim=True) + EPS) * s["w_pre"].float()
    return {"residual": stream, "y": y.to(s["block"].dtype)}


def _plain_norm_backward(s):
    b, r, dy = s["block"].float(), s["residual"].float(), s["d_y"].float()
    rho = torch.rsqrt(r.square().mean(1, keepdim=True) + EPS)
    wdy = dy * s["w_pre"].float()
    d = s["d_residual"].float() + rho * wdy - r * rho ** 3 * (wdy * r).mean(1, keepdim=True)
    d_w_pre = (dy * r * rho).sum(0)
    u = _gate_rows(s) * d
    d_w_post = None
    if s["w_post"] is None:
        n, d_b = b, u
    else:
        sigma = torch.rsqrt(b.square().mean(1, keepdim=True) + EPS)
        w = s["w_post"].float()
        wu = w * u
        d_b = sigma * wu - b * sigma ** 3 * (wu * b).mean(1, keepdim=True)
        d_w_post = (u * b * sigma).sum(0)
        n = b * sigma * w
    d_gate = None
    if s["gate"] is not None:
        shape = s["gate"].shape
        d_gate = (d * n).reshape(shape.numel() // s["cols"], -1, s["cols"]).sum(1).reshape(shape)
    return {"block": d_b.to(s["block"].dtype), "residual": (s["alpha"] * d).to(s["residual"].dtype),
            "w_pre": d_w_pre, "w_post": d_w_post, "gate": d_gate}


def _values(codes, scales, rows, k, fmt):
    """FP32 values of MX weights: codes [n, rows, k], scale tiles [n, bytes]."""
    if fmt == "e4m3":
        v = codes.view(torch.float8_e4m3fn).float()
    elif fmt == "e5m2":
        v = codes.view(torch.float8_e5m2).float()
    else:
        table = torch.tensor(_E2M1 + [-m for m in _E2M1], device=codes.device)
        v = table[torch.stack([codes & 15, codes >> 4], -1).flatten(2).int()]
    # a tile holds block j of row r at byte (r % 32) * 16 + (r // 32) * 4 + j
    tiles = scales.view(codes.shape[0], -(-rows // 128), -(-k // 128), 32, 4, 4)
    byte = tiles.permute(0, 1, 4, 3, 2, 5).flatten(4, 5).flatten(1, 3)[:, :rows]
    bits = byte.int() << 23  # E8M0: 2^(byte - 127)
    scale = torch.where(byte == 0, 0x00400000, bits).view(torch.float32)
    return v * scale.repeat_interleave(32, 2)[:, :, :k]


def _plain_moe(s):
    x = s["x"].float()
    z = x @ s["w_router"].float().T
    p = torch.softmax(z, 1)
    ids = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :s["top_k"]]
    weights = p.gather(1, ids)
    if s["renormalize"]:
        weights = weights / weights.sum(1, keepdim=True)
    active = torch.unique(ids)
    gate = _values(s["gate"][active], s["gate_scales"][active], s["inter"], s["hidden"], s["fmt"])
    a = torch.einsum("th,eih->eti", x, gate)
    del gate
    up = _values(s["up"][active], s["up_scales"][active], s["inter"], s["hidden"], s["fmt"])
    h = a * torch.sigmoid(a) * torch.einsum("th,eih->eti", x, up)
    del up
    # the weight of every token for every active expert, 0 where it was not chosen
    share = torch.zeros_like(p).scatter(1, ids, weights)[:, active].T
    h = torch.where(share.unsqueeze(2) > 0, h * share.unsqueeze(2), 0.0)
    down = _values(s["down"][active], s["down_scales"][active], s["hidden"], s["inter"], s["fmt"])
    y = torch.einsum("eti,ehi->eth", h, down).sum(0)
    return {"y": y.to(torch.bfloat16), "ids": ids.int(), "weights": weights}


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    s = prepare(case, seed)

    def norm():
        rows, cols, alpha = s["rows"], s["cols"], s["alpha"]
        back = s["op"] == "norm_backward"
        many = max(1, s["gates"])
        per = rows // many
        gates = None if s["gate"] is None else s["gate"].double().reshape(many, cols)
        w_pre = s["w_pre"].double()
        w_post = None if s["w_post"] is None else s["w_post"].double()
        d_pre, d_post = torch.zeros_like(w_pre), torch.zeros_like(w_pre)
        d_gate = torch.zeros((many, cols), dtype=torch.float64, device=w_pre.device)
        first = torch.empty((rows, cols), dtype=torch.float64, device=w_pre.device)
        second = torch.empty_like(first)
        chunk = max(1, (1 << 25) // cols)
        for lo in range(0, rows, chunk):
            hi = min(rows, lo + chunk)
            which = torch.arange(lo, hi, device=w_pre.device) // per
            b, r = s["block"][lo:hi].double(), s["residual"][lo:hi].double()
            inv_b = 1 / torch.sqrt((b * b).sum(1) / cols + EPS)[:, None]
            n = b if w_post is None else b * inv_b * w_post
            gate = torch.ones_like(n) if gates is None else gates[which]
            if not back:
                stream = alpha * r + gate * n
                first[lo:hi] = stream
                stored = stream.to(s["residual"].dtype).double()
                second[lo:hi] = stored / torch.sqrt((stored * stored).sum(1) / cols + EPS)[:, None] * w_pre
                continue
            dy = s["d_y"][lo:hi].double()
            inv_r = 1 / torch.sqrt((r * r).sum(1) / cols + EPS)[:, None]
            unit = r * inv_r
            t = dy * w_pre
            d = s["d_residual"][lo:hi].double() + inv_r * (t - unit * ((t * unit).sum(1) / cols)[:, None])
            d_pre += (dy * unit).sum(0)
            u = d * gate
            if w_post is None:
                first[lo:hi] = u
            else:
                unit_b = b * inv_b
                t = u * w_post
                first[lo:hi] = inv_b * (t - unit_b * ((t * unit_b).sum(1) / cols)[:, None])
                d_post += (u * unit_b).sum(0)
            second[lo:hi] = alpha * d
            d_gate.index_add_(0, which, d * n)
        if not back:
            return {"residual": first, "y": second}
        return {"block": first, "residual": second, "w_pre": d_pre,
                "w_post": None if w_post is None else d_post,
                "gate": None if gates is None else d_gate.reshape(s["gate"].shape)}

    def code_table(fmt):
        """Values of the 256 (E2M1: 16) codes, from the formats' definition."""
        ebits, mbits, bias = {"e4m3": (4, 3, 7), "e5m2": (5, 2, 15), "e2m1_packed": (2, 1, 1)}[fmt]
        out = []
        for code in range(1 << (1 + ebits + mbits)):
            e, m = (code >> mbits) & ((1 << ebits) - 1), code & ((1 << mbits) - 1)
            v = math.ldexp(m, 1 - bias - mbits) if e == 0 else math.ldexp((1 << mbits) + m, e - bias - mbits)
            out.append(-v if code >> (ebits + mbits) else v)
        return out

    def weight(name, e, rows, k, table):
        codes = s[name][e].long()
        if s["fmt"] == "e2m1_packed":
            wide = torch.empty((rows, k), dtype=torch.long, device=codes.device)
            wide[:, 0::2], wide[:, 1::2] = codes % 16, codes // 16
            codes = wide
        r = torch.arange(rows, device=codes.device)[:, None]
        j = torch.arange(-(-k // 32), device=codes.device)[None, :]
        at = ((r // 128) * -(-k // 128) + j // 4) * 512 + (r % 32) * 16 + (r % 128 // 32) * 4 + j % 4
        power = s[name + "_scales"][e].double()[at] - 127
        return table[codes] * torch.pow(2.0, power).repeat_interleave(32, 1)[:, :k]

    def moe():
        x = s["x"].double()
        t, k = s["tokens"], s["top_k"]
        z = x @ s["w_router"].double().T
        p = torch.exp(z - z.max(1, keepdim=True).values)
        p = p / p.sum(1, keepdim=True)
        ids = torch.argsort(z, dim=1, descending=True, stable=True)[:, :k]
        weights = torch.stack([p[r, ids[r]] for r in range(t)])
        if s["renormalize"]:
            weights = weights / weights.sum(1, keepdim=True)
        table = torch.tensor(code_table(s["fmt"]), dtype=torch.float64, device=x.device)
        y = torch.zeros_like(x)
        for e in sorted(set(ids.flatten().tolist())):
            rows, place = (ids == e).nonzero(as_tuple=True)
            xe = x[rows]
            a = xe @ weight("gate", e, s["inter"], s["hidden"], table).T
            a = a / (1 + torch.exp(-a)) * (xe @ weight("up", e, s["inter"], s["hidden"], table).T)
            a = a @ weight("down", e, s["hidden"], s["inter"], table).T
            y[rows] += weights[rows, place][:, None] * a
        return {"y": y, "ids": None, "weights": weights}

    return moe() if case["op"] == "moe" else norm()
