"""The operators between the products together, as a training step runs them, and
their calls on given streams, side by side, captured and from several threads."""
import threading

import pytest
import torch

from mxcheck import ensure_built
from test_gpu_block_calls import SLEEP, segment_stream

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def mx():
    ensure_built()
    import mxfp8_block_scaled_mx_gb300 as mx
    return mx


def randn(*shape, seed, scale=1.0, dtype=BF16):
    g = torch.Generator("cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


class Calls:
    """Inputs of every operator, two sets; each call returns a list of its outputs."""

    names = ["rotate", "rotate_back", "route_few", "route", "route_many", "route_back", "loss", "loss_back",
             "loss_few", "loss_few_back"]

    def __init__(self, mx):
        self.mx = mx
        self.rows = [randn(600, 10, 64, seed=s) for s in (1, 2)]
        self.grad = randn(600, 8, 64, seed=3)
        self.w = [randn(64, seed=s, scale=0.1) + 1 for s in (4, 5)]
        self.pos = torch.arange(600, device="cuda")
        self.freq = mx.rotary_frequencies(64)
        self.z = {n: [randn(n, 48, seed=s, dtype=FP32) for s in (6, 7)] for n in (40, 3000, 17000)}
        self.routing = [mx.route(z, 4) for z in self.z[3000]]
        self.dw = randn(3000, 4, seed=8, dtype=FP32)
        self.x = {n: [randn(n, 192, seed=s) for s in (9, 10)] for n in (20, 700)}
        self.v = randn(3000, 192, seed=11, scale=0.1)
        self.labels = {n: torch.arange(n, device="cuda") * 7 % 3000 for n in (20, 700)}
        self.lse = {n: [mx.linear_cross_entropy(x, self.v, self.labels[n])[1] for x in self.x[n]] for n in (20, 700)}
        self.d = {n: torch.full((n,), 1.0 / n, device="cuda") for n in (20, 700)}
        torch.cuda.synchronize()

    def call(self, name, which=0, stream=None):
        mx = self.mx
        heads = self.rows[which]
        args = (heads[:, :6], heads[:, 6:8], *self.w, self.pos, self.freq)
        if name == "rotate":
            return list(mx.norm_rotate(*args, stream=stream))
        if name == "rotate_back":
            return list(vars(mx.norm_rotate_backward(self.grad[:, :6], self.grad[:, 6:], *args, stream=stream)).values())
        if name == "route_back":
            return [mx.route_backward(self.dw, None, self.z[3000][which], self.routing[which], stream=stream)]
        if name.startswith("route"):
            n = {"route_few": 40, "route": 3000, "route_many": 17000}[name]
            return list(vars(mx.route(self.z[n][which], 4, stream=stream)).values())
        n = 20 if "few" in name else 700
        if name.endswith("back"):
            return list(mx.linear_cross_entropy_backward(self.d[n], None, self.x[n][which], self.v, self.labels[n],
                                                         self.lse[n][which], stream=stream))
        return list(mx.linear_cross_entropy(self.x[n][which], self.v, self.labels[n], stream=stream))


@pytest.fixture(scope="module")
def calls(mx):
    return Calls(mx)


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("name", Calls.names)
def test_a_call_on_a_given_stream(mx, calls, name):
    """Outputs from that stream's memory; beside a call on the current stream that is
    still queued, neither takes the other's memory."""
    ref = [calls.call(name, i) for i in (0, 1)]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for t in calls.call(name, 0, s):
        assert segment_stream(t) == s.cuda_stream
    for first, second in ((None, s), (s, None)):
        torch.cuda.synchronize()
        with torch.cuda.stream(first or torch.cuda.current_stream()):
            torch.cuda._sleep(SLEEP)
        got = [calls.call(name, 0, first), calls.call(name, 1, second)]
        torch.cuda.synchronize()
        assert same(ref[0], got[0]) and same(ref[1], got[1])
    # outputs freed on the current stream while copies of them are queued
    outs = calls.call(name, 0, s)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda._sleep(SLEEP)
    kept = [t.clone() for t in outs]
    del outs
    for _ in range(3):
        calls.call(name, 1, s)
    torch.cuda.synchronize()
    assert same(ref[0], kept) and mx.device_status() == 0


@pytest.mark.parametrize("name", Calls.names)
def test_captured_and_replayed(mx, calls, name):
    ref = calls.call(name)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        got = calls.call(name)
        again = calls.call(name)
    for _ in range(2):
        for t in got + again:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert same(ref, got) and same(ref, again)
    # another call beside the replay, and the graph once more
    other = calls.call(name, 1)
    graph.replay()
    torch.cuda.synchronize()
    assert same(ref, got) and same(other, calls.call(name, 1)) and mx.device_status() == 0


def test_from_several_threads(mx, calls):
    ref = {n: [calls.call(n, i) for i in (0, 1)] for n in Calls.names}
    torch.cuda.synchronize()
    bad = []

    def work(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(3):
                for n in Calls.names:
                    got = calls.call(n, i % 2)
                    s.synchronize()
                    if not same(ref[n][i % 2], got):
                        bad.append(n)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad and mx.device_status() == 0


def test_a_backward_pass_in_a_graph(mx):
    """Forward and backward of all three captured, replayed with new inputs in the
    captured buffers: the gradients of an eager pass.  Warmed up and captured on one
    stream, with no eager graph of the same leaves alive."""
    heads = randn(300, 4, 32, seed=1).requires_grad_()
    w = (randn(32, seed=2, scale=0.1) + 1).requires_grad_()
    z = randn(300, 16, seed=3, dtype=FP32).requires_grad_()
    x = randn(300, 64, seed=4).requires_grad_()
    v = randn(900, 64, seed=5, scale=0.2).requires_grad_()
    leaves = [heads, w, z, x, v]
    pos, freq = torch.arange(300, device="cuda"), mx.rotary_frequencies(32)
    labels = torch.arange(300, device="cuda") * 3

    def step():
        q, k = mx.norm_rotate(heads[:, :3], heads[:, 3:], w, w, pos, freq)
        r = mx.route(z, 2)
        loss, lse = mx.linear_cross_entropy(x, v, labels)
        total = (q.float().mean() + k.float().square().mean() + (r.weights ** 2).mean() + r.balance + loss.mean()
                 + 1e-3 * lse.square().mean())
        return torch.autograd.grad(total, leaves)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        got = step()
    for seed in (10, 20):
        with torch.no_grad():
            for i, t in enumerate(leaves):
                t.copy_(randn(*t.shape, seed=seed + i, scale=0.3, dtype=t.dtype))
        graph.replay()
        torch.cuda.synchronize()
        kept = [g.clone() for g in got]
        assert same(kept, step())
    assert mx.device_status() == 0


def test_a_training_step(mx):
    """A block of a mixture-of-experts model and its loss: heads of a product normed
    and rotated, attention, the router with its balance loss, experts mixed by its
    weights, the loss over the vocabulary.  Gradients of all weights against the same
    step in 64 bits with the winners of the first; what lies between the operators
    runs in FP32, heads and the last hidden rows pass through bf16: rounded by 2^-8
    each, together within 2^-5 of each gradient's norm."""
    torch.manual_seed(0)
    T, H, heads, dim, experts, k, vocab = 96, 64, 4, 16, 8, 2, 500
    p = {n: (torch.randn(s, device="cuda", dtype=torch.float64) * c) for n, s, c in (
        ("emb", (vocab, H), 1.0), ("qkv", (H, 3 * heads * dim), 0.15), ("out", (heads * dim, H), 0.2),
        ("router", (H, experts), 0.3), ("up", (experts, H, H), 0.15), ("head", (vocab, H), 0.2))}
    p["w_q"], p["w_k"] = (1 + 0.1 * torch.randn(dim, device="cuda", dtype=torch.float64) for _ in range(2))
    tokens, labels = torch.randint(0, vocab, (2, T), device="cuda")
    labels[::7] = -100
    mask = labels != -100
    pos, freq = torch.arange(T, device="cuda") + 1000, mx.rotary_frequencies(8)
    causal = torch.full((T, T), float("-inf"), device="cuda").triu(1)
    winners = []

    def turned(x, w):
        n = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w
        a = pos[:, None].double() * freq
        c, s = a.cos()[:, None], a.sin()[:, None]
        u, v = n[..., :4], n[..., 4:8]
        return torch.cat([u * c - v * s, u * s + v * c, n[..., 8:]], -1)

    def step(p, own):
        f = FP32 if own else torch.float64
        h = p["emb"][tokens]
        q, kk, v = (h @ p["qkv"]).view(T, 3, heads, dim).unbind(1)
        if own:
            q, kk = (t.float() for t in mx.norm_rotate(q.bfloat16(), kk.bfloat16(), p["w_q"], p["w_k"], pos, freq))
        else:
            q, kk = turned(q, p["w_q"]), turned(kk, p["w_k"])
        s = torch.einsum("thd,shd->hts", q, kk) / dim ** 0.5 + causal.to(f)
        h = h + torch.einsum("hts,shd->thd", torch.softmax(s, -1), v).reshape(T, -1) @ p["out"]
        z = h @ p["router"]
        if own:
            r = mx.route(z, k, mask=mask)
            winners.append(r.ids.long())
            ids, weights, balance = winners[0], r.weights, r.balance
        else:
            ids = winners[0]
            pr = torch.softmax(z, 1)
            weights = pr.gather(1, ids)
            weights = weights / weights.sum(1, keepdim=True)
            n = mask.sum()
            counts = torch.bincount(ids[mask].flatten(), minlength=experts)
            balance = experts * (counts / (n * k) * pr[mask].mean(0)).sum()
        y = torch.einsum("tk,tkh->th", weights, torch.einsum("th,tkhi->tki", h, p["up"][ids]))
        h = h + y
        if own:
            loss, lse = mx.linear_cross_entropy(h.bfloat16(), p["head"].bfloat16(), labels)
            ce = loss.sum() / mask.sum()
        else:
            lse = torch.logsumexp(h @ p["head"].T, 1)
            ce = torch.nn.functional.cross_entropy(h @ p["head"].T, labels)
        return ce + 0.1 * balance + 1e-3 * (lse ** 2).mean()

    mine = {n: t.float().requires_grad_() for n, t in p.items()}
    ref = {n: t.clone().requires_grad_() for n, t in p.items()}
    a = step(mine, True)
    b = step(ref, False)
    assert abs(a.item() - b.item()) < 2.0 ** -7 * abs(b.item())
    got = torch.autograd.grad(a, list(mine.values()))
    want = torch.autograd.grad(b, list(ref.values()))
    for n, g, r in zip(p, got, want):
        assert (g.double() - r).norm() < 2.0 ** -5 * r.norm(), n
    assert mx.device_status() == 0
