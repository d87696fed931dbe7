"""The operators in a row, as a mixture-of-experts layer runs them.

Serving: route -> dispatch -> gate and up products -> down products -> combine,
packed and padded, eager and captured in a HIP graph that is replayed with other
inputs, and two layers on two streams at once.  Training: combine's gradient ->
routing's, and dispatch's (combine without weights), against differences of the
64-bit layer.
"""
import numpy as np
import pytest
import torch

import plain64
from combine_get_dispatch_02_amd import ep

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


class Layer:
    """E experts H -> F -> H with 4-bit weights behind a sigmoid router."""

    def __init__(self, H=256, F=128, E=16, k=4, groups=4, topk_groups=2, seed=0):
        rng = np.random.default_rng(seed)
        self.H, self.F, self.E, self.k, self.groups, self.topk_groups = H, F, E, k, groups, topk_groups
        self.up = rng.integers(0, 256, (E, 2 * F, H // 2), dtype=np.uint8), rng.integers(119, 122, (E, 2 * F, H // 32), dtype=np.uint8)
        self.down = rng.integers(0, 256, (E, H, F // 2), dtype=np.uint8), rng.integers(119, 122, (E, H, F // 32), dtype=np.uint8)
        self.bias = (0.1 * rng.standard_normal(E)).astype(np.float32)
        d = lambda a: torch.from_numpy(a).to(DEV)  # noqa: E731
        self.dev = [d(a) for a in (*self.up, *self.down, self.bias)]

    def inputs(self, T, seed):
        rng = np.random.default_rng([seed, 3])
        x = torch.from_numpy(rng.standard_normal((T, self.H), dtype=np.float32)).bfloat16()
        logits = torch.from_numpy(rng.standard_normal((T, self.E), dtype=np.float32)).bfloat16()
        if T > 3:
            logits[3] = float("-inf")               # a padding token
        return x.to(DEV), logits.to(DEV)

    def run(self, x, logits, capacity=0):
        uc, us, dc, ds, bias = self.dev
        r = ep.ep_route(logits, self.k, score="sigmoid", bias=bias, num_groups=self.groups, topk_groups=self.topk_groups,
                        scale=2.5)
        idx, w = r["topk_idx"], r["topk_weights"]
        if capacity:
            d = ep.ep_dispatch_ll(x, idx, w, self.E, capacity)
            h = ep.ep_expert_linear_w4(d["recv_x"], d["recv_count"], uc, us, capacity=capacity, epilogue="silu_mul")
            y = ep.ep_expert_linear_w4(h, d["recv_count"], dc, ds, capacity=capacity)
            return ep.ep_combine(y.view(self.E * capacity, self.H), d["token_slot"], w), idx, w
        d = ep.ep_dispatch(x, idx, w, self.E, 4)
        h = ep.ep_expert_linear_w4(d["recv_x"], d["recv_expert_offset"], uc, us, epilogue="silu_mul")
        y = ep.ep_expert_linear_w4(h, d["recv_expert_offset"], dc, ds)
        return ep.ep_combine(y, d["token_row"], w), idx, w

    def plain(self, x, logits):
        """The layer in 64 bits, with a bound on what the roundings of the steps
        make of it: (out, bound)."""
        x = x.double().cpu().numpy()
        idx, w = plain64.route(logits.double().cpu().numpy(), self.k, True, self.bias, self.groups, self.topk_groups, 2, True, 2.5)
        up, down = plain64.decode_w4(*self.up), plain64.decode_w4(*self.down)
        out, bound = np.zeros_like(x), np.zeros_like(x)
        for t in range(len(x)):
            for j in range(self.k):
                e = idx[t, j]
                if e < 0:
                    continue
                h, hs = plain64.expert_linear(x[t:t + 1], [(0, 1)], up[e:e + 1], True)
                # h to bf16 (half a step, 2^-8) and its own accumulation; through the
                # down weights; y to bf16; the sum of k rows and its rounding.
                dh = 2.0 ** -8 * np.abs(h) + (self.H + 8) * 2.0 ** -23 * hs
                y, ys = plain64.expert_linear(h, [(0, 1)], down[e:e + 1], False)
                dy = dh @ np.abs(down[e]).T + 2.0 ** -8 * np.abs(y) + (self.F + 8) * 2.0 ** -23 * ys
                out[t] += w[t, j] * y[0]
                bound[t] += abs(w[t, j]) * (1.01 * dy[0] + 2.0 ** -18 * np.abs(y[0]))
        return out, idx, bound + 2.0 ** -8 * (np.abs(out) + bound)


@pytest.mark.parametrize("T", [1, 7, 60])
@pytest.mark.parametrize("padded", [False, True])
def test_layer(T, padded):
    layer = Layer()
    x, logits = layer.inputs(T, T)
    out, idx, _ = layer.run(x, logits, capacity=T if padded else 0)
    ref, ref_idx, bound = layer.plain(x, logits)
    np.testing.assert_array_equal(idx.cpu().numpy(), ref_idx)
    got = out.double().cpu().numpy()
    assert (np.abs(got - ref) <= bound).all()
    if T > 3:
        assert (got[3] == 0).all() and (ref_idx[3] == -1).all()


@pytest.mark.parametrize("capacity", [0, 24])
def test_captured_layer_replays_with_other_inputs(capacity):
    layer, T = Layer(), 40
    x, logits = layer.inputs(T, 1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        layer.run(x, logits, capacity)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, idx, w = layer.run(x, logits, capacity)
    for seed in range(2, 6):
        x2, logits2 = layer.inputs(T, seed)
        eager = layer.run(x2, logits2, capacity)    # work of the program's own between the replays
        x.copy_(x2)
        logits.copy_(logits2)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((out, idx, w), eager):
            assert torch.equal(a, b)


def test_two_layers_on_two_streams():
    layers = [Layer(seed=0), Layer(H=512, F=256, E=64, k=6, groups=8, topk_groups=4, seed=1)]
    ins = [layers[0].inputs(300, 1), layers[1].inputs(900, 2)]
    alone = [la.run(*i) for la, i in zip(layers, ins)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    for _ in range(4):
        for n in (0, 1):
            with torch.cuda.stream(streams[n]):
                got[n].append(layers[n].run(*ins[n]))
    torch.cuda.synchronize()
    for n in (0, 1):
        for g in got[n]:
            for a, b in zip(g, alone[n]):
                assert torch.equal(a, b)


def test_results_do_not_change_from_run_to_run():
    layer = Layer(H=1024, F=512, E=64, k=8, groups=8, topk_groups=4)
    for T in (5, 3000):
        x, logits = layer.inputs(T, T)
        first = layer.run(x, logits)
        for _ in range(5):
            for a, b in zip(layer.run(x, logits), first):
                assert torch.equal(a, b)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
def test_gradients_of_the_layer(score, renormalize):
    """route -> dispatch -> y = a x + b per expert -> combine, loss <c, out>.  The
    kernels' chain of gradients against central differences of the 64-bit layer
    in the logits and in x.  Roundings: the expert outputs, their gradients and
    out are bf16 (2^-8 each); a difference with h = 1e-4 adds 1e-6."""
    T, H, E, k, h = 6, 64, 8, 3, 1e-4
    rng = np.random.default_rng(5)
    x = torch.from_numpy(rng.standard_normal((T, H), dtype=np.float32)).bfloat16()
    logits = rng.standard_normal((T, E)).astype(np.float32)
    c = torch.from_numpy(rng.standard_normal((T, H), dtype=np.float32)).bfloat16()
    a, b = rng.integers(1, 5, E) / 2.0, rng.integers(-2, 3, E) / 2.0
    ld = torch.from_numpy(logits).to(DEV)
    r = ep.ep_route(ld, k, score=score, renormalize=renormalize, scale=2.0)
    idx = r["topk_idx"]
    d = ep.ep_dispatch(x.to(DEV), idx, r["topk_weights"], E, 2)
    expert = torch.searchsorted(d["recv_expert_offset"][1:].long(), torch.arange(T * k, device=DEV), right=True)
    av, bv = (torch.from_numpy(v).to(DEV)[expert][:, None] for v in (a, b))
    y = (av * d["recv_x"].double() + bv).bfloat16()
    back = ep.ep_combine_backward(c.to(DEV), y, d["token_row"], r["topk_weights"])
    dl = ep.ep_route_backward(ld, idx, back["grad_topk_weights"], score=score, renormalize=renormalize, scale=2.0)
    dx = ep.ep_combine((av * back["grad_expert_out"].double()).bfloat16(), d["token_row"], None)
    ids, c64, x64 = idx.cpu().numpy(), c.double().numpy(), x.double().numpy()

    def loss(lv, xv):
        total = 0.0
        for t in range(T):
            s = plain64.scores(lv[t], score == "sigmoid")[ids[t]]
            w = 2.0 * (s / s.sum() if renormalize else s)
            for j in range(k):
                total += w[j] * float((c64[t] * (a[ids[t, j]] * xv[t] + b[ids[t, j]])).sum())
        return total

    l64 = logits.astype(np.float64)
    # |dL/dw| of a slot is off by 2^-8 of the sum of |c y| (y's rounding); the weights'
    # Jacobian has entries of at most 2 * 0.25 * 2 for each of k slots.
    slack = 2.0 ** -8 * max(float(np.abs(c64[t]).sum()) * float(np.abs(a).max() * np.abs(x64[t]).max() + 1) for t in range(T)) * k
    for t in range(T):
        for e in range(E):
            p, m = l64.copy(), l64.copy()
            p[t, e] += h
            m[t, e] -= h
            diff = (loss(p, x64) - loss(m, x64)) / (2 * h)
            assert abs(diff - float(dl[t, e])) <= slack
        for i in (0, 31, 63):
            p, m = x64.copy(), x64.copy()
            p[t, i] += h
            m[t, i] -= h
            diff = (loss(l64, p) - loss(l64, m)) / (2 * h)
            # Two roundings a row, each 2^-8 of a term, and that of the sum.
            assert abs(diff - float(dx[t, i])) <= 4 * 2.0 ** -8 * 2.0 * float(np.abs(c64[t, i])) * a.max() + 1e-6


def test_captured_gradients_beside_eager_ones():
    """The gradients captured into a graph and replayed, with eager calls on the
    same tensors between the replays."""
    T, H, E, k = 50, 128, 32, 4
    gen = torch.Generator().manual_seed(0)
    logits = torch.randn(T, E, generator=gen).to(DEV)
    x, g = (torch.randn(T, H, generator=gen).bfloat16().to(DEV) for _ in range(2))

    def run():
        r = ep.ep_route(logits, k)
        d = ep.ep_dispatch(x, r["topk_idx"], r["topk_weights"], E, 4)
        b = ep.ep_combine_backward(g, d["recv_x"], d["token_row"], r["topk_weights"])
        return b["grad_expert_out"], b["grad_topk_weights"], ep.ep_route_backward(logits, r["topk_idx"], b["grad_topk_weights"])

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = run()
    for seed in range(1, 5):
        fresh = torch.Generator().manual_seed(seed)
        logits.copy_(torch.randn(T, E, generator=fresh))
        eager = run()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(captured, eager):
            assert torch.equal(a, b)
