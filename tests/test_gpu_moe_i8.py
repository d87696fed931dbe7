"""ep_moe_i8 against the 64-bit form of plain64_i8.py, and the layer as larger batches run
it: dispatch, products, cast, products, combine.

Out is rounded to bf16, half a step (2^-8) of the value; what the roundings before it
make of it is plain64_i8.moe's bound.
"""
import numpy as np
import pytest
import torch

import plain64_i8 as plain
from combine_get_dispatch_02_amd import ep

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


class Layer:
    def __init__(self, H, F, E, seed=0):
        rng = np.random.default_rng([seed, H, F, E])
        self.H, self.F, self.E = H, F, E
        self.up = rng.integers(-127, 128, (E, 2 * F, H), dtype=np.int8)
        self.us = ((rng.random((E, 2 * F)) + 0.5) / (74 * H ** 0.5)).astype(np.float32)
        self.down = rng.integers(-127, 128, (E, H, F), dtype=np.int8)
        self.ds = ((rng.random((E, H)) + 0.5) / (74 * F ** 0.5)).astype(np.float32)
        self.dev = [torch.from_numpy(a).to(DEV) for a in (self.up, self.us, self.down, self.ds)]

    def inputs(self, T, k, seed=0, empty=0.1, experts=None):
        rng = np.random.default_rng([seed, T, k])
        x = torch.from_numpy(rng.standard_normal((T, self.H), dtype=np.float32)).bfloat16()
        idx = rng.integers(0, experts or self.E, (T, k))
        idx[rng.random((T, k)) < empty] = -1
        w = rng.random((T, k), dtype=np.float32)
        return x, idx, w

    def run(self, x, idx, w, **kw):
        return ep.ep_moe_i8(x.to(DEV), torch.from_numpy(idx).to(DEV), None if w is None else torch.from_numpy(w).to(DEV), *self.dev, **kw)

    def check(self, x, idx, w, got=None):
        print("[moe_i8]", self.H, self.F, self.E, idx.shape, flush=True)
        got = (self.run(x, idx, w) if got is None else got).double().cpu().numpy()
        ref, tol = plain.moe(x.double().numpy(), idx, w, self.up, self.us, self.down, self.ds)
        assert np.array_equal(np.isnan(got), np.isnan(ref))
        bad = np.abs(got - ref) > tol + 2.0 ** -8 * (np.abs(ref) + tol) + 2.0 ** -130
        assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], ref[bad][:5], tol[bad][:5])


@pytest.mark.parametrize("H,F,E", [(128, 128, 1), (128, 384, 8), (640, 128, 60), (1024, 512, 16), (4224, 256, 8), (256, 2176, 4),
                                   (1920, 128, 20), (2048, 256, 8), (2176, 128, 60)])
@pytest.mark.parametrize("T,k", [(1, 1), (1, 8), (3, 2), (16, 6), (64, 8)])
def test_layer(T, k, H, F, E):
    layer = Layer(H, F, E)
    layer.check(*layer.inputs(T, k))


@pytest.mark.parametrize("T,k", [(1, 8), (2, 3)])
def test_long_rows(T, k):
    layer = Layer(7168, 2048, 8)
    layer.check(*layer.inputs(T, k, empty=0))
    layer = Layer(128, 16384, 2)
    layer.check(*layer.inputs(T, k, empty=0))
    layer = Layer(16384, 128, 2)
    layer.check(*layer.inputs(T, k, empty=0))


def test_many_experts():
    layer = Layer(128, 128, 2048)
    layer.check(*layer.inputs(64, 8))
    layer.check(*layer.inputs(8, 64))


@pytest.mark.parametrize("T,k", [(64, 8), (8, 64), (512, 1), (100, 5)])
def test_all_slots_on_one_expert(T, k):
    """The same expert in every slot, and twice in a token."""
    layer = Layer(256, 256, 5)
    x, idx, w = layer.inputs(T, k, experts=1)
    layer.check(x, np.where(idx < 0, -1, 4), w)


def test_empty_slots_and_unit_weights():
    layer = Layer(384, 256, 8)
    x, idx, w = layer.inputs(6, 4)
    idx[2], idx[4, 1:] = -1, [8, 2 ** 40, -2 ** 40]                # outside [0, E): empty
    layer.check(x, idx, w)
    layer.check(x, idx, None)
    got = layer.run(x, np.full_like(idx, -1), w)
    assert (got == 0).all()
    assert (layer.run(x, idx, w)[2] == 0).all()


def test_rows_of_zeros_infinities_and_nan():
    layer = Layer(256, 128, 4)
    x, idx, w = layer.inputs(8, 2, empty=0)
    x[1] = 0
    x[3, 5], x[5, 200] = float("inf"), float("nan")
    got = layer.run(x, idx, w)
    assert torch.isnan(got[[3, 5]]).all() and (got[1] == 0).all()
    keep = [0, 1, 2, 4, 6, 7]
    layer.check(x[keep], idx[keep], w[keep], got[keep])
    w[0, 0], w[2, 1] = float("nan"), float("inf")
    got = layer.run(x, idx, w)
    assert torch.isnan(got[0]).all() and not torch.isfinite(got[2]).any()


def test_a_token_s_result_does_not_depend_on_the_batch():
    layer = Layer(512, 384, 16)
    x, idx, w = layer.inputs(64, 8)
    whole = layer.run(x, idx, w)
    for n in (1, 5, 33):
        assert torch.equal(layer.run(x[:n], idx[:n], w[:n]), whole[:n])
    for _ in range(3):
        assert torch.equal(layer.run(x, idx, w), whole)


def test_out_and_workspace_of_the_caller():
    layer = Layer(256, 128, 8)
    x, idx, w = layer.inputs(5, 3)
    n = ep.ep_moe_i8_workspace_bytes(5, 3, 128)
    assert n == 5 * 3 * (128 + 128 // 32) * 4
    ws = torch.full((n + 64,), 255, dtype=torch.uint8, device=DEV)
    room = torch.full((7, 256), 7.0, dtype=torch.bfloat16, device=DEV)
    got = layer.run(x, idx, w, out=room[1:6], workspace=ws[:n])
    assert got.data_ptr() == room[1:6].data_ptr()
    layer.check(x, idx, w, got)
    assert (room[0] == 7).all() and (room[6] == 7).all() and (ws[n:] == 255).all()


def test_offsets_past_32_bits():
    H, F, E = 4096, 1024, 600                                       # 5 GB of up rows, 2.5 GB of down rows
    small = Layer(H, F, 1)
    up = torch.zeros(E, 2 * F, H, dtype=torch.int8, device=DEV)
    us, down = torch.zeros(E, 2 * F, device=DEV), torch.zeros(1200, H, F, dtype=torch.int8, device=DEV)[:E]
    ds = torch.zeros(E, H, device=DEV)
    for big, one in zip((up, us, down, ds), small.dev):
        big[-1] = one[0]
    x, idx, w = small.inputs(3, 2, empty=0)
    want = small.run(x, idx, w)
    got = ep.ep_moe_i8(x.to(DEV), torch.from_numpy(idx + E - 1).to(DEV), torch.from_numpy(w).to(DEV), up, us, down, ds)
    assert torch.equal(got, want)


# ---- the layer of larger batches, each step from the one before ---------------------------


def chain(layer, x, idx, w, capacity=0):
    up, us, down, ds = layer.dev
    if capacity:
        d = ep.ep_dispatch_ll_i8(x, idx, w, layer.E, capacity)
        rows, to = d["recv_count"], d["token_slot"]
    else:
        d = ep.ep_dispatch_i8(x, idx, w, layer.E, 1)
        rows, to = d["recv_expert_offset"], d["token_row"]
    h = ep.ep_expert_linear_i8(d["recv_x_i8"], d["recv_scales"], rows, up, us, capacity=capacity, epilogue="silu_mul")
    q = ep.ep_quantize_i8(h, rows, capacity=capacity)
    y = ep.ep_expert_linear_i8(q["x_i8"], q["x_scales"], rows, down, ds, capacity=capacity)
    return d, rows, h, q, y, ep.ep_combine(y.view(-1, layer.H), to, w)


@pytest.mark.parametrize("T,k", [(1, 8), (60, 4), (500, 6)])
@pytest.mark.parametrize("padded", [False, True])
def test_chain(T, k, padded):
    layer = Layer(512, 256, 16)
    x, idx, w = layer.inputs(T, k)
    capacity = T * k if padded else 0
    idx_d, w_d = torch.from_numpy(idx).to(DEV), torch.from_numpy(w).to(DEV)
    d, rows, h, q, y, out = chain(layer, x.to(DEV), idx_d, w_d, capacity)
    flat = lambda t: t.reshape(-1, *t.shape[2 if capacity else 1:]).cpu()  # noqa: E731
    m = rows.cpu().numpy()
    spans = [(e * capacity, int(m[e])) if capacity else (int(m[e]), int(m[e + 1] - m[e])) for e in range(layer.E)]
    on = np.concatenate([np.arange(a, a + n) for a, n in spans])
    for got, a, s, wt, ws, silu in ((h, d["recv_x_i8"], d["recv_scales"], layer.up, layer.us, True),
                                    (y, q["x_i8"], q["x_scales"], layer.down, layer.ds, False)):
        ref, tol = plain.linear(flat(a).numpy(), flat(s).numpy(), spans, wt, ws, silu)
        got = flat(got).double().numpy()
        assert (np.abs(got - ref)[on] <= (tol + 2.0 ** -8 * (np.abs(ref) + tol))[on] + 2.0 ** -130).all()
    codes, scales = plain.cast(flat(h).double().numpy()[on])
    assert np.array_equal(flat(q["x_i8"]).numpy()[on], codes) and np.array_equal(flat(q["x_scales"]).numpy()[on], scales)
    # Against the layer: h and y are rounded to bf16 between the steps.  Half a step of
    # h (2^-8) moves a code by up to 127 / 256 and a rounding, so by one at most; with the
    # largest |h| (its own half step moves all codes alike) that is one scale and 2^-8 a
    # product at most, times the sum of the weights' magnitudes.
    ref, tol = plain.moe(x.double().numpy(), idx, w, layer.up, layer.us, layer.down, layer.ds)
    more = np.zeros_like(ref)
    xq, xs = plain.cast(x.double().numpy())
    for t in range(T):
        for j in range(k):
            e = idx[t, j]
            if e >= 0:
                hv, _ = plain.linear(xq[t:t + 1], xs[t:t + 1], [(0, 1)], layer.up[e:e + 1], layer.us[e:e + 1], True)
                a = np.abs(hv).max()
                each = np.abs(layer.down[e].astype(np.float64)).sum(axis=1) * layer.ds[e]
                yv = (np.abs(layer.down[e].astype(np.float64)) @ np.abs(hv[0])) * layer.ds[e]
                more[t] += w[t, j] * (1.01 * a / 127 * each + 3 * 2.0 ** -8 * yv)
    got = out.double().cpu().numpy()
    assert (np.abs(got - ref) <= tol + more + 2.0 ** -8 * (np.abs(ref) + tol + more)).all()


def both(layer, x, idx, w):
    return (ep.ep_moe_i8(x, idx, w, *layer.dev), chain(layer, x, idx, w)[-1], chain(layer, x, idx, w, 32)[-1])


def test_captured_layers_replay_with_other_inputs():
    layer, T, k = Layer(256, 128, 16), 40, 4
    x, idx, w = layer.inputs(T, k)
    x, idx, w = x.to(DEV), torch.from_numpy(idx).to(DEV), torch.from_numpy(w).to(DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        both(layer, x, idx, w)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = both(layer, x, idx, w)
    for seed in range(1, 6):
        x2, i2, w2 = layer.inputs(T, k, seed)
        x2, i2, w2 = x2.to(DEV), torch.from_numpy(i2).to(DEV), torch.from_numpy(w2).to(DEV)
        eager = both(layer, x2, i2, w2)
        x.copy_(x2)
        idx.copy_(i2)
        w.copy_(w2)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(captured, eager):
            assert torch.equal(a, b)


def test_two_layers_on_two_streams():
    layers = [Layer(256, 128, 16), Layer(1024, 256, 64, seed=1)]
    ins = []
    for la, (T, k) in zip(layers, ((60, 4), (64, 8))):
        x, idx, w = la.inputs(T, k)
        ins.append((x.to(DEV), torch.from_numpy(idx).to(DEV), torch.from_numpy(w).to(DEV)))
    alone = [both(la, *i) for la, i in zip(layers, ins)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    for _ in range(4):
        for n in (0, 1):
            with torch.cuda.stream(streams[n]):
                got[n].append(both(layers[n], *ins[n]))
    torch.cuda.synchronize()
    for n in (0, 1):
        for g in got[n]:
            for a, b in zip(g, alone[n]):
                assert torch.equal(a, b)
